"""Measured cases of the router, the residual RMS norm with 8-bit output, and the MXFP4 expert product.

Three operators of a routed MoE layer: `gate` (router logits -> expert ids and gates), `norm` (residual
addition + RMS norm -> the new residual stream, its normalised rows, and the same rows in 8 bits with one
power-of-two scale per 32 values) and `product` (bf16 rows -> microscaled 4-bit or 8-bit rows in routed
order -> the grouped product with microscaled 4-bit expert weights).  With `own` false `run` computes them
with elementary torch operations, with `own` true through grouped_sparse_gemm_b200.
"""
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gate(name, T, E, k, scoring, bias=False, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0,
          dtype="f32"):
    return {"op": "gate", "name": name, "T": T, "E": E, "k": k, "scoring": scoring, "bias": bias,
            "n_group": n_group, "topk_group": topk_group, "group_top": group_top, "renorm": renorm,
            "scale": scale, "dtype": dtype}


def _norm(name, T, K, residual, weight, y):
    return {"op": "norm", "name": name, "T": T, "K": K, "residual": residual, "weight": weight, "y": y}


def _product(name, E, N, K, T, k, fmt, zipf=0.0):
    return {"op": "product", "name": name, "E": E, "N": N, "K": K, "T": T, "k": k, "fmt": fmt, "zipf": zipf}


def listed():
    return [
        # one decoded token through a 384-expert router with a balance bias: pure latency
        _gate("gate_decode_1", 1, 384, 8, "sigmoid", bias=True, scale=2.5),
        # a 512-token prefill chunk over 128 experts, softmax scores renormalised, bf16 logits
        _gate("gate_30b_512", 512, 128, 8, "softmax", dtype="bf16"),
        # an odd-sized batch with group-limited choice (4 of 8 groups by their two best experts)
        _gate("gate_grouped_4099", 4099, 256, 8, "sigmoid", bias=True, n_group=8, topk_group=4, group_top=2,
              scale=2.5, dtype="bf16"),
        # the router of a large prefill: 65,536 tokens over 384 experts with a balance bias
        _gate("gate_1t_65536", 65536, 384, 8, "sigmoid", bias=True, scale=2.5),
        # one decoded token's row: the residual stream and its 8-bit form
        _norm("norm_decode_1", 1, 7168, "bf16", "bf16", False),
        # a 512-token chunk of the 30B-shaped model, bf16 rows for the router beside the 8-bit ones
        _norm("norm_30b_512", 512, 2048, "bf16", "bf16", True),
        # a large prefill of the 1T-shaped model with an fp32 residual stream
        _norm("norm_1t_8192", 8192, 7168, "f32", "f32", True),
        # smallest layer: 4 experts, 32 tokens, 4-bit rows
        _product("product_tiny", 4, 128, 256, 32, 2, 4),
        # 30B-shaped down-projection of 64 decoded tokens, 8-bit rows: a weight stream
        _product("product_30b_down_decode", 128, 2048, 768, 64, 8, 8),
        # 30B-shaped up-projection of a 512-token chunk, skewed routing, 4-bit rows
        _product("product_30b_up_prefill", 128, 1536, 2048, 512, 8, 4, zipf=1.0),
        # a shared expert's up-projection (one expert, every token), 8-bit rows, an odd token count
        _product("product_shared_1t_1023", 1, 4096, 7168, 1023, 1, 8),
        # 1T-shaped up-projection on 64 of its experts at the full batch's rows per expert, 4-bit rows
        _product("product_1t_up_e64", 64, 4096, 7168, 1368, 8, 4, zipf=1.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["gate", "norm", "product"])
    if op == "gate":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * _log_int(rng, 8, 512 // n_group)
        T = min(_log_int(rng, 1, 65536), 65536 * 384 // E)
        topk_group = 1 if n_group == 1 else rng.randint(1, n_group)
        k = min(rng.randint(1, 16), topk_group * E // n_group)
        c = _gate("", T, E, k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, n_group, topk_group,
                  rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.choice(["f32", "bf16"]))
    elif op == "norm":
        K = 256 * rng.randint(1, 64)
        T = min(_log_int(rng, 1, 65536), 8192 * 7168 // K)
        c = _norm("", T, K, rng.choice(["none", "bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    else:
        N, K = 128 * rng.randint(1, 32), 256 * rng.randint(1, 28)
        E = _log_int(rng, 1, 128)
        E = max(1, min(E, 64 * 4096 * 7168 // (N * K)))
        k = rng.randint(1, min(8, E))
        T = min(_log_int(rng, 1, 8192), 1368 * 8 // k)
        T = max(1, min(T, 1368 * 8 * 4096 * 7168 // (k * N * K)))
        c = _product("", E, N, K, T, k, rng.choice([4, 8]), rng.choice([0.0, 1.0]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _pow2(e):
    """Two to whole exponents in [-127, 127], exactly (a power function may be off by a unit)."""
    e = e.to(torch.int32)
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weights_mxfp4(g, E, N, K):
    """Microscaled 4-bit expert weights as checkpoints hold them: codes [E, N, K/2] (low nibble first)
    and power-of-two scales [E, N, K/32], of normally distributed weights."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    for e in range(E):
        b = (_randn(g, N, K) * 0.02).view(N, K // 32, 32)
        s = (torch.frexp(b.abs().amax(-1))[1] - 3).clamp(-127, 127)
        v = (b * _pow2(-s).unsqueeze(-1)).view(N, K)
        a = v.abs()
        c = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
        for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                         (5.0, False)):
            c += (a >= edge) if up else (a > edge)
        c |= torch.signbit(v).to(torch.uint8) << 3
        codes[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[e] = (s + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "gate":
        c["logits"] = _randn(g, c["T"], c["E"]).to(_DT[c["dtype"]])
        c["b"] = _randn(g, c["E"]) * 0.02 if c["bias"] else None
    elif c["op"] == "norm":
        T, K = c["T"], c["K"]
        spread = torch.ones(K, device="cuda")   # a few outlier channels, as trained models have
        spread[torch.randperm(K, generator=g, device="cuda")[: max(1, K // 128)]] = 20.0
        c["x"] = (_randn(g, T, K) * spread).to(torch.bfloat16)
        c["r"] = None if c["residual"] == "none" else (_randn(g, T, K) * spread * 2).to(_DT[c["residual"]])
        c["w"] = (1 + 0.1 * _randn(g, K)).to(_DT[c["weight"]])
    else:
        E, T, k = c["E"], c["T"], c["k"]
        spread = torch.ones(c["K"], device="cuda")
        spread[torch.randperm(c["K"], generator=g, device="cuda")[: max(1, c["K"] // 128)]] = 20.0
        c["x"] = (_randn(g, T, c["K"]) * spread).to(torch.bfloat16)
        p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).pow(-c["zipf"])
        p = p[torch.randperm(E, generator=g, device="cuda")]
        ids = torch.multinomial(p.expand(T, E), k, generator=g).reshape(-1)
        perm = torch.sort(ids, stable=True)[1]
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(T * k, device="cuda")
        counts = torch.bincount(ids, minlength=E)
        c["token"] = perm // k
        c["inv"] = inv.to(torch.int32)
        c["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        c["counts"] = counts.tolist()   # the histogram of the routing, as a batch scheduler reads it
        c["most"] = max(c["counts"])
        c["codes"], c["scales"] = _weights_mxfp4(g, E, c["N"], c["K"])
        if own:   # the model's weights in the product's layout, once when it is loaded
            import grouped_sparse_gemm_b200 as gsg
            c["packed"] = gsg.pack_mxfp4_codes(c.pop("codes"), c.pop("scales"))
    return c


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import grouped_sparse_gemm_b200 as gsg
        if s["op"] == "gate":
            return gsg.moe_gate(s["logits"], s["k"], scoring=s["scoring"], bias=s["b"], n_group=s["n_group"],
                                topk_group=s["topk_group"], group_top=s["group_top"], renormalize=s["renorm"],
                                scale=s["scale"])
        if s["op"] == "norm":
            n = gsg.add_rmsnorm_mx(s["x"], s["w"], residual=s["r"], eps=1e-6, fmt=8, want_y=s["y"])
            return {"h": n.h, "y": n.y, "codes": n.act.codes.view(torch.float8_e4m3fn),
                    "scales": n.act.scales.view(torch.float8_e8m0fnu)}
        act = gsg.quantize_act_mx(s["x"], s["fmt"], inv_perm=s["inv"], top_k=s["k"])
        return gsg.grouped_mx_gemm(act, s["packed"], s["offsets"], max_rows_per_expert=s["most"])
    return {"gate": _run_gate, "norm": _run_norm, "product": _run_product}[s["op"]](s)


def _run_gate(s):
    x, b, k, G = s["logits"].float(), s["b"], s["k"], s["n_group"]
    T, E = x.shape
    x = x.double()   # scores next to one another decide the ids
    score = torch.exp(x - x.amax(-1, keepdim=True)) if s["scoring"] == "softmax" else 1 / (1 + torch.exp(-x))
    if s["scoring"] == "softmax":
        score = score / score.sum(-1, keepdim=True)
    choice = score if b is None else score + b.double()
    if b is None and s["group_top"] == 1:
        choice = x
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=-1, descending=True)[0][..., : s["group_top"]].sum(-1)
        keep = torch.sort(best, dim=-1, descending=True, stable=True)[1][:, : s["topk_group"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, keep, True)
        choice = torch.where(open_.repeat_interleave(E // G, dim=1), choice, float("-inf"))
    ids = torch.sort(choice, dim=-1, descending=True, stable=True)[1][:, :k]
    gates = torch.gather(score, 1, ids)
    if s["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    return ids.to(torch.int32), (gates * s["scale"]).float()


def _block_scale(v, emax):
    """Exponents [..., K/32] of the blocks of 32 values and the values divided by two to that power."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127), -127)
    return e, (b * _pow2(-e).unsqueeze(-1)).flatten(-2)


def _e2m1(v):
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _quad(e):
    """Scale exponents [T, K/32] as the product reads them: [K/128, T, 4, 4], entry (kb, r, c, j) the
    scale of block 4 kb + j of row r + 32 c, zero bytes past the last row."""
    T, nb = e.shape
    rows = torch.zeros(T + 96, nb, dtype=torch.uint8, device=e.device)
    rows[:T] = (e + 127).to(torch.uint8)
    rows = rows.view(T + 96, nb // 4, 4).transpose(0, 1)
    return torch.stack([rows[:, 32 * c: 32 * c + T] for c in range(4)], dim=2).reshape(-1)


def _run_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = (h + s["r"].float()).to(s["r"].dtype).float()
    ms = h.double().square().mean(-1, keepdim=True)
    y = h * torch.rsqrt(ms + 1e-6).float() * s["w"].float()
    e, v = _block_scale(y, 8)
    return {"h": h.to(s["r"].dtype) if s["r"] is not None else None, "y": y.to(torch.bfloat16) if s["y"] else None,
            "codes": v.clamp(-448, 448).to(torch.float8_e4m3fn), "scales": _quad(e).view(torch.float8_e8m0fnu)}


def _run_product(s):
    x = s["x"].float()
    e, v = _block_scale(x, 8 if s["fmt"] == 8 else 2)
    v = v.clamp(-448, 448).to(torch.float8_e4m3fn).float() if s["fmt"] == 8 else _e2m1(v)
    a = (v.unflatten(-1, (-1, 32)) * _pow2(e).unsqueeze(-1)).flatten(-2)[s["token"]]
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    value = torch.cat([half, -half])
    out = torch.empty(a.shape[0], s["N"], dtype=torch.bfloat16, device=x.device)
    at = 0
    for n, codes, scales in zip(s["counts"], s["codes"], s["scales"]):   # one product for each expert
        if n:
            w = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1).view(s["N"], -1, 32)
            w = (w * _pow2(scales.int() - 127).unsqueeze(-1)).view(s["N"], -1)
            out[at: at + n] = (a[at: at + n] @ w.T).to(torch.bfloat16)
            at += n
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * (4 if c["dtype"] == "f32" else 2) + 8 * T * k + (4 * E if c["bias"] else 0),
                "flops": 2 * T * E}
    if c["op"] == "norm":
        n, res = c["T"] * c["K"], {"none": 0, "bf16": 2, "f32": 4}[c["residual"]]
        return {"bytes": n * (2 + 2 * res + (2 if c["y"] else 0) + 1) + n // 32
                + c["K"] * (2 if c["weight"] == "bf16" else 4), "flops": 6 * n}
    rows = c["T"] * c["k"]
    touched = min(c["E"], rows)
    if c["k"] < c["E"]:   # experts that a uniform routing of this many tokens is expected to reach
        touched = min(touched, c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"]))
    return {"bytes": 2 * c["T"] * c["K"] + touched * c["N"] * c["K"] * 17 / 32 + 2 * rows * c["N"],
            "flops": 2 * rows * c["N"] * c["K"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_to(v, mantissa, emin, most):
    """v to the nearest number with `mantissa` bits after the leading one, ties to even, of at most `most`."""
    e = torch.frexp(v)[1].clamp(min=emin + 1) - 1
    step = _two_to(e - mantissa)
    return (torch.round(v / step) * step).clamp(-most, most)


def _mx64(v, fmt):
    """v [..., K] in blocks of 32: (values over their scale, exponents), in 64 bits."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, (torch.frexp(top)[1] - (9 if fmt == 8 else 3)).clamp(-127, 127), -127)
    q = b / _two_to(e).unsqueeze(-1)
    return (_round_to(q, 3, -6, 448.0) if fmt == 8 else _round_to(q, 1, 0, 6.0)), e


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if s["op"] == "gate":
        x = s["logits"].double()
        p = torch.softmax(x, -1) if s["scoring"] == "softmax" else torch.sigmoid(x)
        c = x if s["b"] is None and s["group_top"] == 1 else p + (0 if s["b"] is None else s["b"].double())
        G, size = s["n_group"], s["E"] // s["n_group"]
        order = lambda v, n: torch.argsort(v, dim=1, descending=True, stable=True)[:, :n]  # noqa: E731
        if G > 1:
            tops = torch.stack([torch.topk(c[:, g * size: (g + 1) * size], s["group_top"], dim=1)[0].sum(1)
                                for g in range(G)], 1)
            group = torch.arange(s["E"], device=x.device) // size
            c = c.masked_fill(~(order(tops, s["topk_group"]).unsqueeze(-1) == group).any(1), float("-inf"))
        ids = order(c, s["k"])
        w = p.gather(1, ids)
        w = w / w.sum(1, keepdim=True) if s["renorm"] else w
        return ids.to(torch.int32), w * s["scale"]
    if s["op"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(s["r"].dtype).double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["w"].double()
        q, e = _mx64(y, 8)
        T, K = y.shape
        at = torch.arange(T, device=y.device).view(1, -1, 1, 1) + 32 * torch.arange(4, device=y.device).view(1, 1, 4, 1)
        block = 4 * torch.arange(K // 128, device=y.device).view(-1, 1, 1, 1) + torch.arange(4, device=y.device)
        scales = torch.where(at < T, _two_to(e)[at.clamp(max=T - 1), block], 2.0 ** -127)
        return {"h": h if s["r"] is not None else None, "y": y if s["y"] else None, "codes": q.reshape(T, K),
                "scales": scales.reshape(-1)}
    q, e = _mx64(s["x"].double(), s["fmt"])
    a = (q * _two_to(e).unsqueeze(-1)).reshape(s["T"], s["K"])
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=a.device) / 2
    Y, lo = [], 0
    for i, n in enumerate(s["counts"]):
        if n == 0:
            continue
        nib = torch.stack([s["codes"][i] % 16, s["codes"][i] // 16], -1).long()
        w = grid[nib % 8] * (1 - 2 * (nib // 8))
        w = w.reshape(s["N"], -1, 32) * _two_to(s["scales"][i].int() - 127).unsqueeze(-1)
        Y.append(a[s["token"][lo: lo + n]] @ w.reshape(s["N"], s["K"]).T)
        lo += n
    return torch.cat(Y)
