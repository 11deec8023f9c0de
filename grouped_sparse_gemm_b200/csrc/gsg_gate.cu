// gsg_gate.cu -- the router: logits -> the k experts of every token and their gates.
//
// For a token with logits x[e], score s[e] = softmax(x)[e] or 1 / (1 + exp(-x[e])), choice
// c[e] = s[e] + bias[e]; an expert whose logit or bias is -inf is unavailable (c = -inf).  With groups,
// the experts of all but the topk_group best groups (by the sum of their group_top largest c) are
// unavailable too.  The k largest c in descending order, ties to the lowest index, are the token's
// experts; its gates are their scores (0 for an unavailable one), divided by their sum when renormalised.
//
// The choice is that of exact arithmetic: where it only needs the order of the logits (no bias, groups
// by their best expert) the kernel compares those, and elsewhere it compares fp32 scores and settles every
// comparison closer than their error bound in 64 bits.  Equal logits with equal biases are equal scores,
// so they need no second look.
//
// One warp per token, expert e in register e / 32 of lane e % 32.
#include "gsg_internal.cuh"
#include "gsg_launch.h"

namespace gsg {

struct GateParams {
  const void* logits;   // [T][E]
  const float* bias;    // [E] or nullptr
  int T, E, k;
  int sigmoid;          // scoring
  int by_score;         // the choice needs scores (a bias, or groups by the sum of two)
  int n_group, topk_group, group_top, group_size;
  uint32_t group_magic; // e / group_size = e * magic >> 20 for e < 1024
  int renorm;
  float scale;
  int32_t* ids;
  float* gates;
  int* status;
};

constexpr int kGateWarps = 4;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }
// Order-preserving unsigned key of a float (no NaN); -0 counts as +0.  Every key is above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u ^ ((u >> 31) != 0u ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) != 0u ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ unsigned long long order_key(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(__dadd_rn(v, 0.0));
  return u ^ ((u >> 63) != 0ull ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (unsigned long long)hi << 32 | lo;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T>
__device__ __forceinline__ float load_logit(const void* p, size_t i);
template <>
__device__ __forceinline__ float load_logit<float>(const void* p, size_t i) {
  return __ldg(static_cast<const float*>(p) + i);
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const void* p, size_t i) {
  return bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p) + i));
}

__device__ __forceinline__ float bias_of(const GateParams& p, int e) {
  return p.bias != nullptr ? __ldg(p.bias + e) : 0.0f;
}

// Choice of one expert in 32 bits; softmax: mx the row's largest logit, inv_sum its denominator.
__device__ __forceinline__ float choice32(const GateParams& p, float mx, float inv_sum, float x, float b) {
  if (x == neg_inf() || b == neg_inf()) return neg_inf();
  if (!p.by_score) return x;
  const float s = p.sigmoid ? __fdividef(1.0f, __fadd_rn(1.0f, __expf(-x)))
                            : __fmul_rn(__expf(__fsub_rn(x, mx)), inv_sum);
  return __fadd_rn(s, b);
}

// Choice of expert e: from the warp's shared row, or evaluated in 64 bits from the logits.
struct SharedChoice {
  const float* sh;
  __device__ __forceinline__ float operator()(int e) const { return sh[e]; }
};
template <typename T>
struct ExactChoice {
  const GateParams& p;
  size_t row;
  double mx, inv_sum;   // softmax: the row's largest logit and 1 / its denominator
  __device__ __forceinline__ float logit(int e) const {   // NaN or +inf: unavailable
    const float x = load_logit<T>(p.logits, row + e);
    return x < INFINITY && bias_of(p, e) < INFINITY ? x : neg_inf();
  }
  __device__ __forceinline__ double operator()(int e) const {
    const double x = (double)logit(e), b = (double)bias_of(p, e);
    const double q = exp(p.sigmoid ? -x : x - mx);
    const double c = (p.sigmoid ? 1.0 / (1.0 + q) : q * inv_sum) + b;
    return x > -INFINITY && b > -INFINITY ? c : -INFINITY;
  }
};

// Group scores: lanes_per_group lanes walk a group's choices (value(e)), then merge their two largest.
template <typename V, typename F>
__device__ __forceinline__ V group_score(const GateParams& p, int lane, int lpg, F value) {
  const int g = lane / lpg, sub = lane % lpg;
  V a = -INFINITY, b = -INFINITY;   // the two largest
  if (g < p.n_group)
    for (int j = sub; j < p.group_size; j += lpg) {
      const V v = value(g * p.group_size + j);
      b = v > a ? a : (v > b ? v : b);
      a = v > a ? v : a;
    }
  for (int o = 1; o < lpg; o <<= 1) {
    const V a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
    const V lo = a < a2 ? a : a2;
    a = a > a2 ? a : a2;
    b = b > b2 ? b : b2;
    b = b > lo ? b : lo;
  }
  return p.group_top == 2 ? a + b : a;
}

// Bit g set: group g is among the topk_group best (ties to the lowest index).  tol >= 0: *close is set
// when a kept and a dropped group are no further apart than that.
template <typename V>
__device__ __forceinline__ uint32_t keep_groups(const GateParams& p, int lane, int lpg, V score, V tol, bool* close) {
  const int g = lane / lpg;
  int rank = 0;
  for (int o = 0; o < p.n_group; ++o) {
    const V v = __shfl_sync(0xffffffffu, score, o * lpg);
    rank += (v > score || (v == score && o < g)) ? 1 : 0;
  }
  const bool leader = g < p.n_group && lane % lpg == 0;
  const uint32_t kept = __ballot_sync(0xffffffffu, leader && rank < p.topk_group);
  bool near = false;
  for (int o = 0; o < p.n_group; ++o) {
    const V v = __shfl_sync(0xffffffffu, score, o * lpg);
    const bool o_kept = (kept >> (o * lpg)) & 1u;
    if (leader && o_kept != (rank < p.topk_group)) near |= v > -INFINITY && !(fabs(v - score) > tol);
  }
  *close = __any_sync(0xffffffffu, near);
  uint32_t bits = 0;
  for (int o = 0; o < p.n_group; ++o) bits |= ((kept >> (o * lpg)) & 1u) << o;
  return bits;
}

template <typename T, int NV>
__global__ void __launch_bounds__(32 * kGateWarps)
moe_gate_kernel(const GateParams p) {
  extern __shared__ float gate_sh[];   // with groups: the choices of each warp's token, [kGateWarps][E]
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kGateWarps + warp;
  if (t >= p.T) return;
  float x[NV];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    x[i] = e < p.E ? load_logit<T>(p.logits, (size_t)t * p.E + e) : neg_inf();
  }
  float mx = neg_inf();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    const float b = e < p.E ? bias_of(p, e) : 0.0f;
    // NaN or +inf: an error; the expert counts as unavailable
    if (!(x[i] < INFINITY) || !(b < INFINITY)) { bad = true; x[i] = neg_inf(); }
    mx = fmaxf(mx, x[i]);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, GSG_ERR_NONFINITE);
  mx = warp_max(mx);
  // softmax denominator, where the scores (not only the chosen experts' ratios) are needed
  float inv_sum = 0.0f;
  if (!p.sigmoid && (p.by_score || !p.renorm) && mx > neg_inf()) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s = __fadd_rn(s, __expf(__fsub_rn(x[i], mx)));
    inv_sum = __frcp_rn(warp_sum(s));
  }
  // choices as keys; 0 = no such expert, or taken
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    key[i] = e < p.E ? order_key(choice32(p, mx, inv_sum, x[i], bias_of(p, e))) : 0u;
  }
  // how far apart two fp32 choices have to be for their order to be certain: twice the error of a
  // score (at most 1, its exponential and quotient good to 2^-21; a softmax denominator of E terms to
  // 2^-18) and of the sum with the bias
  const float tol1 = p.sigmoid ? 0x1p-19f : 0x1p-17f;
  bool close = false;
  uint32_t kept = 0xFFFFFFFFu;
  const int lpg = p.n_group > 16 ? 1 : p.n_group > 8 ? 2 : p.n_group > 4 ? 4 : p.n_group > 2 ? 8 : 16;
  float* sh = gate_sh + (size_t)warp * p.E;
  if (p.n_group > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (32 * i + lane < p.E) sh[32 * i + lane] = key_value(key[i]);
    __syncwarp();
    const float score = group_score<float>(p, lane, lpg, SharedChoice{sh});
    kept = keep_groups<float>(p, lane, lpg, score, p.by_score ? __fmaf_rn(fabsf(score), 0x1p-20f, 2.0f * tol1) : -1.0f, &close);
    if (!p.by_score) close = false;
    if (!close) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t e = 32 * i + lane;
        if (key[i] != 0u && !((kept >> ((e * p.group_magic) >> 20)) & 1u)) key[i] = order_key(neg_inf());
      }
    }
  }
  // k rounds of the largest choice
  int my_id = 0;
  float my_x = neg_inf();     // the logit of the expert that this lane (j < k) reports; -inf: unavailable
  if (!close) {
    uint32_t taken = 0u;      // bit i: this lane's register i
    for (int j = 0; j < p.k; ++j) {
      uint32_t m = 0u;
      int mi = 0;
      float mxv = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t ki = (taken >> i) & 1u ? 0u : key[i];
        if (ki > m) { m = ki; mi = i; mxv = x[i]; }
      }
      const uint32_t best = __reduce_max_sync(0xffffffffu, m);
      const uint32_t e = __reduce_min_sync(0xffffffffu, m == best ? (uint32_t)(32 * mi + lane) : 0xFFFFFFFFu);
      const float c = key_value(best);
      const float xw = __shfl_sync(0xffffffffu, mxv, (int)(e & 31u));
      if ((e & 31u) == (uint32_t)lane) taken |= 1u << (e >> 5);
      if (lane == j) { my_id = (int)e; my_x = c == neg_inf() ? c : xw; }
      if (p.by_score && c > neg_inf()) {
        // another expert within the error bound, other than by the same logit and bias
        const float lim = __fsub_rn(c, __fmaf_rn(fabsf(c), 0x1p-21f, tol1));
        bool near = false;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (!((taken >> i) & 1u) && key[i] > order_key(neg_inf()) && key_value(key[i]) >= lim)
            near |= x[i] != xw || bias_of(p, 32 * i + lane) != bias_of(p, (int)e);
        if (__any_sync(0xffffffffu, near)) { close = true; break; }
      }
    }
  }
  if (close) {
    // the same in 64 bits: rare, so the logits are read again and the choices evaluated where they are
    // compared, which keeps this path's registers out of the usual one's
    ExactChoice<T> choice = {p, (size_t)t * p.E, (double)mx, 0.0};
    if (!p.sigmoid) {
      double s = 0.0;
#pragma unroll 1
      for (int e = lane; e < p.E; e += 32) s += exp((double)choice.logit(e) - choice.mx);
      choice.inv_sum = 1.0 / warp_sum(s);
    }
    kept = 0xFFFFFFFFu;
    if (p.n_group > 1) {
      const double score = group_score<double>(p, lane, lpg, choice);
      bool unused;
      kept = keep_groups<double>(p, lane, lpg, score, -1.0, &unused);
    }
    uint32_t taken = 0u;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
      unsigned long long m = 0ull;
      int me = 0;
#pragma unroll 1
      for (int e = lane; e < p.E; e += 32) {
        if ((taken >> (e >> 5)) & 1u) continue;
        const bool open = p.n_group <= 1 || ((kept >> (((uint32_t)e * p.group_magic) >> 20)) & 1u);
        const unsigned long long ke = order_key(open ? choice(e) : -INFINITY);
        if (ke > m) { m = ke; me = e; }
      }
      const unsigned long long best = warp_max_u64(m);
      const uint32_t e = __reduce_min_sync(0xffffffffu, m == best ? (uint32_t)me : 0xFFFFFFFFu);
      if ((e & 31u) == (uint32_t)lane) taken |= 1u << (e >> 5);
      if (lane == j) {
        my_id = (int)e;
        my_x = best == order_key(-(double)INFINITY) ? neg_inf() : choice.logit((int)e);
      }
    }
  }
  // gates of the chosen experts.  Renormalised ones are ratios of scores, so a common factor may go:
  // exp(x - max of the chosen) for softmax; for the sigmoid exp(x - m) / (1 + exp(x)), m = min(0, that max),
  // which keeps scores that would underflow apart.
  const float mc = warp_max(lane < p.k ? my_x : neg_inf());
  float g = 0.0f;
  if (lane < p.k && my_x > neg_inf()) {
    if (p.sigmoid) {
      const float m = p.renorm ? fminf(mc, 0.0f) : 0.0f;
      g = my_x > 0.0f ? __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-my_x)))
                      : __fdiv_rn(expf(__fsub_rn(my_x, m)), __fadd_rn(1.0f, expf(my_x)));
    } else {
      g = p.renorm ? expf(__fsub_rn(my_x, mc)) : __fmul_rn(expf(__fsub_rn(my_x, mx)), inv_sum);
    }
  }
  if (p.renorm) {
    const float sum = warp_sum(g);
    g = sum > 0.0f ? __fdiv_rn(g, sum) : 0.0f;
  }
  if (lane < p.k) {
    p.ids[(size_t)t * p.k + lane] = my_id;
    p.gates[(size_t)t * p.k + lane] = __fmul_rn(g, p.scale);
  }
}

template <typename T, int NV>
static cudaError_t launch_gate_nv(const GateParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)((p.T + kGateWarps - 1) / kGateWarps);
  const size_t sh = p.n_group > 1 ? (size_t)kGateWarps * p.E * sizeof(float) : 0;
  return launch_pdl(moe_gate_kernel<T, NV>, grid, 32 * kGateWarps, sh, stream, p);
}

template <typename T>
static cudaError_t launch_gate_t(const GateParams& p, cudaStream_t stream) {
  const int nv = (p.E + 31) / 32;
  if (nv <= 2) return launch_gate_nv<T, 2>(p, stream);
  if (nv <= 4) return launch_gate_nv<T, 4>(p, stream);
  if (nv <= 8) return launch_gate_nv<T, 8>(p, stream);
  if (nv <= 12) return launch_gate_nv<T, 12>(p, stream);
  if (nv <= 16) return launch_gate_nv<T, 16>(p, stream);
  return launch_gate_nv<T, 32>(p, stream);
}

cudaError_t launch_gate(const void* logits, bool f32, const float* bias, int T, int E, int k, bool sigmoid, int n_group,
                        int topk_group, int group_top, bool renorm, float scale, int32_t* ids, float* gates,
                        int* status, cudaStream_t stream) {
  GateParams p;
  p.logits = logits; p.bias = bias; p.T = T; p.E = E; p.k = k;
  p.sigmoid = sigmoid; p.by_score = bias != nullptr || (n_group > 1 && group_top == 2);
  p.n_group = n_group; p.topk_group = topk_group; p.group_top = group_top; p.group_size = E / n_group;
  p.group_magic = (uint32_t)(((1u << 20) + p.group_size - 1) / p.group_size);
  p.renorm = renorm; p.scale = scale; p.ids = ids; p.gates = gates; p.status = status;
  return f32 ? launch_gate_t<float>(p, stream) : launch_gate_t<uint16_t>(p, stream);
}

}  // namespace gsg
