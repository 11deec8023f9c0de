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
// One warp per token, expert e in register e / 32 of lane e % 32.  The k-th largest of the 32 lanes' maxima (a
// warp-wide sort) is no more than the k-th largest choice, so the few experts that come up to it (less the error
// bound) hold the answer: they are gathered, one to a lane, and ranked by counting, in 64 bits where two are
// close.  Large batches are bound by instructions issued, about 620 a token (70 % of the issue slots): 65,536
// tokens x 384 experts 55 us = 1.9 TB/s (k rounds of a warp-wide maximum instead: 257 us).  One token: 3.1 us, launch.
#include "gsg_internal.cuh"
#include "gsg_launch.h"

namespace gsg {

struct GateParams {
  const void* logits;   // [T][E]
  const float* bias;    // [E] or nullptr
  int T, E, k;
  int sigmoid;          // scoring: 1 sigmoid, 0 softmax
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
// blocks per SM (registers: 64, 72, 128 and 168 a thread)
constexpr int gate_blocks(int nv) { return nv <= 8 ? 8 : nv <= 12 ? 7 : nv <= 16 ? 4 : 3; }

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
  return __ldca(static_cast<const float*>(p) + i);
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const void* p, size_t i) {
  return bf16_bits_to_f32(__ldca(static_cast<const uint16_t*>(p) + i));
}

// The same where lane < left, else the lowest number (a predicated load: a branch costs several times more).
template <typename T>
__device__ __forceinline__ float load_logit_if(const T* p, int lane, int left);
template <>
__device__ __forceinline__ float load_logit_if<float>(const float* p, int lane, int left) {
  float v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.lt.s32 q, %2, %3;\n\tmov.b32 %0, 0xFF7FFFFF;\n\t@q ld.global.f32 %0, [%1];\n\t}"
      : "=f"(v) : "l"(p), "r"(lane), "r"(left));
  return v;
}
template <>
__device__ __forceinline__ float load_logit_if<uint16_t>(const uint16_t* p, int lane, int left) {
  uint16_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.lt.s32 q, %2, %3;\n\tmov.b16 %0, 0xFF7F;\n\t@q ld.global.u16 %0, [%1];\n\t}"
      : "=h"(v) : "l"(p), "r"(lane), "r"(left));
  return bf16_bits_to_f32(v);
}

template <typename T>
__device__ __forceinline__ float lowest_logit() { return __uint_as_float(sizeof(T) == 4 ? 0xFF7FFFFFu : 0xFF7F0000u); }

__device__ __forceinline__ float bias_of(const GateParams& p, int e) {
  return p.bias != nullptr ? __ldca(p.bias + e) : 0.0f;
}

// Scores in 32 bits; softmax: mx the row's largest logit, inv_sum 1 / its denominator.  Two hardware
// approximations each (2^x and 1 / x, results below the normal range flushed): see order_margin.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmul_rn(x, 1.44269504f)));
  return r;
}
__device__ __forceinline__ float score_sigmoid(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, fast_exp(-x))));
  return r;
}
__device__ __forceinline__ float score_softmax(float x, float mx, float inv_sum) {
  return __fmul_rn(fast_exp(__fsub_rn(x, mx)), inv_sum);
}
// Is expert e in one of the kept groups?
__device__ __forceinline__ bool group_open(const GateParams& p, uint32_t kept, int e) {
  return (kept >> (((uint32_t)e * p.group_magic) >> 20)) & 1u;
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
  __device__ __forceinline__ float raw_logit(int e) const {    // NaN and +inf: unavailable
    const float x = load_logit<T>(p.logits, row + e);
    return x < INFINITY ? x : neg_inf();
  }
  __device__ __forceinline__ float clean_bias(int e) const {
    const float b = bias_of(p, e);
    return b < INFINITY ? b : neg_inf();
  }
  __device__ __forceinline__ double operator()(int e) const {
    const double x = (double)raw_logit(e), b = (double)clean_bias(e);
    const double q = exp(p.sigmoid ? -x : x - mx);
    const double c = (p.sigmoid ? 1.0 / (1.0 + q) : q * inv_sum) + b;
    return x > -INFINITY && b > -INFINITY ? c : -INFINITY;
  }
};

// Group scores: lanes_per_group lanes walk a group's choices (value(e)), then merge their two largest.
// size: the sum of the terms' magnitudes, which the error of the score goes by.
template <typename V, typename F>
__device__ __forceinline__ V group_score(const GateParams& p, int lane, int lpg, F value, V* size) {
  const int g = lane / lpg, sub = lane % lpg;
  V a = -INFINITY, b = -INFINITY;   // the two largest
  if (g < p.n_group)
    for (int j = sub; j < p.group_size; j += lpg) {
      // (each group starts lpg further on than the one before: other banks where the size is a multiple of 32)
      int at = j + g * lpg % p.group_size;
      at = at < p.group_size ? at : at - p.group_size;
      const V v = value(g * p.group_size + at);
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
  *size = p.group_top == 2 ? fabs(a) + fabs(b) : fabs(a);
  const V sum = p.group_top == 2 ? a + b : a;
  // (a sum below the range is the lowest number, for -inf is a group without group_top available experts)
  return sum == -INFINITY && b > -INFINITY ? (V)-3.402823466e38f : sum;
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

// The order in 64 bits of the choices that lanes < n hold one each: this lane's rank.
__device__ __forceinline__ int exact_rank(double v, int e, int n) {
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(0xffffffffu, v, j);
    const int oe = __shfl_sync(0xffffffffu, e, j);
    rank += (o > v || (o == v && oe < e)) ? 1 : 0;
  }
  return rank;
}

// Two fp32 choices this far apart are in their true order.  Twice the error of one: a sigmoid from the fast
// exponential (2 + 1.16 |x| units, times s (1 - s)) and quotient (2 units) is within 2^-21.3; a softmax score
// within 2^-18.4 of itself (a denominator of 1024 terms, at most 37 additions in a row) and at most 1 / the
// denominator; the sum with the bias within half a unit of c.
__device__ __forceinline__ float order_margin(float tol, float c) { return __fmaf_rn(fabsf(c), 0x1p-22f, tol); }

template <typename T, int NV>
__global__ void __launch_bounds__(32 * kGateWarps, gate_blocks(NV))
moe_gate_kernel(const GateParams p) {
  extern __shared__ float gate_sh[];   // with groups: the choices of each warp's token, [kGateWarps][E]
  __shared__ int cand_sh[kGateWarps][32];
  __shared__ unsigned long long key_sh[kGateWarps][32];
  __shared__ float sort_sh[kGateWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lpg = p.n_group > 16 ? 1 : p.n_group > 8 ? 2 : p.n_group > 4 ? 4 : p.n_group > 2 ? 8 : 16;
  float* sh = gate_sh + (size_t)warp * p.E;
  float b[NV];   // the biases; -inf: no such expert, or never available
  uint32_t there = 0u;   // bit i: expert 32 i + lane exists
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    if (e < p.E) there |= 1u << i;
    b[i] = e < p.E ? bias_of(p, e) : neg_inf();
    if (!(b[i] < INFINITY)) { bad = true; b[i] = neg_inf(); }
  }
  for (unsigned t = blockIdx.x * kGateWarps + warp; t < (unsigned)p.T; t += gridDim.x * kGateWarps) {
    const size_t row = (size_t)t * p.E;
    float c[NV];   // the logits, then the choices (experts that do not exist: the lowest number, until the bias)
    float probe = 0.0f, mx = neg_inf();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      c[i] = load_logit_if<T>(static_cast<const T*>(p.logits) + row + lane + 32 * i, lane, p.E - 32 * i);
#pragma unroll
    for (int i = 0; i < NV; ++i) probe = __fmaf_rn(c[i], 0.0f, probe);
    // bit i: expert 32 i + lane is unavailable by its logit (NaN and +inf are errors)
    uint32_t closed = 0u;
    if (__any_sync(0xffffffffu, probe != 0.0f)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!(c[i] < INFINITY)) { bad = true; c[i] = neg_inf(); }
        if (!((there >> i) & 1u)) c[i] = neg_inf();
        if (c[i] == neg_inf()) closed |= 1u << i;
      }
    }
    float inv_sum = 0.0f;
    if (!p.sigmoid) {
#pragma unroll
      for (int i = 0; i < NV; ++i) mx = fmaxf(mx, c[i]);
      mx = warp_max(mx);
      // the denominator, where the scores (not only the chosen experts' ratios) are needed
      if ((p.by_score || !p.renorm) && mx > neg_inf()) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) s = __fadd_rn(s, fast_exp(__fsub_rn(c[i], mx)));
        // (a row of the lowest number throughout: what stands for missing experts counted as much as they do, 1 each)
        if (mx == lowest_logit<T>()) s -= (float)__popc(~(there | closed) & (0xFFFFFFFFu >> (32 - NV)));
        inv_sum = __frcp_rn(warp_sum(s));
      }
    }
    const float tol = !p.by_score ? 0.0f : p.sigmoid ? 0x1p-20f : __fmul_rn(inv_sum, 0x1p-17f);
    if (p.by_score) {
      if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = __fadd_rn(score_sigmoid(c[i]), b[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = __fadd_rn(score_softmax(c[i], mx, inv_sum), b[i]);
      }
      if (__any_sync(0xffffffffu, closed != 0u)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((closed >> i) & 1u) c[i] = neg_inf();
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = __fadd_rn(c[i], b[i]);   // (0 or -inf)
    }
    ExactChoice<T> exact = {p, row, (double)mx, 0.0};
    bool have_exact_sum = false;
    auto exact_sum = [&]() {   // the softmax denominator in 64 bits
      if (p.sigmoid || have_exact_sum) return;
      double s = 0.0;
#pragma unroll 1
      for (int e = lane; e < p.E; e += 32) s += exp((double)exact.raw_logit(e) - exact.mx);
      exact.inv_sum = 1.0 / warp_sum(s);
      have_exact_sum = true;
    };
    uint32_t kept = 0xFFFFFFFFu;   // groups
    if (p.n_group > 1) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (32 * i + lane < p.E) sh[32 * i + lane] = c[i];
      __syncwarp();
      float size = 0.0f;   // (twice its error: the terms' and the sum's rounding, and that of two scores)
      const float score = group_score<float>(p, lane, lpg, SharedChoice{sh}, &size);
      bool close = false;
      kept = keep_groups<float>(p, lane, lpg, score, p.by_score ? __fmaf_rn(size, 0x1p-20f, 2.0f * tol) : -1.0f, &close);
      if (close && p.by_score) {
        exact_sum();
        double size64;
        const double score64 = group_score<double>(p, lane, lpg, exact, &size64);
        kept = keep_groups<double>(p, lane, lpg, score64, -1.0, &close);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (32 * i + lane < p.E && !group_open(p, kept, 32 * i + lane)) c[i] = neg_inf();
    }
    // At least k experts have the k-th largest of the 32 lanes' maxima or more; the chosen ones, and all
    // whose order with them is uncertain, are among those that come up to it less the margin.
    float m = c[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, c[i]);
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
      for (int stride = size / 2; stride > 0; stride /= 2) {   // bitonic sort, descending
        const float o = __shfl_xor_sync(0xffffffffu, m, stride);
        m = ((lane & size) == 0) == ((lane & stride) == 0) ? fmaxf(m, o) : fminf(m, o);
      }
    const float kth = __shfl_sync(0xffffffffu, m, p.k - 1);
    const float lim = p.by_score ? __fsub_rn(kth, order_margin(tol, kth)) : kth;
    uint32_t mask = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) mask |= c[i] >= lim ? 1u << i : 0u;
    mask &= there;
    int end = __popc(mask);       // candidates in this lane and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    const int n = __shfl_sync(0xffffffffu, end, 31);
    int my_e = 0, rank = 32;      // this lane's chosen expert and its place among the k (>= k: none)
    float my_x = neg_inf();       // its logit; -inf: unavailable
    if (n <= 32) {
      // one candidate per lane
      for (; mask != 0u; mask &= mask - 1u) cand_sh[warp][--end] = 32 * (__ffs(mask) - 1) + lane;
      __syncwarp();
      float v = neg_inf();
      if (lane < n) {
        my_e = cand_sh[warp][lane];
        const float be = exact.clean_bias(my_e);
        my_x = exact.raw_logit(my_e);
        if (be == neg_inf() || !group_open(p, kept, my_e)) my_x = neg_inf();
        if (my_x > neg_inf())
          v = !p.by_score ? my_x : __fadd_rn(p.sigmoid ? score_sigmoid(my_x) : score_softmax(my_x, mx, inv_sum), be);
      }
      // its rank: how many of the others come first by value, then by index
      const unsigned long long key = lane < n ? (unsigned long long)order_key(v) << 32 | (uint32_t)~my_e : 0ull;
      key_sh[warp][lane] = key;
      __syncwarp();
      rank = 0;
      // (twelve at once, the usual number at most; keys past the last candidate are 0)
#pragma unroll
      for (int j = 0; j < 12; ++j) rank += key_sh[warp][j] > key ? 1 : 0;
      for (int j = 12; j < n; ++j) rank += key_sh[warp][j] > key ? 1 : 0;
      if (p.by_score) {
        // in order, is each of the first k (and the next) further than the margin above the one after it?
        if (lane < n) sort_sh[warp][rank] = v;
        __syncwarp();
        bool near = false;
        if (lane < p.k && lane + 1 < n) {
          const float hi = sort_sh[warp][lane], lo = sort_sh[warp][lane + 1];
          near = __fsub_rn(hi, lo) <= order_margin(tol, fmaxf(fabsf(hi), fabsf(lo)));
        }
        if (__any_sync(0xffffffffu, near)) {
          exact_sum();
          rank = exact_rank(my_x > neg_inf() ? exact(my_e) : -(double)INFINITY, my_e, n);
        }
      }
      if (lane >= n) rank = 32;
      __syncwarp();   // the candidates are read before the next token's are written
    } else {
      // many near the k-th (k above 16, long ties, unavailable experts): k rounds of the largest choice
      bool close = false;
      uint32_t taken = 0u;      // bit i: expert 32 i + lane
#pragma unroll 1
      for (int j = 0; j < p.k; ++j) {
        uint32_t best_key = 0u;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const uint32_t ki = (taken >> i) & 1u || 32 * i + lane >= p.E ? 0u : order_key(c[i]);
          if (ki > best_key) { best_key = ki; bi = i; }
        }
        const uint32_t best = __reduce_max_sync(0xffffffffu, best_key);
        const int e = (int)__reduce_min_sync(0xffffffffu, best_key == best ? (uint32_t)(32 * bi + lane) : 0xFFFFFFFFu);
        const float v = key_value(best);
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        if (lane == j) { my_e = e; rank = j; my_x = v == neg_inf() ? v : exact.raw_logit(e); }
        if (p.by_score && v > neg_inf()) {
          // another expert whose order is uncertain, other than by the same logit and bias (an equal score)
          const float near_lim = __fsub_rn(v, order_margin(tol, v));
          uint32_t near_mask = 0u;
#pragma unroll
          for (int i = 0; i < NV; ++i) near_mask |= c[i] >= near_lim && c[i] > neg_inf() ? 1u << i : 0u;
          near_mask &= ~taken;
          const float xe = exact.raw_logit(e), be = exact.clean_bias(e);
          bool near = false;
          for (; near_mask != 0u; near_mask &= near_mask - 1u) {
            const int o = 32 * (__ffs(near_mask) - 1) + lane;
            near |= exact.raw_logit(o) != xe || exact.clean_bias(o) != be;
          }
          close = __any_sync(0xffffffffu, near);
          if (close) break;
        }
      }
      if (close) {   // the same in 64 bits; choices evaluated where they are compared
        exact_sum();
        taken = 0u;
#pragma unroll 1
        for (int j = 0; j < p.k; ++j) {
          unsigned long long best_key = 0ull;
          int best_e = 0;
#pragma unroll 1
          for (int e = lane; e < p.E; e += 32) {
            if ((taken >> (e >> 5)) & 1u) continue;
            const unsigned long long ke = order_key(group_open(p, kept, e) ? exact(e) : -(double)INFINITY);
            if (ke > best_key) { best_key = ke; best_e = e; }
          }
          const unsigned long long best = warp_max_u64(best_key);
          const int e = (int)__reduce_min_sync(0xffffffffu, best_key == best ? (uint32_t)best_e : 0xFFFFFFFFu);
          if ((e & 31) == lane) taken |= 1u << (e >> 5);
          if (lane == j) {
            my_e = e;
            rank = j;
            my_x = best == order_key(-(double)INFINITY) ? neg_inf() : exact.raw_logit(e);
          }
        }
      }
    }
    // gates of the chosen experts.  Renormalised ones are ratios of scores, so a common factor may go:
    // exp(x - max of the chosen) for softmax; for the sigmoid exp(x - m) / (1 + exp(x)), m = min(0, that max),
    // which keeps scores that would underflow apart.
    const bool chosen = rank < p.k;
    float g = 0.0f;
    if (p.sigmoid) {
      float off = 0.0f;
      if (p.renorm && !__any_sync(0xffffffffu, chosen && my_x >= 0.0f)) off = warp_max(chosen ? my_x : neg_inf());
      const float q = expf(-fabsf(my_x));
      float num = my_x > 0.0f ? 1.0f : q;
      if (off != 0.0f) num = expf(__fsub_rn(my_x, off));
      if (chosen && my_x > neg_inf()) g = __fdiv_rn(num, __fadd_rn(1.0f, q));
    } else {
      const float top = p.renorm ? warp_max(chosen ? my_x : neg_inf()) : mx;
      if (chosen && my_x > neg_inf()) {
        g = expf(__fsub_rn(my_x, top));
        if (!p.renorm) g = __fmul_rn(g, inv_sum);
      }
    }
    if (p.renorm) {
      const float sum = warp_sum(g);
      if (g > 0.0f) g = __fdiv_rn(g, sum);   // (elsewhere 0; a division of 0 would take its slow path)
    }
    if (chosen) {
      p.ids[(size_t)t * p.k + rank] = my_e;
      p.gates[(size_t)t * p.k + rank] = __fmul_rn(g, p.scale);
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, GSG_ERR_NONFINITE);
}

template <typename T, int NV>
static cudaError_t launch_gate_nv(const GateParams& p, int num_sms, cudaStream_t stream) {
  // a warp keeps the biases and takes token after token; as many blocks as fit the device
  unsigned grid = (unsigned)((p.T + kGateWarps - 1) / kGateWarps);
  const unsigned most = (unsigned)num_sms * gate_blocks(NV);
  if (grid > most) grid = most;
  const size_t sh = p.n_group > 1 ? (size_t)kGateWarps * p.E * sizeof(float) : 0;
  return launch_pdl(moe_gate_kernel<T, NV>, grid, 32 * kGateWarps, sh, stream, p);
}

template <typename T>
static cudaError_t launch_gate_t(const GateParams& p, int num_sms, cudaStream_t stream) {
  const int nv = (p.E + 31) / 32;
  if (nv <= 1) return launch_gate_nv<T, 1>(p, num_sms, stream);
  if (nv <= 2) return launch_gate_nv<T, 2>(p, num_sms, stream);
  if (nv <= 4) return launch_gate_nv<T, 4>(p, num_sms, stream);
  if (nv <= 8) return launch_gate_nv<T, 8>(p, num_sms, stream);
  if (nv <= 12) return launch_gate_nv<T, 12>(p, num_sms, stream);
  if (nv <= 16) return launch_gate_nv<T, 16>(p, num_sms, stream);
  return launch_gate_nv<T, 32>(p, num_sms, stream);
}

cudaError_t launch_gate(const void* logits, bool f32, const float* bias, int T, int E, int k, bool sigmoid, int n_group,
                        int topk_group, int group_top, bool renorm, float scale, int32_t* ids, float* gates,
                        int* status, int num_sms, cudaStream_t stream) {
  GateParams p;
  p.logits = logits; p.bias = bias; p.T = T; p.E = E; p.k = k;
  p.sigmoid = sigmoid; p.by_score = bias != nullptr || (n_group > 1 && group_top == 2);
  p.n_group = n_group; p.topk_group = topk_group; p.group_top = group_top; p.group_size = E / n_group;
  p.group_magic = (uint32_t)(((1u << 20) + p.group_size - 1) / p.group_size);
  p.renorm = renorm; p.scale = scale; p.ids = ids; p.gates = gates; p.status = status;
  return f32 ? launch_gate_t<float>(p, num_sms, stream) : launch_gate_t<uint16_t>(p, num_sms, stream);
}

}  // namespace gsg
