// gsg_norm.cu -- residual addition, RMS norm and microscaled output in one pass over the row.
//
//   h = x + r, rounded to r's type and stored (no r: h = x);   v = mean(h^2) + eps
//   y = h * w / sqrt(v);   outputs: h, y in bf16, y in MXFP8 or MXFP4 (from the unrounded y)
//
// A block holds one row in registers, so every input is read once and every output written once: bound by HBM, 8192
// x 7168 with an fp32 residual, bf16 y and 8-bit codes 119 us = 6.4 TB/s; 512 x 2048 5.1 us, one row 3.5 us (latency).
// Kept up for seconds it takes 134 to 141 us, at the board's power limit; squares summed in plain fp32 did not change
// that, and in fp32 with the rounding errors carried along they took 9 us more.
// The squares are summed in 64 bits, and 1 / sqrt(v) is taken in 64 bits and applied as a sum of two fp32
// numbers (in 64 bits throughout where those leave the fp32 range's middle).  y is rounded to fp32 "to odd"
// (see round_odd), so that its later rounding to a code or to bf16 is the rounding of the value before it,
// not of a value that has been rounded onto a border between two codes: with sums of eight squares in fp32,
// which is 2^-31 off, a few of 58.7 million codes still came out on the wrong side.  (h may be the
// residual's own buffer: each thread reads its values before it stores them.)
#include "gsg_launch.h"
#include "gsg_mx.cuh"

namespace gsg {

struct NormParams {
  const uint16_t* x;   // [T][K] bf16
  const void* r;       // [T][K] bf16 or fp32 (kRes 1, 2)
  const void* w;       // [K] bf16 or fp32
  void* h;             // [T][K] in r's type
  uint16_t* y;         // [T][K] bf16 or nullptr
  uint8_t* codes;      // nullptr: no microscaled output
  uint8_t* scales;
  int T, K;
  float eps;
  int w_f32;
  int* status;
};

// 16 bytes where `on`, else zeros.  (An ordinary load, see pdl_wait; from L2, since a row is read once.)
__device__ __forceinline__ uint4 load_l2(bool on, const void* p) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)on));
  return v;
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ void unpack8_bf16(uint4 q, float v[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// v + rest (|rest| at most half a unit of v) rounded to odd: the exact numbers stay, any other becomes
// whichever of its two fp32 neighbours has the odd last bit.  An odd number is no border of a shorter
// format, so rounding it again to fewer bits gives what rounding v + rest would have given.
__device__ __forceinline__ float round_odd(float v, float rest) {
  uint32_t u = __float_as_uint(v);
  // towards zero where v was rounded away from it: rest, signed by v, is negative (a product of the two may underflow)
  u -= (uint32_t)(__uint_as_float(__float_as_uint(rest) ^ (u & 0x80000000u)) < 0.0f);
  u |= (uint32_t)(rest != 0.0f);
  return __uint_as_float(u);
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
constexpr uint32_t kBf16Inf = 0x7F7F8000u;   // the least magnitude that bf16 has no finite number for

constexpr int kNormThreads = 512;

// kRes: 0 no residual, 1 bf16, 2 fp32.  kBits: 0 no microscaled output, 4, 8.  A thread holds kU units
// of eight consecutive values, unit i * blockDim.x + threadIdx.x of the row; four neighbouring lanes
// hold a 32-block and sixteen a 128-wide k-block (K % 256 == 0 with microscaled output, so the lanes
// of a k-block are all in the row or all past its end).  With two units and codes three blocks of 512 threads share an
// SM, at 40 registers; at 42 only two do (8192 x 7168, fp32 residual: 130 us for 119; no residual, 4-bit: 95 for 80).
template <int kRes, int kBits, int kU>
__global__ void __launch_bounds__(kNormThreads, kU == 2 && kBits != 0 ? 3 : 0)
add_rmsnorm_kernel(const NormParams p) {
  __shared__ double red[32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int t = blockIdx.x, upr = p.K / 8;
  const size_t row = (size_t)t * p.K;
  float v[kU][8];
  uint4 xq[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int u = i * blockDim.x + threadIdx.x;
    xq[i] = load_l2(u < upr, p.x + row + 8 * (size_t)u);
  }
  if (kRes == 1) {
    uint4 rq[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = i * blockDim.x + threadIdx.x;
      rq[i] = load_l2(u < upr, static_cast<const uint16_t*>(p.r) + row + 8 * (size_t)u);
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = i * blockDim.x + threadIdx.x;
      float a[8], b[8];
      unpack8_bf16(xq[i], a);
      unpack8_bf16(rq[i], b);
      const uint4 hq = make_uint4(pack2_bf16(__fadd_rn(a[0], b[0]), __fadd_rn(a[1], b[1])),
                                  pack2_bf16(__fadd_rn(a[2], b[2]), __fadd_rn(a[3], b[3])),
                                  pack2_bf16(__fadd_rn(a[4], b[4]), __fadd_rn(a[5], b[5])),
                                  pack2_bf16(__fadd_rn(a[6], b[6]), __fadd_rn(a[7], b[7])));
      if (u < upr) reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h) + row)[u] = hq;
      unpack8_bf16(hq, v[i]);
    }
  } else if (kRes == 2) {
    uint4 rq[kU][2];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = i * blockDim.x + threadIdx.x;
      const float* src = static_cast<const float*>(p.r) + row + 8 * (size_t)u;
      rq[i][0] = load_l2(u < upr, src);
      rq[i][1] = load_l2(u < upr, src + 4);
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = i * blockDim.x + threadIdx.x;
      unpack8_bf16(xq[i], v[i]);
      const uint32_t rb[8] = {rq[i][0].x, rq[i][0].y, rq[i][0].z, rq[i][0].w,
                              rq[i][1].x, rq[i][1].y, rq[i][1].z, rq[i][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = __fadd_rn(v[i][j], __uint_as_float(rb[j]));
      if (u < upr) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.h) + row) + 2 * u;
        dst[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        dst[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kU; ++i) unpack8_bf16(xq[i], v[i]);
  }
  // ---- mean square
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kU; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __fma_rn((double)v[i][j], (double)v[i][j], sum);
  sum = warp_sum_d(sum);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = warp_sum_d(lane < nw ? red[lane] : 0.0);
  const double var = sum / (double)p.K + (double)p.eps;
  if (kBits == 0 && p.y == nullptr) {   // h alone
    if (!(var < (double)INFINITY) && threadIdx.x == 0) set_status(p.status, GSG_ERR_NONFINITE);
    return;
  }
  const double rd = rsqrt(var);
  const float rh = (float)rd, rl = (float)(rd - (double)rh);
  // |h| rh is at most sqrt(K), whatever the weights: a product with w past the range is a y past the range.  What is
  // carried along underflows for y below 2^-100 or h below 2^-100 of the row's rms only.
  const bool middle = rh > 0x1p-60f && rh < 0x1p60f;
  // ---- scaled row
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int u = i * blockDim.x + threadIdx.x;
    const bool in = u < upr;
    float w[8];
    if (p.w_f32) {
      const float4* src = reinterpret_cast<const float4*>(p.w) + 2 * u;
      const float4 a = in ? __ldca(src) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 b = in ? __ldca(src + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
      unpack8_bf16(in ? __ldca(reinterpret_cast<const uint4*>(p.w) + u) : make_uint4(0u, 0u, 0u, 0u), w);
    }
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // h * (rh + rl) * w, the first product's rounding error carried along
      const float q = __fmul_rn(v[i][j], rh);
      const float c = __fmul_rn(__fmaf_rn(v[i][j], rl, __fmaf_rn(v[i][j], rh, -q)), w[j]);
      const float s = __fmaf_rn(q, w[j], c);
      y[j] = round_odd(s, __fadd_rn(__fmaf_rn(q, w[j], -s), c));
    }
    if (!middle) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float h = v[i][j];
        // (the weight from memory again: the eight of a unit held until here would be registers that every row misses)
        const float wj = !in       ? 0.0f
                         : p.w_f32 ? static_cast<const volatile float*>(p.w)[8 * u + j]
                                   : bf16_bits_to_f32(static_cast<const volatile uint16_t*>(p.w)[8 * u + j]);
        asm volatile("" : "+f"(h));   // not the sum's conversion kept in a register pair until here
        const double d = (double)h * (double)wj * rd;
        const float s = (float)d;
        y[j] = round_odd(s, (float)(d - (double)s));
      }
    }
    // a y that is not finite, as every one is of a row without a norm (v 0, infinite or NaN), or that bf16 does not
    // hold
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(y[j]));
    uint32_t am = __float_as_uint(top);
    if (am >= kBf16Inf) set_status(p.status, GSG_ERR_NONFINITE);
    if (p.y != nullptr && in)
      reinterpret_cast<uint4*>(p.y + row)[u] =
          make_uint4(pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3]), pack2_bf16(y[4], y[5]), pack2_bf16(y[6], y[7]));
    if (kBits != 0) {
      constexpr int kB = kBits == 0 ? 8 : kBits;
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const uint32_t sc = mx_scale_byte<kB>(am);
      const float inv = mx_inv_scale(sc);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(y[j], inv);
      if (in) {
        if (kB == 8)
          reinterpret_cast<uint2*>(p.codes + row)[u] =
              make_uint2(e4m3_encode4_cvt(y[0], y[1], y[2], y[3]), e4m3_encode4_cvt(y[4], y[5], y[6], y[7]));
        else
          reinterpret_cast<uint32_t*>(p.codes + row / 2)[u] = e2m1_encode8_cvt(y);
      }
      const int g = lane & 16;
      const uint32_t word = __shfl_sync(0xffffffffu, sc, g) | (__shfl_sync(0xffffffffu, sc, g + 4) << 8) |
                            (__shfl_sync(0xffffffffu, sc, g + 8) << 16) | (__shfl_sync(0xffffffffu, sc, g + 12) << 24);
      const int c = lane & 15;
      if (in && c < 4) {   // quad entries (kb, t - 32 c, c), and zeros where t + 32 c is past the last row
        uint32_t* sw = reinterpret_cast<uint32_t*>(p.scales) + (size_t)(u >> 4) * p.T * 4 + c;
        if (t >= 32 * c) sw[(size_t)(t - 32 * c) * 4] = word;
        if (t + 32 * c >= p.T) sw[(size_t)t * 4] = 0u;
      }
    }
  }
}

template <int kRes, int kBits>
static cudaError_t launch_norm_u(const NormParams& p, cudaStream_t stream) {
  const int upr = p.K / 8;
  // units per thread: as few as a block of 512 threads allows, to hide the loads of one row
  const int kU = upr <= kNormThreads ? 1 : upr <= 2 * kNormThreads ? 2 : upr <= 4 * kNormThreads ? 4 : 8;
  const int threads = (((upr + kU - 1) / kU) + 31) / 32 * 32;
  if (kU == 1) return launch_pdl(add_rmsnorm_kernel<kRes, kBits, 1>, p.T, threads, 0, stream, p);
  if (kU == 2) return launch_pdl(add_rmsnorm_kernel<kRes, kBits, 2>, p.T, threads, 0, stream, p);
  if (kU == 4) return launch_pdl(add_rmsnorm_kernel<kRes, kBits, 4>, p.T, threads, 0, stream, p);
  return launch_pdl(add_rmsnorm_kernel<kRes, kBits, 8>, p.T, threads, 0, stream, p);
}

template <int kRes>
static cudaError_t launch_norm_b(const NormParams& p, int bits, cudaStream_t stream) {
  if (bits == 8) return launch_norm_u<kRes, 8>(p, stream);
  if (bits == 4) return launch_norm_u<kRes, 4>(p, stream);
  return launch_norm_u<kRes, 0>(p, stream);
}

cudaError_t launch_add_rmsnorm(const uint16_t* x, const void* r, int r_f32, const void* w, int w_f32, int T, int K,
                               float eps, void* h, uint16_t* y, int bits, uint8_t* codes, uint8_t* scales, int* status,
                               cudaStream_t stream) {
  NormParams p;
  p.x = x; p.r = r; p.w = w; p.h = h; p.y = y; p.codes = codes; p.scales = scales;
  p.T = T; p.K = K; p.eps = eps; p.w_f32 = w_f32; p.status = status;
  if (r == nullptr) return launch_norm_b<0>(p, bits, stream);
  return r_f32 ? launch_norm_b<2>(p, bits, stream) : launch_norm_b<1>(p, bits, stream);
}

}  // namespace gsg
