// gsg_mx.cu -- microscaled formats: the MXFP4 weight packers and the MXFP4 / MXFP8 activation quantizer
// fused with the MoE dispatch.  The block rule is in gsg_mx.cuh, the layouts in include/gsg.h.
#include "gsg_launch.h"
#include "gsg_mx.cuh"

namespace gsg {

// ------------------------------------------------------------------ weight packers (offline)
// One thread per 32-block of W: its codes are 16 bytes of the row's 128 in the chunk block, its scale
// one byte of the chunk block's scale atoms.
__device__ __forceinline__ uint8_t* mx_chunk(uint8_t* packed, long long e, int n, int kc, int NT, int KC) {
  return packed + ((size_t)(e * NT + n / kTileN) * KC + kc) * kMxChunkBytes;
}
__device__ __forceinline__ int mx_scale_at(int r, int b) {   // row r of the tile, block b (0..7) of the chunk
  return kMxCodeBytes + (b >> 2) * 512 + 16 * (r & 31) + 4 * (r >> 5) + (b & 3);
}

template <bool kF32>
__global__ void __launch_bounds__(256)
pack_mxfp4_kernel(const void* __restrict__ W, long long blocks, int N, int K, uint8_t* __restrict__ packed,
                  int* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int bpr = K / 32, NT = N / kTileN, KC = K / kChunkK;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < blocks;
       i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / bpr;
    const int b = (int)(i % bpr), n = (int)(row % N);
    float v[32];
    if (kF32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(W) + i * 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 x = __ldca(src + j);
        v[4 * j] = x.x; v[4 * j + 1] = x.y; v[4 * j + 2] = x.z; v[4 * j + 3] = x.w;
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + i * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = __ldca(src + j);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[8 * j + 2 * q] = __uint_as_float(w[q] << 16);
          v[8 * j + 2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
      }
    }
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) am = max(am, abs_bits(v[j]));
    if (am >= kF32Inf) set_status(status, GSG_ERR_NONFINITE);
    const uint32_t sc = mx_scale_byte<4>(am);
    const float inv = mx_inv_scale(sc);
    uint32_t cw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float xs[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) xs[q] = __fmul_rn(v[8 * j + q], inv);
      cw[j] = e2m1_encode8_cvt(xs);
    }
    uint8_t* cb = mx_chunk(packed, row / N, n, b >> 3, NT, KC);
    const int r = n % kTileN;
    *reinterpret_cast<uint4*>(cb + r * 128 + (b & 7) * 16) = make_uint4(cw[0], cw[1], cw[2], cw[3]);
    cb[mx_scale_at(r, b & 7)] = (uint8_t)sc;
  }
}

// Codes [E][N][K/2] and scales [E][N][K/32] as checkpoints store them: the same bytes, rearranged.
__global__ void __launch_bounds__(256)
pack_mxfp4_codes_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long blocks, int N,
                        int K, uint8_t* __restrict__ packed, int* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int bpr = K / 32, NT = N / kTileN, KC = K / kChunkK;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < blocks;
       i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / bpr;
    const int b = (int)(i % bpr), n = (int)(row % N), r = n % kTileN;
    const uint4 c = __ldca(reinterpret_cast<const uint4*>(codes) + i);
    const uint8_t sc = __ldca(scales + i);
    if (sc == 0xFFu) set_status(status, GSG_ERR_NONFINITE);   // UE8M0's NaN
    uint8_t* cb = mx_chunk(packed, row / N, n, b >> 3, NT, KC);
    *reinterpret_cast<uint4*>(cb + r * 128 + (b & 7) * 16) = c;
    cb[mx_scale_at(r, b & 7)] = sc;
  }
}

static unsigned pack_grid(long long blocks) {
  const long long g = (blocks + 255) / 256;
  return (unsigned)(g < 65535 ? g : 65535);
}

cudaError_t launch_pack_mxfp4(const void* W, bool w_f32, int E, int N, int K, uint8_t* packed, int* status,
                              cudaStream_t stream) {
  const long long blocks = (long long)E * N * (K / 32);
  return w_f32 ? launch_pdl(pack_mxfp4_kernel<true>, pack_grid(blocks), 256, 0, stream, W, blocks, N, K, packed, status)
               : launch_pdl(pack_mxfp4_kernel<false>, pack_grid(blocks), 256, 0, stream, W, blocks, N, K, packed,
                            status);
}

cudaError_t launch_pack_mxfp4_codes(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* packed,
                                    int* status, cudaStream_t stream) {
  const long long blocks = (long long)E * N * (K / 32);
  return launch_pdl(pack_mxfp4_codes_kernel, pack_grid(blocks), 256, 0, stream, codes, scales, blocks, N, K, packed,
                    status);
}

// ------------------------------------------------------------------ activation quantizer + dispatch
// A lane makes 16 bytes of codes: a whole 32-block in 4 bits, half of one in 8 bits (two lanes share the
// block's maximum).  Every token is read and quantized once and written to its k routed rows.  Bound by the scattered
// scale words' sectors and the codes' writes.  Alone, in a graph of calls on buffers that change: 512 tokens x 8 rows x
// 2048, 4-bit, 3.8 us; 1023 rows x 7168, 8-bit, 6.4 us; 1368 tokens x 8 x 7168, 4-bit, 20.7 us.
struct MxQuantParams {
  const uint16_t* X;
  const int32_t* inv_perm;
  int T, K, k, R;
  uint8_t* codes;
  uint8_t* scales;
  uint32_t* raw;   // non-null: scale words go to raw[row][K/128], then launch_scales_quad
  int* status;
};

constexpr int kMxQuantThreads = 128;
constexpr int kMxRowsAhead = 8;   // routed rows loaded with the values (the rest on demand)

template <int kBits>
__global__ void __launch_bounds__(kMxQuantThreads)
act_quant_mx_kernel(const MxQuantParams p) {
  constexpr int kVals = 128 / kBits;          // values per lane
  constexpr int kLanesPerKb = 128 / kVals;    // lanes of one 128-wide k-block (4 or 8)
  constexpr int kLanesPerBlk = 32 / kVals;    // 1 or 2
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const unsigned upr = (unsigned)(p.K / kVals);                        // lanes of work per token (K % 256 == 0)
  const unsigned U = (unsigned)p.T * upr;                              // < 2^31, checked on the host
  const unsigned step = gridDim.x * blockDim.x;
  uint32_t* sw = reinterpret_cast<uint32_t*>(p.scales);
  for (unsigned u0 = blockIdx.x * blockDim.x + (threadIdx.x & ~31u); u0 < U; u0 += step) {
    const unsigned u = u0 + lane;                 // a warp's lanes past the end quantize zeros, store nothing
    const bool valid = u < U;
    const int t = (int)((valid ? u : 0) / upr);
    const int c = (int)((valid ? u : 0) % upr);   // unit of the row
    const uint4* src = reinterpret_cast<const uint4*>(p.X + (size_t)t * p.K) + (size_t)c * (kVals / 8);
    uint32_t w[kVals / 2];
#pragma unroll
    for (int i = 0; i < kVals / 8; ++i) {
      const uint4 x = valid ? __ldca(src + i) : make_uint4(0u, 0u, 0u, 0u);
      w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
    }
    int rows[kMxRowsAhead];
#pragma unroll
    for (int j = 0; j < kMxRowsAhead; ++j)
      rows[j] = (valid && j < p.k) ? (p.inv_perm != nullptr ? __ldca(p.inv_perm + (size_t)t * p.k + j) : t) : -1;
    uint32_t m2 = 0;   // maxima of the even and the odd values' magnitudes, as bf16 bits
#pragma unroll
    for (int i = 0; i < kVals / 2; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
    uint32_t am = max(m2 << 16, m2 & 0xFFFF0000u);
    if (kLanesPerBlk == 2) am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    if (am >= kF32Inf) set_status(p.status, GSG_ERR_NONFINITE);
    const uint32_t sc = mx_scale_byte<kBits>(am);
    const float inv = mx_inv_scale(sc);
    uint32_t cw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kBits == 4) {
        float xs[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xs[2 * j] = __fmul_rn(__uint_as_float(w[(kVals / 8) * i + j] << 16), inv);
          xs[2 * j + 1] = __fmul_rn(__uint_as_float(w[(kVals / 8) * i + j] & 0xFFFF0000u), inv);
        }
        cw[i] = e2m1_encode8_cvt(xs);
      } else {
        const uint32_t a = w[2 * i], b = w[2 * i + 1];
        cw[i] = e4m3_encode4_cvt(__fmul_rn(__uint_as_float(a << 16), inv), __fmul_rn(__uint_as_float(a & 0xFFFF0000u), inv),
                                 __fmul_rn(__uint_as_float(b << 16), inv), __fmul_rn(__uint_as_float(b & 0xFFFF0000u), inv));
      }
    }
    const int g = lane & ~(kLanesPerKb - 1);
    const uint32_t word = __shfl_sync(0xffffffffu, sc, g) | (__shfl_sync(0xffffffffu, sc, g + kLanesPerBlk) << 8) |
                          (__shfl_sync(0xffffffffu, sc, g + 2 * kLanesPerBlk) << 16) |
                          (__shfl_sync(0xffffffffu, sc, g + 3 * kLanesPerBlk) << 24);
    if (!valid) continue;
    const int kb = c / kLanesPerKb, cq = lane & (kLanesPerKb - 1);
    auto dispatch = [&](int row) {
      if (row < 0 || row >= p.R) { set_status(p.status, GSG_ERR_BAD_ROUTING); return; }
      *reinterpret_cast<uint4*>(p.codes + ((size_t)row * upr + c) * 16) = make_uint4(cw[0], cw[1], cw[2], cw[3]);
      if (p.raw != nullptr) {
        if (cq == 0) p.raw[(size_t)row * (p.K / 128) + kb] = word;
        return;
      }
      // quad entries (kb, row - 32 cq, cq); the entries whose row lies past the last are zeroed by the
      // rows 96 .. 1 before the end
      if (cq < 4) {
        const int rr = row - 32 * cq;
        if (rr >= 0) sw[((size_t)kb * p.R + rr) * 4 + cq] = word;
        if (row + 32 * cq >= p.R) sw[((size_t)kb * p.R + row) * 4 + cq] = 0u;
      }
    };
#pragma unroll
    for (int j = 0; j < kMxRowsAhead; ++j)
      if (j < p.k) dispatch(rows[j]);
    for (int j = kMxRowsAhead; j < p.k; ++j) dispatch(__ldca(p.inv_perm + (size_t)t * p.k + j));
  }
}

// Bytes of the row-major scale words of the two-launch path (0: direct stores).  A direct store of a scale
// word is four scattered 4-byte stores, and at large sizes those, not the codes, take the time: 1368 tokens x 8
// rows x 7168, 4-bit, 21.4 us direct and 18.1 us in two launches, 2048 tokens 35.4 and 23.8 us; but 512 tokens x
// 8 x 7168 10.9 and 11.9 us, and 8192 rows in token order (k = 1, neighbours' words side by side) 29.0 and 33.9 us.
size_t quant_mx_raw_bytes(long long R, int K, int k) {
  return R * (long long)K >= (k > 1 ? 1ll << 26 : 1ll << 27) ? (size_t)(R * (long long)(K / 128) * 4) : 0;
}

constexpr int kSmSharedBytes = 228 * 1024;   // an SM's shared memory, of which every block takes 1 KB beside its own
// Shared memory with which an SM holds `fair` blocks and not one more.
constexpr int mx_spread_smem(int fair) { return kSmSharedBytes / (fair + 1); }
constexpr bool mx_spread_holds(int fair, int blocks) {
  return blocks * (mx_spread_smem(fair) + 1024) <= kSmSharedBytes;
}
static_assert(mx_spread_holds(1, 1) && !mx_spread_holds(1, 2) && mx_spread_holds(2, 2) && !mx_spread_holds(2, 3) &&
              mx_spread_holds(3, 3) && !mx_spread_holds(3, 4), "blocks per SM");

cudaError_t quant_mx_set_smem_attrs() {
  cudaError_t e = cudaFuncSetAttribute(act_quant_mx_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       mx_spread_smem(1));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(act_quant_mx_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             mx_spread_smem(1));
  return e;
}

cudaError_t launch_quant_mx(const uint16_t* X, int T, int K, int bits, const int32_t* inv_perm, int k, uint8_t* codes,
                            uint8_t* scales, uint32_t* raw, int* status, int num_sms, cudaStream_t stream) {
  MxQuantParams p;
  p.X = X; p.inv_perm = inv_perm; p.T = T; p.K = K; p.k = k; p.R = T * k;
  p.codes = codes; p.scales = scales; p.raw = raw; p.status = status;
  const long long units = (long long)T * K * bits / 128;
  long long blocks = (units + kMxQuantThreads - 1) / kMxQuantThreads;
  if (blocks > (long long)num_sms * 16) blocks = (long long)num_sms * 16;
  // Launched early, behind a GEMM that fills the SMs, the blocks of a small grid would all settle on the first
  // SMs to come free and share them (measured: 4096 rows x 2048, quantizer + product 53.4 us instead of 45.3).
  // The shared memory that each asks for, and does not use, leaves room for its fair number per SM only.  (With room
  // for one more: 4096 rows x 2048 46.6 us instead of 45.8, the quantizer alone 4.9 instead of 3.8.)
  const long long fair = (blocks + num_sms - 1) / num_sms;
  const size_t smem = fair < 4 ? (size_t)mx_spread_smem((int)fair) : 0;
  const cudaError_t e = bits == 8
      ? launch_pdl(act_quant_mx_kernel<8>, (unsigned)blocks, kMxQuantThreads, smem, stream, p)
      : launch_pdl(act_quant_mx_kernel<4>, (unsigned)blocks, kMxQuantThreads, smem, stream, p);
  if (e != cudaSuccess || raw == nullptr) return e;
  return launch_scales_quad(raw, p.R, K / 128, p.R, reinterpret_cast<uint32_t*>(scales), stream);
}

}  // namespace gsg
