// gsg_gemm.cu -- persistent grouped NVFP4 expert GEMM on the Blackwell tensor cores.
//
// "Hardware-Native Joint Sparse-Quantization for Trillion-Scale Mixture-of-Experts"
// (paperlayer.ai summary): §3.4 (pp.5-6) -- grouped execution of routing-dependent expert
// problems in one launch using Blackwell sparse MMA, the sparse weight placed as operand A;
// §2 "Hardware opportunity" (p.3) -- paired 4:8 NVFP4 runs at twice the dense NVFP4 rate;
// §D.2 (p.19) -- a dense control that differs from the sparse kernel only in sparsity.
//
// One CTA per SM, 352 threads (11 warps; 480 = 15 warps for wide pair tiles), warp-specialised
// around one shared-memory ring whose stages hold 256 to 768 logical K of one tile (weights,
// activation codes and both scales):
//   warp 0      weight producer: per stage one bulk copy per interleaved packed weight block and
//               one TMA box of the activation scale atoms, each from its own lane.
//   warp 2      activation producer: tensor-map TMA boxes (128B swizzle, 64 or 32 rows) of only the
//               token rows the tile holds, each from its own lane.
//   warps 7..10 scale/metadata loaders, one per TMEM lane quadrant: read the stage's metadata and
//               scale atoms from shared memory and tcgen05.st them into one of three TMEM sets.
//   warp 1      TMEM owner and MMA issuer: per stage only tcgen05.mma(.sp) kind::mxf4nvf4
//               block_scale (M = 128 weight rows, N = the tile's token count rounded to 16, K = 128
//               logical sparse / 64 dense) and one tcgen05.commit; up to eight TMEM accumulators.
//   warps 3..6  epilogue: tcgen05.ld accumulator lanes, multiply by s_x * s_w[e], store rows of Y.
//   warps 11..14 (wide pair tiles only) a second epilogue, for the tile's second n-tile pair.
// The microscaled formats (see kFmtMx4) differ in four things.  Their scales come as copies of their own, so a
// last warp produces them into a ring of their own, ahead of the operands.  The copies of both CTAs of a pair
// complete on the leader's barriers.  Tiles past 64 tokens are wide pair tiles of 128 or 192 tokens
// (mx_pick_bn) for any N, whose last group of n-tiles may be short.  And an expert's token tiles share its rows
// evenly.
// What a stage costs is the MMA warp's instructions as much as the tensor pipe: by SM clock, with operands that
// the compiler does not know to be warp-uniform, a wide stage took 800 cycles (120 for each of the two barriers,
// 50 for each MMA) whatever its tokens; with uniform() 620 at 128 tokens and the tensor pipe's 768 at 192.  Copying
// the scales into TMEM with tcgen05.cp from that warp instead of the loader warps: 10 % slower (4096 x 4096 x 7168,
// 4-bit: 63 -> 74 us), the copies and the MMAs share a pipe.
// Every TMA and tcgen05 instruction is issued by an elected lane of a converged warp.
// 128-token tiles run on CTA pairs (cta_group::2, M = 256 weight rows).  Where N holds whole
// groups of four n-tiles, a pair tile is wide: 512 weight rows (two MMAs per k-block into two
// accumulators) against one 128-token activation tile, so the activations cross from L2 to the
// SMs once for 512 weight rows instead of once per 256.  Its two accumulators fill TMEM beside the
// metadata sets, so there is one accumulator buffer; the MMA warp waits for the epilogue between
// tiles, and the two epilogue warp groups halve that wait.
// Tiles are (expert e, 128 weight rows nt, token tile mt) in e -> nt -> mt order; CTAs take
// tiles round-robin and decode their own tile list into shared memory once, at set-up.
// Experts with no rows produce no tiles.  Every mbarrier wait is bounded:
// on expiry the kernel records GSG_ERR_DEVICE_TIMEOUT, drains its own copies and MMAs, frees
// TMEM and returns.
#include <atomic>

#include <cuda.h>

#include "gsg_internal.cuh"
#include "gsg_launch.h"

namespace gsg {

constexpr int kGemmThreads = 352;
// a wide pair tile adds four epilogue warps (11..14) that drain the tile's second n-tile while
// warps 3..6 drain the first
constexpr int kGemmThreadsWide = 480;
constexpr int kScaleRing = 4;              // microscaled formats: stages of the scale ring
constexpr int kMaxE = 1024;
constexpr int kMaxAcc = 8;
constexpr int kNSets = 3;                  // TMEM sets of metadata + scales
constexpr uint64_t kWaitTimeoutNs = 2000000000ull;   // 2 s
constexpr uint32_t kTmemCols = 512;
constexpr int kOutStageBytes = 16 * 32 * 4;           // epilogue transpose buffer per warp
constexpr int kGluStageBytes = 32 * 36 * 4;           // SwiGLU epilogue: 32 tokens x 32 features (+4 pad)

// Operand formats of an instantiation (weights x activations).
//  kFmtDense, kFmtSparse: NVFP4 both, UE4M3 block scales and fp32 tensor scales (kind::mxf4nvf4).
//  kFmtMx4: microscaled 4-bit weights and activations, one UE8M0 scale per 32 values and no tensor
//    scale (kind::mxf4, K = 64 per MMA).
//  kFmtMx8: the same weights, E4M3 activations with UE8M0 scales (kind::mxf8f6f4, K = 32 per MMA).
//    That MMA reads 4-bit operands from 16-byte groups of 16 values (8 bytes of codes, 8 of padding);
//    the TMA writes that form into shared memory from the packed codes, so HBM and L2 carry 4 bits.
constexpr int kFmtDense = kGemmDense, kFmtSparse = kGemmSparse, kFmtMx4 = kGemmMx4, kFmtMx8 = kGemmMx8;

__host__ __device__ constexpr bool fmt_mx(int fmt) { return fmt == kFmtMx4 || fmt == kFmtMx8; }
// (the microscaled formats have a warp more, the scale producer)
__host__ __device__ constexpr int gemm_threads(int fmt, bool wide) {
  return (wide ? kGemmThreadsWide : kGemmThreads) + (fmt_mx(fmt) ? 32 : 0);
}

struct GemmParams {
  const uint8_t* a_scales;
  const float* x_scale;
  const uint8_t* w_packed;
  const float* w_scale;
  const int32_t* off;
  void* Y;                 // Y [R][N] (bf16 or fp32); with the SwiGLU epilogue: h codes [R][N/4]
  int* status;
  int E, N, K, R, y_f32, rcap;
  int stages, nacc, tcap;
  int sched;               // tile schedule: kSchedRoundRobin or kSchedRuns (see tile_of)
  uint8_t* h_scales;       // SwiGLU epilogue: h scales, quad layout [N/256][R+256][4][4]
  const float* h_scale;    // SwiGLU epilogue: tensor scale of h
  // combine epilogue (perm_src non-null): Y is the slot buffer [T*k][N] bf16 (row = flat index
  // t*k + j of the routed pair), counters [T][N/32] (zero on entry, left zero), out [T][N] bf16
  const int32_t* perm_src;
  const float* gates;
  int* counters;
  uint16_t* out;
  int k;
  // test hook (0 = off): before its second tile (its first, if it has only one) the MMA warp waits
  // this long on a barrier that nothing arrives on, so that the bounded wait runs out and the
  // abort path -- status word, drain of copies and MMAs, TMEM release -- runs as it would after
  // a real stall
  unsigned long long stall_ns;
};

// ------------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---- CTA pairs (thread-block clusters of two CTAs on two SMs; see kCG below)
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The shared::cluster address of the same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
// Arrive on an mbarrier given by its shared::cluster address (a barrier of this CTA or of the
// other CTA of the pair).  Default semantics (no cluster-scope release, which costs a fence per
// arrive): what the arrive hands over is already complete when it is issued -- copies that landed
// (their full barrier completed) and TMEM stores waited on with tcgen05.wait::st -- and is read
// only by the leader's tensor-core work issued after the leader observed the phase.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cl_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cl_addr) : "memory");
}
// Every thread of both CTAs of the cluster: all earlier writes (barrier initialisation included)
// are visible to the other CTA afterwards.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The issue wrappers below are executed by a whole converged warp: elect.sync picks one lane
// and predicates the instruction on it, so the warp never diverges around a TMA or tcgen05
// instruction (issuing them from a lone lane of a diverged warp costs several times more).
#define GSG_ELECT "elect.sync _|P, 0xffffffff;\n\t"
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .pred P;\n\t" GSG_ELECT "@P mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
               "r"(bytes)
               : "memory");
}
// Per-lane forms: every lane of the (converged) warp executes the instruction and the lanes with
// `on` set each issue their own copy.  The TMA unit works through the copies of one issuing thread
// one after another, so the copies of a stage are spread over lanes to be in flight together.
__device__ __forceinline__ void bulk_g2s_lane(bool on, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %4, 0;\n\t"
      "@P cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_lane(bool on, uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %5, 0;\n\t"
      "@P cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"((uint32_t)on)
      : "memory");
}
// Pair form: the copy goes to this CTA's own shared memory and completes on a barrier that may be the
// other CTA's (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_lane_pair(bool on, uint32_t dst, const CUtensorMap* map, int x, int y,
                                                      uint32_t cluster_bar) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %5, 0;\n\t"
      "@P cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(cluster_bar), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void lds128(uint32_t saddr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(saddr) : "memory");
}
// tcgen05.st of N consecutive 32-bit columns for the 32 lanes of this warp's quadrant.
__device__ __forceinline__ void tc_st_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tc_st_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tc_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Writes `kCols` (a multiple of 4) columns from registers, largest pieces first.
template <int kCols>
__device__ __forceinline__ void tc_st_cols(uint32_t taddr, const uint32_t* r) {
  int c = 0;
#pragma unroll
  for (; c + 16 <= kCols; c += 16) tc_st_x16(taddr + c, r + c);
  if constexpr (kCols % 16 >= 8) {
    tc_st_x8(taddr + (kCols / 16) * 16, r + (kCols / 16) * 16);
  }
  if constexpr (kCols % 8 >= 4) {
    tc_st_x4(taddr + (kCols / 8) * 8, r + (kCols / 8) * 8);
  }
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("{\n\t.reg .pred P;\n\t" GSG_ELECT
               "@P tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
               : "memory");
}
// Pair form: once the pair's earlier tensor-core work has completed, arrive once on the barrier at
// this shared-memory offset in every CTA of `mask` (bit r = CTA rank r).
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile("{\n\t.reg .pred P;\n\t" GSG_ELECT
               "@P tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               "\n\t}" ::"r"(bar), "h"(mask)
               : "memory");
}
__device__ __forceinline__ void tc_mma_sparse(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate, uint32_t sfa, uint32_t sfb, uint32_t meta) {
  asm volatile(
      "{\n\t.reg .pred p, P;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t" GSG_ELECT
      "@P tcgen05.mma.sp.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, [%7], %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(meta)
      : "memory");
}
__device__ __forceinline__ void tc_mma_dense(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate, uint32_t sfa, uint32_t sfb) {
  asm volatile(
      "{\n\t.reg .pred p, P;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t" GSG_ELECT
      "@P tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// The same two MMAs issued for a CTA pair (M = 256: each CTA supplies its 128 weight rows and half
// of the tile's token columns from its own shared memory at the same offsets, and holds its rows'
// accumulator, metadata and scales -- the scales of all N token columns -- in its own TMEM at the
// same addresses).
__device__ __forceinline__ void tc_mma_sparse_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                   uint32_t accumulate, uint32_t sfa, uint32_t sfb, uint32_t meta) {
  asm volatile(
      "{\n\t.reg .pred p, P;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t" GSG_ELECT
      "@P tcgen05.mma.sp.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, [%7], %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(meta)
      : "memory");
}
__device__ __forceinline__ void tc_mma_dense_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t accumulate, uint32_t sfa, uint32_t sfb) {
  asm volatile(
      "{\n\t.reg .pred p, P;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t" GSG_ELECT
      "@P tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// Descriptor bits for the byte of the 32-bit scale words (one byte per 32 values of a 128-wide k-block)
// that an MMA's first 32 values use, in both operands.
__host__ __device__ constexpr uint32_t idesc_sf(int sf) { return ((uint32_t)sf << 4) | ((uint32_t)sf << 29); }

// The four MMAs of a microscaled chunk (dense, one UE8M0 scale per 32 values): 4-bit weights against 4-bit
// (kM8 false, K = 64 each) or 8-bit activations (K = 32), for one CTA or a CTA pair.  Each takes the next 32
// bytes of the operands' rows; idesc names the bytes of the scale words used (see idesc_sf): with 8-bit
// activations one word holds all four MMAs' scales, else two words (four columns each, kSfbStep for the
// tokens') two each.  `accumulate` is for the first of them.  (One election for the four: a stage's issue
// bounds short tiles; 30B down-projection decode, 8-bit, 26.8 -> 25.8 us.  A predicate from a register in place
// of elect.sync: 33.6 us.)
template <bool kM8, bool kPair, int kSfbStep>
__device__ __forceinline__ void tc_mma_mx_chunk(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate, uint32_t sfa, uint32_t sfb) {
#define GSG_MX_MMA(CG, KIND, A, B, I, SA, SB, ACC) \
  "@P tcgen05.mma.cta_group::" CG ".kind::" KIND ".block_scale.block32 [%0], " A ", " B ", " I ", [" SA "], [" SB "], " ACC ";\n\t"
#define GSG_MX_CHUNK(CG, KIND, S1, S2, S3)                                                              \
  asm volatile(                                                                                         \
      "{\n\t.reg .pred P, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t.reg .b32 i1, i2, i3, sa, sb;\n\t" \
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"                       \
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"                               \
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"                               \
      "or.b32 i1, %3, %7;\n\tor.b32 i2, %3, %8;\n\tor.b32 i3, %3, %9;\n\t"                              \
      "add.s32 sa, %5, %10;\n\tadd.s32 sb, %6, %11;\n\t" GSG_ELECT                                                \
      GSG_MX_MMA(CG, KIND, "%1", "%2", "%3", "%5", "%6", "p")                                           \
      GSG_MX_MMA(CG, KIND, "a1", "b1", "i1", "%5", "%6", "q")                                           \
      GSG_MX_MMA(CG, KIND, "a2", "b2", "i2", "sa", "sb", "q")                                           \
      GSG_MX_MMA(CG, KIND, "a3", "b3", "i3", "sa", "sb", "q") "}" ::                            \
      "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "n"(idesc_sf(S1)), \
      "n"(idesc_sf(S2)), "n"(idesc_sf(S3)), "n"(kM8 ? 0 : 4), "n"(kM8 ? 0 : kSfbStep)                   \
      : "memory")
  if constexpr (kM8) {
    if constexpr (kPair) GSG_MX_CHUNK("2", "mxf8f6f4", 1, 2, 3);
    else GSG_MX_CHUNK("1", "mxf8f6f4", 1, 2, 3);
  } else {
    if constexpr (kPair) GSG_MX_CHUNK("2", "mxf4", 2, 0, 2);
    else GSG_MX_CHUNK("1", "mxf4", 2, 0, 2);
  }
#undef GSG_MX_CHUNK
#undef GSG_MX_MMA
}
// Two accumulators times `scale` (the microscaled formats have none), rounded to bf16, lo in the low half.
template <bool kScaled>
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi, float scale) {
  const __nv_bfloat162 v = kScaled ? __floats2bfloat162_rn(__fmul_rn(lo, scale), __fmul_rn(hi, scale))
                                   : __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 32 accumulator columns of this lane's TMEM row, times `scale`, rounded to bf16 and packed in
// pairs: h[i] = column 2i (low half) and column 2i + 1 (high half).
template <bool kScaled>
__device__ __forceinline__ void tc_ld_32_bf16(uint32_t taddr, float scale, uint32_t h[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    h[i] = pack_bf16<kScaled>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), scale);
  }
}

__device__ __forceinline__ void tc_ld_16(uint32_t taddr, float v[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Stores kPairs * 2 tokens of a warp's 32 features, h[i] this lane's feature of tokens 2i (low half) and 2i + 1:
// neighbouring lanes trade halves, so that each holds two features of one token, and every store instruction
// writes 64 whole bytes of two tokens' rows.  (Through shared memory, in 16-byte stores, it took twice the
// load/store unit's time: 750 cycles for 32 tokens of a wide pair tile's eight epilogue warps.)
// dst: this lane's place, token (lane & 1), features (lane & ~1) and the next; left: valid tokens from the first.
template <int kPairs>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* dst, size_t ld, int left, int lane, const uint32_t* h) {
  const uint32_t sel = (lane & 1) ? 0x3276 : 0x5410;
  left -= lane & 1;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const uint32_t w = __byte_perm(h[i], __shfl_xor_sync(0xffffffffu, h[i], 1), sel);
    if (2 * i < left) *reinterpret_cast<uint32_t*>(dst) = w;
    dst += 2 * ld;
  }
}

// Shared-memory matrix descriptor (tcgen05 format): start, leading/stride byte offsets,
// version 1, layout type (0 = no swizzle, 2 = 128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | ((uint64_t)layout << 61);
}

// Instruction descriptor of kind::mxf4nvf4 block-scaled MMA: A/B E2M1, UE4M3 scales,
// K-major A and B, M = 128 (256 for a CTA pair), N = BN; bit 2 marks the sparse form (K = 128
// logical).
__host__ __device__ inline uint32_t make_idesc(bool sparse, int BN, int M = 128) {
  return (sparse ? (1u << 2) : 0u) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// The microscaled descriptors: UE8M0 scales (bit 23), E2M1 x E2M1 (kind::mxf4) or E2M1 weights x
// E4M3 activations (kind::mxf8f6f4).
__host__ __device__ inline uint32_t make_idesc_mx(bool act8, int BN, int M) {
  return (act8 ? (5u << 7) : (1u << 7) | (1u << 10)) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24);
}
struct Ctl {
  int abort;
  uint32_t tmem_base;
  int tile_begin, tile_end;   // this CTA's contiguous range of tiles
};

// A value that every lane of the warp holds alike, made known to the compiler as such: what follows from it
// stays in the uniform registers that the tensor-core instructions take, without a move per operand.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Bounded wait: true when the phase completed; false on timeout or when another role aborted.
__device__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                             uint64_t limit_ns = kWaitTimeoutNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > limit_ns) {
        *abort_flag = 1;
        set_status(status, GSG_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
  }
}

// Warp-uniform bounded wait: every lane polls, and the warp agrees on the outcome so that the
// .sync instructions that follow (elect.sync, tcgen05.ld/st) always see a converged warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          uint64_t limit_ns = kWaitTimeoutNs) {
  const bool ok = wait_bounded(bar, parity, abort_flag, status, limit_ns);
  return __all_sync(0xffffffffu, ok);
}

// Both barriers, polled together (the usual case, both complete, then costs one round trip).
__device__ __forceinline__ bool wait_warp2(uint32_t bar_a, uint32_t par_a, uint32_t bar_b, uint32_t par_b,
                                           volatile int* abort_flag, int* status) {
  const bool a = mbar_try_wait(bar_a, par_a), b = mbar_try_wait(bar_b, par_b);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return wait_warp(bar_a, par_a, abort_flag, status) && wait_warp(bar_b, par_b, abort_flag, status);
}

// One tile of this CTA: expert, n-tile, first routed row and number of rows.
struct TileDesc {
  int e, nt, r0, valid;
};

// Largest e with pref[e] <= t (pref[0] = 0, pref[E] = total tiles), then the tile's rows.
// even: the expert's token tiles share its rows evenly, in whole MMA steps of 16 tokens.
__device__ __forceinline__ TileDesc decode_tile(int t, const int* pref, const int* offs, int E, int BN, bool even) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= t) lo = mid; else hi = mid;
  }
  const int local = t - pref[lo];
  const int rows = offs[lo + 1] - offs[lo];
  const int mte = (rows + BN - 1) / BN;
  TileDesc d;
  d.e = lo;
  if (mte == 1) {   // (no divisions: this runs before the launch's first copy)
    d.nt = local;
    d.r0 = offs[lo];
    d.valid = rows;
    return d;
  }
  const int step = even ? ((rows + mte - 1) / mte + 15) & ~15 : BN;
  d.nt = local / mte;
  d.r0 = offs[lo] + (local % mte) * step;
  d.valid = max(min(step, offs[lo + 1] - d.r0), 0);
  return d;
}

// Tile schedules (tiles numbered expert-major, then n-tile, then token tile):
//  kSchedRoundRobin: tile j * grid + CTA.  Neighbouring tiles run at the same time on different
//    CTAs, so the token tiles of one weight tile and the n-tiles of one activation tile are read
//    from DRAM once and shared through L2.
//  kSchedRuns: each CTA takes a contiguous run of tiles holding an equal share of the bytes (see
//    tile_at_cost) and streams its own stretch of the weight array.  Used when every expert has
//    one token tile and the CTAs hold dozens of tiles (decode batches of 32-256 tokens on 384
//    experts: 5-10 % faster); with several token tiles per expert it loses the sharing above
//    (the 30B and 1T prefill GEMMs ran 20-60 % slower), and with a handful of tiles per CTA
//    (one token on 8 experts) it measured 20 % slower; microscaled wide tiles, 64 experts x 4096 x 7168 with
//    10944 rows: 214 us round-robin, 294 us in runs.  A reversed-order (snake) round-robin,
//    tried for the load balance of heavy token tiles, measured slower than the plain one.
constexpr int kSchedRoundRobin = 0;
constexpr int kSchedRuns = 1;

// `unit` / `nunits`: this CTA's index and the number of CTAs, or for CTA pairs the pair's index
// and the number of pairs (both CTAs of a pair take the same tiles).
__device__ __forceinline__ int tile_of(int j, int sched, int tb, int unit, int nunits) {
  if (sched == kSchedRuns) return tb + j;
  return j * nunits + unit;
}

// The j-th tile of this CTA: from the shared-memory table filled at set-up, or decoded on the
// spot past its capacity.
__device__ __forceinline__ TileDesc my_tile(int j, const int4* table, int tcap, const int* pref, const int* offs,
                                            int E, int BN, bool even, int sched, int tb, int unit, int nunits) {
  if (j < tcap) {
    const int4 v = table[j];
    return TileDesc{v.x, v.y, v.z, v.w};
  }
  return decode_tile(tile_of(j, sched, tb, unit, nunits), pref, offs, E, BN, even);
}

// Tile schedule: every CTA takes a contiguous run of tiles (expert-major, then n-tile, then token
// tile) holding an equal share of the launch's bytes.  A tile's cost is its weight bytes wc plus
// ac per token row (activation codes and scales, output); costp[e] = cost of experts < e.  Returns
// the first tile that starts at or after `target` bytes (total_tiles when none does).
__device__ __forceinline__ int tile_at_cost(long long target, const long long* costp, const int* pref,
                                            const int* offs, int E, int BN, long long wc, long long ac) {
  if (target >= costp[E]) return pref[E];
  int lo = 0, hi = E;   // largest e with costp[e] <= target: a non-empty expert
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (costp[mid] <= target) lo = mid; else hi = mid;
  }
  const int rows = offs[lo + 1] - offs[lo];
  const int mte = (rows + BN - 1) / BN;
  const long long cn = mte * wc + rows * ac;            // one n-tile's token tiles
  const long long rel = target - costp[lo];
  long long nt = rel / cn;
  const long long rem = rel - nt * cn;
  const long long cf = wc + (long long)BN * ac;         // a full token tile (all but the last)
  long long tt = (rem + cf - 1) / cf;
  if (tt >= mte) { ++nt; tt = 0; }
  return pref[lo] + (int)(nt * mte + tt);
}

// Format constants.  K values of a chunk (the packed weights' 256; half of it with 8-bit activations, whose
// operands take a byte per value in shared memory, so that a chunk is 128 bytes of a row in every format),
// 512-byte scale atoms per chunk, bytes of a weight chunk in a ring stage (the microscaled formats' scales
// have a ring of their own) and bytes per 32 weights in HBM.
__host__ __device__ constexpr int fmt_chunk_k(int fmt) { return fmt == kFmtMx8 ? kChunkK / 2 : kChunkK; }
__host__ __device__ constexpr int fmt_sf_chunk(int fmt) { return fmt == kFmtDense ? 4 : fmt == kFmtMx8 ? 1 : 2; }
__host__ __device__ constexpr int fmt_w_chunk(int fmt) {
  return fmt == kFmtSparse ? kSparseChunkBytes : fmt == kFmtDense ? kDenseChunkBytes : kMxCodeBytes;
}
__host__ __device__ constexpr int fmt_w_bytes32(int fmt) { return fmt == kFmtSparse ? 11 : fmt == kFmtDense ? 18 : 17; }
__host__ __device__ constexpr int fmt_act_row(int fmt, int K) {   // activation codes + scales of a row
  return K / fmt_chunk_k(fmt) * (128 + 4 * fmt_sf_chunk(fmt));
}
// K chunks per ring stage: short token tiles take longer stages (fewer waits per weight byte); 128-token
// tiles keep two-chunk stages, also on CTA pairs (three-chunk stages, three of them in shared memory,
// measured slower than five two-chunk stages).  Wide pair tiles: two-chunk stages for the sparse weights
// (three 62 KB stages; six one-chunk stages measured slower), one chunk for the dense control's larger
// blocks.  The microscaled formats follow the dense control.
__host__ __device__ constexpr int stage_chunks(int fmt, int BN, bool glu, int cg, bool wide = false) {
  return wide  ? (fmt == kFmtSparse ? 2 : 1)
         : glu || fmt == kFmtMx8 ? 2
         : fmt == kFmtSparse ? (BN <= 32 ? 3 : 2) : (BN <= 32 ? 2 : 1);
}
// 512-byte scale atoms that hold the scales of a tile's tokens (128 each)
__host__ __device__ constexpr int sfb_atoms(int BN) { return BN > 128 ? 2 : 1; }
// Columns of a TMEM set: the microscaled formats have no metadata and fill at most 32.
__host__ __device__ constexpr uint32_t set_cols(int fmt) { return fmt_mx(fmt) ? 32 : 64; }
__host__ __device__ constexpr uint32_t col_acc(int fmt) { return kNSets * set_cols(fmt); }   // first accumulator

// Compile-time stage geometry of one (sparse/dense, token tile, SwiGLU, CTA group) instantiation.
// With the SwiGLU epilogue a tile holds two weight n-tiles (gate rows nt*128.., up rows
// N/2 + nt*128..) that share the activation tile: two MMAs per k-block into two accumulators side
// by side.  With kCG = 2 a tile is 256 weight rows (n-tiles 2*np and 2*np + 1) x kBN tokens, run
// by a pair of CTAs on two SMs: CTA r holds n-tile 2*np + r and half of the token rows, and the
// pair's MMAs (M = 256) read both CTAs' shared memory, so each SM stages its own weights but only
// half of the shared activation tile.
template <int kFmt, int kBN, bool kGLU = false, int kCG = 1, bool kWide = false>
struct Geo {
  static_assert(kCG == 1 || (kCG == 2 && !kGLU && kBN >= 128), "CTA pairs: tiles of 128 tokens or more, plain epilogue");
  static_assert(kBN <= 128 || (kWide && fmt_mx(kFmt)), "192-token tiles: wide pair tiles of the microscaled formats");
  static_assert(!kWide || kCG == 2, "wide tiles run on CTA pairs");
  static constexpr bool kSparse = kFmt == kFmtSparse;
  static constexpr bool kMx = fmt_mx(kFmt);
  static constexpr int kNT = (kGLU || kWide) ? 2 : 1;              // weight n-tiles per tile (per CTA)
  static constexpr int kKbLogical = kSparse ? 128 : kFmt == kFmtMx8 ? 32 : 64;   // logical K per MMA
  static constexpr int kCK = fmt_chunk_k(kFmt);                    // K values of a chunk
  static constexpr int kKbPerChunk = kCK / kKbLogical;             // MMAs per chunk: 2 sparse, else 4
  static constexpr int kSfPerChunk = fmt_sf_chunk(kFmt);           // scale atoms per chunk
  static constexpr int kCPS = stage_chunks(kFmt, kBN, kGLU, kCG, kWide);
  static constexpr int kSfps = kCPS * kSfPerChunk;                 // scale atoms per stage
  static constexpr int kCB = fmt_w_chunk(kFmt);                    // weight chunk block in shared memory
  static constexpr int kCBMeta = 8192;                             // metadata offset in a chunk block
  static constexpr int kCBScale = kSparse ? 10240 : kCB - 2048;    // scale atoms offset in a chunk block (NVFP4)
  static constexpr int kBRows = kBN / kCG;                         // token rows this CTA stages
  static constexpr int kBChunk = kBRows * 128;                     // activation codes per chunk
  static constexpr int kSfbA = sfb_atoms(kBN);                     // scale atoms of the tokens per k-block
  static constexpr int kOffW = kCPS * kBChunk;                     // stage layout: B chunks | W blocks | SFB
  static constexpr int kOffSFB = kOffW + kNT * kCPS * kCB;
  static constexpr int kStage = (kOffSFB + (kMx ? 0 : kSfps * 512) + 1023) / 1024 * 1024;
  // microscaled formats: a scale ring stage, [weight n-tile][atom], then [128 tokens][atom]
  static constexpr int kScaleStage = kMx ? (kNT + kSfbA) * kSfps * 512 : 0;
  static constexpr int kScaleOffB = kNT * kSfps * 512;
  static constexpr int kMetaCols = kSparse ? 4 * kCPS * kNT : 0;   // TMEM set: meta | SFA | SFB
  static constexpr int kColSFA = kMetaCols;
  static constexpr int kColSFB = kMetaCols + 4 * kSfps * kNT;
  static constexpr int kSetUsed = kColSFB + 4 * kSfbA * kSfps;
  static constexpr uint32_t kSetCols = set_cols(kFmt), kColAcc = col_acc(kFmt);
  static constexpr uint32_t kBStep = kSparse ? 64 : 32;            // B bytes per row per MMA
  static constexpr int kBoxH = kBRows < 32 ? kBRows : 32;          // token rows per TMA box
  static constexpr int kAccStride = kBN < 32 ? 32 : kBN;
  static_assert(kSetUsed <= (int)kSetCols, "TMEM set too small");
  static_assert(kColAcc + kNT * kAccStride <= kTmemCols, "TMEM too small for one accumulator buffer");
};

// kCG = 2: launched as clusters of two CTAs (a CTA pair on two SMs) that run 256-row weight tiles
// together; see Geo.  CTA rank 0 of the pair (the leader) issues the pair's MMAs and owns the
// barriers the MMAs wait on (tfull, acce: arrived on by both CTAs' loader and epilogue warps);
// every MMA completion is signalled to the barriers of both CTAs (empty, accf).
// kNative: the dense control in the activation-stationary orientation -- the tile's 128 token rows
// are MMA operand A (M = 128, padded when fewer rows are routed) and the weight n-tile is operand
// B (N = 128); the accumulator then holds a token per TMEM lane and a feature per column.
// Combine epilogue, second phase: once every CTA of the launch has written its routed rows to their
// token slots (a bounded grid barrier on two counters of the workspace: every CTA is resident, one
// per SM), the CTAs sum each token's k slots in j order -- the scatter's arithmetic: fp32 products
// and running sum from 0, one bf16 rounding, eight outputs per thread (16-byte slot loads, the
// token's slots all in flight).  The last CTA to leave sets both counters back to zero.
__device__ void combine_tokens(const GemmParams& p, volatile int* abort_flag) {
  __shared__ int go;
  int* arrive = p.counters;
  int* depart = p.counters + 1;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();   // this CTA's slot stores before its arrival
    atomicAdd(arrive, 1);
    const uint64_t t0 = globaltimer_ns();
    int ok = 1;
    while (*reinterpret_cast<volatile int*>(arrive) < (int)gridDim.x) {
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
        set_status(p.status, GSG_ERR_DEVICE_TIMEOUT);
        ok = 0;
        break;
      }
    }
    __threadfence();   // the other CTAs' slot stores before this CTA's loads
    go = ok && !*abort_flag;
  }
  __syncthreads();
  if (go) {
    const int T = p.R / p.k;
    const unsigned n8 = (unsigned)p.N / 8u;
    const unsigned total = (unsigned)T * n8;   // T * N / 8 < 2^31 (checked on the host)
    const uint16_t* slots = static_cast<const uint16_t*>(p.Y);
    for (unsigned u = blockIdx.x * blockDim.x + threadIdx.x; u < total; u += gridDim.x * blockDim.x) {
      const int t = int(u / n8), c = int(u % n8);
      float acc[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
      for (int j0 = 0; j0 < p.k; j0 += 8) {
        float g[8];
        uint4 v[8];
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          const bool in = j0 + jj < p.k;
          g[jj] = in ? __ldca(p.gates + (size_t)t * p.k + j0 + jj) : 0.0f;
          v[jj] = in ? __ldcg(reinterpret_cast<const uint4*>(slots + ((size_t)t * p.k + j0 + jj) * p.N) + c)
                     : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          if (j0 + jj >= p.k) break;
          const uint32_t w[4] = {v[jj].x, v[jj].y, v[jj].z, v[jj].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[2 * q] = __fadd_rn(acc[2 * q], __fmul_rn(g[jj], __uint_as_float(w[q] << 16)));
            acc[2 * q + 1] = __fadd_rn(acc[2 * q + 1], __fmul_rn(g[jj], __uint_as_float(w[q] & 0xFFFF0000u)));
          }
        }
      }
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * q]));
        const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * q + 1]));
        o[q] = lo | (hi << 16);
      }
      reinterpret_cast<uint4*>(p.out + (size_t)t * p.N)[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (atomicAdd(depart, 1) == (int)gridDim.x - 1) {   // every CTA has passed the barrier
      *reinterpret_cast<volatile int*>(arrive) = 0;
      *reinterpret_cast<volatile int*>(depart) = 0;
    }
  }
}

template <int kFmt, int kBN, bool kGLU, int kCG, bool kNative = false, bool kWide = false>
__global__ void __launch_bounds__(gemm_threads(kFmt, kWide), 1)
grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap_b, const __grid_constant__ CUtensorMap tmap_b64,
                    const __grid_constant__ CUtensorMap tmap_sfb, const __grid_constant__ CUtensorMap tmap_w,
                    const GemmParams p) {
  using G = Geo<kFmt, kBN, kGLU, kCG, kWide>;
  constexpr bool kSparse = G::kSparse, kMx = G::kMx;
  constexpr int kThreads = gemm_threads(kFmt, kWide);
  constexpr bool kPair = kCG == 2;
  constexpr bool kEven = kMx && kBN >= 128;   // (shorter tiles: the schedule by bytes counts full ones)
  static_assert(!kNative || (kFmt == kFmtDense && kBN == 128 && !kGLU && kCG == 1), "native orientation: dense, 128 tokens");
  extern __shared__ uint8_t smem_raw[];
  // NT: weight n-tiles; tiles run over NT / (kNT * kCG) columns (the gate n-tiles with the SwiGLU
  // epilogue, n-tile pairs for CTA pairs)
  const int E = p.E, NT = p.N / kTileN, NTt = kMx ? ceil_div_i(NT, G::kNT * kCG) : NT / (G::kNT * kCG), KC = p.K / G::kCK;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;         // this CTA's rank in its pair
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int nunits = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int S = p.stages, NACC = kWide ? 1 : p.nacc;   // (a wide tile's two accumulators fill TMEM)
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t scale_ring = smem_u32(base) + (uint32_t)(S * G::kStage);   // microscaled formats
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + (size_t)S * G::kStage + (kMx ? kScaleRing * G::kScaleStage : 0));
  // bars: full[S], empty[S], tfull[kNSets], accf[NACC], acce[NACC], drain, never (test hook),
  // microscaled formats also sfull[kScaleRing], sempty[kScaleRing]
  const int nbars = 2 * S + kNSets + 2 * NACC + 2 + (kMx ? 2 * kScaleRing : 0);
  Ctl* ctl = reinterpret_cast<Ctl*>(bars + nbars);
  int* offs = reinterpret_cast<int*>(ctl + 1);   // [E+1]
  int* pref = offs + (E + 1);                    // [E+1]
  float* wsc = reinterpret_cast<float*>(pref + (E + 1));   // [E]
  long long* costp = reinterpret_cast<long long*>((reinterpret_cast<uintptr_t>(wsc + E) + 15) & ~uintptr_t(15));
  int4* ttab = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(costp + (E + 1)) + 15) & ~uintptr_t(15));
  // per-epilogue-warp staging buffer: 16 tokens x 32 output features (fp32 worst case), or the
  // SwiGLU epilogue's 32 x 36 fp32
  uint8_t* ostage = reinterpret_cast<uint8_t*>(ttab + p.tcap);   // [4][kOutStageBytes or kGluStageBytes]
  volatile int* abort_flag = &ctl->abort;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t sbase = smem_u32(base);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int s) { return bar0 + 8u * (2 * S + s); };
  auto accf_bar = [&](int a) { return bar0 + 8u * (2 * S + kNSets + a); };
  auto acce_bar = [&](int a) { return bar0 + 8u * (2 * S + kNSets + NACC + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + kNSets + 2 * NACC);
  const uint32_t never_bar = drain_bar + 8u;
  auto sfull_bar = [&](int s) { return never_bar + 8u * (1 + s); };
  auto sempty_bar = [&](int s) { return never_bar + 8u * (1 + kScaleRing + s); };

  // ---- set-up: barriers, TMEM, tile schedule, tensor scales (global memory only after pdl_wait)
  pdl_launch_dependents();
  if (warp == 2 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
    if (kBN >= 64) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b64)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_sfb)) : "memory");
    if (kMx) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full_bar(s), 2); mbar_init(empty_bar(s), 1); }
    for (int s = 0; s < kNSets; ++s) mbar_init(tfull_bar(s), 4 * kCG);
    for (int a = 0; a < NACC; ++a) { mbar_init(accf_bar(a), 1); mbar_init(acce_bar(a), 4 * kCG * (kWide ? 2 : 1)); }
    mbar_init(drain_bar, 1);
    mbar_init(never_bar, 1);
    if (kMx)
      for (int s = 0; s < kScaleRing; ++s) { mbar_init(sfull_bar(s), 1); mbar_init(sempty_bar(s), 4); }
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (kPair) {   // the same columns in both CTAs of the pair (both warps 1 allocate)
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&ctl->tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&ctl->tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  pdl_wait();
  if (kGLU) {
    // h scale entries that refer to rows >= R (no tile writes them): zero, shared by the CTAs
    const int r_lo = p.R > 96 ? p.R - 96 : 0, span = p.rcap - r_lo, kbh = p.N / 256;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < kbh * span * 4; i += gridDim.x * blockDim.x) {
      const int cc = i & 3, rest = i >> 2, rr = r_lo + rest % span, kb = rest / span;
      if (rr + 32 * cc >= p.R) *reinterpret_cast<uint32_t*>(p.h_scales + ((size_t)kb * p.rcap + rr) * 16 + cc * 4) = 0u;
    }
  }
  // expert offsets, clamped to [0, R] so a corrupt array can never send a copy or a store out
  // of bounds (a decreasing pair makes that expert empty), and the exclusive scan pref of
  // tiles_e = ceil(rows_e / BN) * NTt: a chunk of experts per thread, the threads' sums by warp.
  // (This runs once per launch, its instructions cold in the caches, so it is kept short: three
  // block barriers in all, and every thread works out the totals it needs itself.)
  bool bad = false;
  auto offset_at = [&](int i) {
    const int v = __ldca(p.off + i);
    if (v < 0 || v > p.R) bad = true;
    return min(max(v, 0), p.R);
  };
  auto tiles_of = [&](int e) { return (max(offs[e + 1] - offs[e], 0) + kBN - 1) / kBN * NTt; };
  const int per = (E + kThreads - 1) / kThreads;
  const int e0 = min((int)threadIdx.x * per, E), e1 = min(e0 + per, E);
  int local = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = offset_at(e), hi = offset_at(e + 1);
    if (hi < lo) bad = true;
    offs[e] = lo;
    if (e == E - 1) offs[E] = hi;
    if (!kMx) wsc[e] = __ldca(p.w_scale + e);
    local += (max(hi - lo, 0) + kBN - 1) / kBN * NTt;
  }
  __shared__ int wsum[kThreads / 32];
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int run = incl - local, total_tiles = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int n = wsum[w];
    if (w < warp) run += n;
    total_tiles += n;
  }
  for (int e = e0; e < e1; ++e) {
    pref[e] = run;
    run += tiles_of(e);
  }
  if (threadIdx.x == 0) pref[E] = total_tiles;
  if (bad) set_status(p.status, GSG_ERR_BAD_ROUTING);
  // bytes per tile: weights wc, plus ac per token row (codes, scales, output row segment)
  const long long wc = (long long)G::kNT * kCG * kTileN * p.K * fmt_w_bytes32(kFmt) / 32;
  const long long ac = fmt_act_row(kFmt, p.K) + (long long)G::kNT * kCG * kTileN * (p.y_f32 ? 4 : 2);
  if (p.sched == kSchedRuns) {   // (only the byte-balanced schedule reads the costs; uniform branch)
    // the same scan of cost_e = NTt * (ceil(rows_e / BN) * wc + rows_e * ac)
    long long local = 0;
    for (int e = e0; e < e1; ++e) {
      const int rows = max(offs[e + 1] - offs[e], 0);
      local += (long long)NTt * (((rows + kBN - 1) / kBN) * wc + rows * ac);
    }
    long long incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    __shared__ long long csum[kThreads / 32];
    if (lane == 31) csum[warp] = incl;
    __syncthreads();
    long long run = incl - local;
    for (int w = 0; w < warp; ++w) run += csum[w];
    for (int e = e0; e < e1; ++e) {
      costp[e] = run;
      const int rows = max(offs[e + 1] - offs[e], 0);
      run += (long long)NTt * (((rows + kBN - 1) / kBN) * wc + rows * ac);
    }
    if (e0 < E && e1 == E) costp[E] = run;
  }
  __syncthreads();
  int tb = 0, n_my;
  if (p.sched == kSchedRuns) {
    if (threadIdx.x == 0) {
      const long long C = costp[E];
      ctl->tile_begin = tile_at_cost(C * unit / nunits, costp, pref, offs, E, kBN, wc, ac);
      ctl->tile_end = unit == nunits - 1 ? total_tiles
                                         : tile_at_cost(C * (unit + 1) / nunits, costp, pref, offs, E, kBN, wc, ac);
    }
    __syncthreads();
    tb = uniform(ctl->tile_begin);
    n_my = uniform(ctl->tile_end) - tb;
  } else {
    // total / nunits without the integer division's instructions (a quotient below 2^22 is at most one off)
    int rounds = total_tiles >> 22 != 0 ? total_tiles / nunits
                                        : __float2int_rz(__fdividef((float)total_tiles, (float)nunits));
    int rest = total_tiles - rounds * nunits;
    if (rest < 0) { --rounds; rest += nunits; }
    if (rest >= nunits) { ++rounds; rest -= nunits; }
    n_my = uniform(rounds + (unit < rest ? 1 : 0));
  }
  // this CTA's tiles, decoded once
  for (int j = threadIdx.x; j < n_my && j < p.tcap; j += blockDim.x) {
    const TileDesc d = decode_tile(tile_of(j, p.sched, tb, unit, nunits), pref, offs, E, kBN, kEven);
    ttab[j] = make_int4(d.e, d.nt, d.r0, d.valid);
  }
  tc_fence_before();
  if constexpr (kPair) {
    cluster_sync_all();   // both CTAs' barriers initialised before either arrives on the other's
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)ctl->tmem_base);

  if (kMx && warp == kThreads / 32 - 1) {
    // =============================== scale producer (microscaled formats): the scale atoms of each stage,
    // in a ring of their own that runs ahead of the operands', so that the loader warps have them in TMEM
    // when the operands land
    int s = 0, g = 0;
    uint32_t ph = 0;
    for (int j = 0; j < n_my && !*abort_flag; ++j) {
      const TileDesc c = my_tile(j, ttab, p.tcap, pref, offs, E, kBN, kEven, p.sched, tb, unit, nunits);
      constexpr int kCPB = kChunkK / G::kCK;     // chunks of a packed chunk block
      const int KB = KC / kCPB;
      // (n-tiles past the last, in a wide tile at the end of N, are the last one again; see the epilogue)
      const int nt0 = min(c.nt * kCG * G::kNT + (int)rank, NT - 1), nt1 = min(nt0 + kCG, NT - 1);
      const size_t wblk = ((size_t)c.e * NT + nt0) * KB, wup = (size_t)(nt1 - nt0) * KB;
      bool ok = true;
      for (int kc = 0; kc < KC; kc += G::kCPS) {
        const int nch = KC - kc >= G::kCPS ? G::kCPS : KC - kc;
        if (!wait_warp(sempty_bar(s), ph ^ 1u, abort_flag, p.status)) { ok = false; break; }
        const uint32_t st = scale_ring + (uint32_t)(s * G::kScaleStage), fb = sfull_bar(s);
        mbar_arrive_expect_tx(fb, (uint32_t)(G::kNT * nch * G::kSfPerChunk * 512 + G::kSfbA * G::kSfps * 512));
        // lane t * blocks + b copies weight n-tile t's atoms of the stage's b-th block (blocks of two chunks
        // with 8-bit activations, of which a stage holds one half or both); the last lanes copy the tokens'
        const int blocks = (nch + kCPB - 1) / kCPB, t = lane / blocks, b = lane - t * blocks;
        bulk_g2s_lane(lane < G::kNT * blocks, st + (t * G::kSfps + b * kCPB * G::kSfPerChunk) * 512,
                      p.w_packed + (wblk + (t == 0 ? 0 : wup) + kc / kCPB + b) * kMxChunkBytes +
                          kMxCodeBytes + kc % kCPB * (G::kSfPerChunk * 512),
                      (nch < kCPB ? nch : kCPB) * (G::kSfPerChunk * 512u), fb);
        tma_load_2d_lane(lane > 31 - G::kSfbA, st + G::kScaleOffB + (31 - lane) * (G::kSfps * 512), &tmap_sfb,
                         2 * (c.r0 + 128 * (31 - lane)), kc * G::kSfPerChunk, fb);
        ++g;
        if (++s == kScaleRing) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
    }
    if (*abort_flag && lane == 0) {   // as the operands' producers below
      const uint64_t t0 = globaltimer_ns();
      for (int g2 = g > kScaleRing ? g - kScaleRing : 0; g2 < g; ++g2) {
        while (!mbar_try_wait(sfull_bar(g2 % kScaleRing), (uint32_t)(g2 / kScaleRing) & 1u) &&
               globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
    }
  } else if (warp == 0 || warp == 2) {
    // =============================== producers: warp 0 weights, warp 2 activations.  The copies of
    // a stage are issued from separate lanes (see bulk_g2s_lane): the TMA unit works through one
    // thread's copies one after another, so one lane issuing every copy would keep a single copy
    // in flight per producer.
    const bool wprod = warp == 0;
    int s = 0, g = 0;   // ring slot and stage counter
    uint32_t ph = 0;
    for (int j = 0; j < n_my && !*abort_flag; ++j) {
      const TileDesc c = my_tile(j, ttab, p.tcap, pref, offs, E, kBN, kEven, p.sched, tb, unit, nunits);
      // this CTA's first weight n-tile: tile c.nt spans n-tiles [c.nt * kCG * kNT, +kCG * kNT) of the
      // expert (SwiGLU: the gate n-tiles only), CTA r of a pair takes every other one from r
      constexpr int kPackedCB = kMx ? kMxChunkBytes : G::kCB;   // chunk block in the packed weights
      constexpr int kCPB = kChunkK / G::kCK;     // chunks that a block holds (two with 8-bit activations)
      const int KB = KC / kCPB;
      const int nt0 = kMx ? min(c.nt * kCG * G::kNT + (int)rank, NT - 1) : c.nt * kCG * (kWide ? 2 : 1) + (int)rank;
      const size_t wblk = ((size_t)c.e * NT + nt0) * KB;   // its first chunk block
      const uint8_t* wsrc = p.w_packed + wblk * kPackedCB;
      // its second n-tile: SwiGLU, the matching up n-tile; a wide pair tile, the next pair's
      const size_t wup = (size_t)(kMx ? min(kCG, NT - 1 - nt0) : kWide ? kCG : NT / 2) * KB;
      const uint8_t* wsrc_up = wsrc + wup * kPackedCB;
      // this CTA's token rows [r0, r0 + cnt): all of the tile's, or for a CTA pair the half of the
      // MMA's N = valid rounded up to 16 that this CTA supplies (rank 1: the upper half)
      const int nh = kPair ? ((c.valid + 15) & ~15) / 2 : kBN;
      const int r0 = c.r0 + (int)rank * nh;
      // (The leader of a microscaled pair also announces the other CTA's rows.  At least one, also where the leader's
      // half holds the whole tile: the pair's barrier has to wait for this warp of the other CTA in every stage.  A
      // warp that it does not wait for may fall a round of the ring behind, and then misreads a phase's parity.)
      const int least = kMx && kPair ? 1 : 0;
      const int cnt = min(max(c.valid - (int)rank * nh, least), nh);
      const int cnt1 = kMx && kPair ? min(max(c.valid - nh, least), nh) : 0;
      // token rows to fetch: whole 32-row boxes (BN <= 32: one box of BN rows), as few 64-row
      // boxes as possible for the larger tiles -- every TMA instruction costs the issuing warp
      const int rows = (cnt + G::kBoxH - 1) / G::kBoxH * G::kBoxH;
      const int n64 = G::kBRows >= 64 ? rows / 64 : 0;
      const int n32 = (rows - 64 * n64) / G::kBoxH;
      bool ok = true;
      for (int kc = 0; kc < KC; kc += G::kCPS) {
        const int nch = KC - kc >= G::kCPS ? G::kCPS : KC - kc;
        if (!wait_warp(empty_bar(s), ph ^ 1u, abort_flag, p.status)) { ok = false; break; }
        const uint32_t st = sbase + (uint32_t)s * G::kStage;
        const uint32_t fb = full_bar(s);
        // microscaled pairs: both CTAs' copies complete on the leader's barrier, where the MMAs wait
        const uint32_t cfb = kMx && kPair ? cluster_addr(fb, 0u) : fb;
        if (wprod) {
          // weights (+ metadata + weight scales): lane t * nch + ch copies chunk block ch of weight
          // n-tile t (t = 1: the SwiGLU up n-tile); lane 31 copies the activation scale atoms of the
          // whole tile's tokens from its first row (in both CTAs of a pair: each CTA's MMA share
          // needs the scales of all N token columns)
          if constexpr (kMx) {
            // per chunk: the 128 rows of its codes (256 values, or for 8-bit activations the chunk's half of
            // the block's, which the TMA widens to 128 bytes a row; it counts the bytes read)
            if (rank == 0) mbar_arrive_expect_tx(fb, (uint32_t)(G::kNT * nch * (kMxCodeBytes / kCPB) * kCG));
            const int t = lane / nch, ch = kc + lane - t * nch;
            const int row = (int)((wblk + (t == 0 ? 0 : wup) + ch / kCPB) * kMxChunkRows);
            const bool on = lane < G::kNT * nch;
            const uint32_t dst = st + G::kOffW + (t * G::kCPS + ch - kc) * G::kCB;
            if constexpr (kPair) tma_load_2d_lane_pair(on, dst, &tmap_w, ch % kCPB * G::kCK, row, cfb);
            else tma_load_2d_lane(on, dst, &tmap_w, ch % kCPB * G::kCK, row, cfb);
          } else {
            mbar_arrive_expect_tx(fb, (uint32_t)(G::kNT * nch * G::kCB + G::kSfps * 512));
            const int t = lane / nch, ch = lane - t * nch;
            bulk_g2s_lane(lane < G::kNT * nch, st + G::kOffW + (t * G::kCPS + ch) * G::kCB,
                          (t == 0 ? wsrc : wsrc_up) + (size_t)(kc + ch) * G::kCB, G::kCB, fb);
            tma_load_2d_lane(lane == 31, st + G::kOffSFB, &tmap_sfb, 2 * c.r0, kc * G::kSfPerChunk, fb);
          }
        } else {
          // activation codes: lane ch * nb + b copies box b (64-row boxes first) of chunk ch
          const int rows1 = (cnt1 + G::kBoxH - 1) / G::kBoxH * G::kBoxH;
          if (!(kMx && kPair) || rank == 0) mbar_arrive_expect_tx(fb, (uint32_t)(nch * (rows + rows1) * 128));
          const int nb = n64 + n32;
          const int ch = nb > 0 ? lane / nb : 0, b = lane - ch * nb;
          const bool b64 = b < n64;
          const int roff = b64 ? 64 * b : 64 * n64 + (b - n64) * G::kBoxH;
          const uint32_t dst = st + ch * G::kBChunk + roff * 128;
          if constexpr (kMx && kPair)
            tma_load_2d_lane_pair(lane < nch * nb, dst, b64 ? &tmap_b64 : &tmap_b, (kc + ch) * 128, r0 + roff, cfb);
          else
            tma_load_2d_lane(lane < nch * nb, dst, b64 ? &tmap_b64 : &tmap_b, (kc + ch) * 128, r0 + roff, fb);
        }
        ++g;
        if (++s == S) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
    }
    if (*abort_flag && lane == 0) {
      // wait (2 s in all) for copies still landing in the stages this warp filled: the last S
      // before stage g (the first one it did not issue)
      // (the second CTA of a microscaled pair has no barrier of its own for them: it gives them 10 ms, a
      // thousand times what a copy takes, and leaves only after the leader's wait, at the cluster barrier)
      const uint64_t t0 = globaltimer_ns();
      if (kMx && kPair && rank != 0)
        while (globaltimer_ns() - t0 < 10000000ull) {
        }
      else
      for (int g2 = g > S ? g - S : 0; g2 < g; ++g2) {
        while (!mbar_try_wait(full_bar(g2 % S), (uint32_t)(g2 / S) & 1u) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
    }
  } else if (warp >= 7 && warp <= 10) {
    // =============================== metadata / scale loaders (TMEM quadrant q = warp % 4)
    const int q = warp & 3;
    const int row = 32 * q + lane;
    const uint32_t tlane = (uint32_t)(32 * q) << 16;
    int s = 0, set = 0, i = 0;
    uint32_t ph = 0;
    for (int j = 0; j < n_my && !*abort_flag; ++j) {
      bool ok = true;
      for (int kc = 0; kc < KC; kc += G::kCPS) {
        const int nch = KC - kc >= G::kCPS ? G::kCPS : KC - kc;
        // the TMEM set is free once the MMAs of the stage that last used it have completed
        if (i >= kNSets) {
          const int j = i - kNSets;
          if (!wait_warp(empty_bar(j % S), (uint32_t)(j / S) & 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
        }
        if (!wait_warp(kMx ? sfull_bar(s) : full_bar(s), ph, abort_flag, p.status)) { ok = false; break; }
        const uint32_t st = kMx ? scale_ring + (uint32_t)(s * G::kScaleStage) : sbase + (uint32_t)s * G::kStage;
        uint32_t r[G::kSetUsed];
        if (kSparse) {
#pragma unroll
          for (int t = 0; t < G::kNT; ++t)
#pragma unroll
            for (int ch = 0; ch < G::kCPS; ++ch)
              if (ch < nch) {
                const int m = 4 * (t * G::kCPS + ch);
                lds128(st + G::kOffW + (t * G::kCPS + ch) * G::kCB + G::kCBMeta + row * 16, r[m], r[m + 1], r[m + 2],
                       r[m + 3]);
              }
        }
#pragma unroll
        for (int kb = 0; kb < G::kSfps; ++kb) {
          if (kb < nch * G::kSfPerChunk) {
#pragma unroll
            for (int t = 0; t < G::kNT; ++t) {
              const uint32_t sfa = kMx ? st + (t * G::kSfps + kb) * 512
                                       : st + G::kOffW + (t * G::kCPS + kb / G::kSfPerChunk) * G::kCB + G::kCBScale +
                                             (kb % G::kSfPerChunk) * 512;
              const int m = G::kColSFA + 4 * (t * G::kSfps + kb);
              lds128(sfa + lane * 16, r[m], r[m + 1], r[m + 2], r[m + 3]);
            }
#pragma unroll
            for (int a = 0; a < G::kSfbA; ++a) {   // (tokens 128 and up: the next four columns)
              const int m = G::kColSFB + 4 * (G::kSfbA * kb + a);
              lds128(st + (kMx ? G::kScaleOffB : G::kOffSFB) + (a * G::kSfps + kb) * 512 + lane * 16, r[m], r[m + 1],
                     r[m + 2], r[m + 3]);
            }
          }
        }
        tc_st_cols<G::kSetUsed>(tmem + tlane + (uint32_t)set * G::kSetCols, r);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {   // the set (and, for a pair, this CTA's stage) is ready for the MMA issuer
          // The scale ring's stage is free only now that the stores above have taken the atoms from their registers.
          // Right after the loads it is not: an arrive does not wait for them, and behind the epilogue's stores they
          // may still be on their way when the next copy lands (one launch in 1500 of 192-token tiles came out wrong).
          if constexpr (kMx) mbar_arrive(sempty_bar(s));
          if constexpr (kPair) mbar_arrive_cluster(cluster_addr(tfull_bar(set), 0u));
          else mbar_arrive(tfull_bar(set));
        }
        ++i;
        if (++set == kNSets) set = 0;
        if (++s == (kMx ? kScaleRing : S)) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
    }
  } else if (warp == 1) {
    // =============================== MMA issuer (whole warp, one elected lane issues); for a CTA
    // pair only the leader's, whose MMAs run on both SMs (the other CTA's warp 1 has no tiles)
    int s = 0, set = 0, acc = 0;
    uint32_t ph = 0, sph = 0, aph = 0;   // phases of the ring, the TMEM sets, the accumulators
    bool any = false;
    const int n_mma = rank == 0u ? n_my : 0;
    for (int j = 0; j < n_mma && !*abort_flag; ++j) {
      const TileDesc c = my_tile(j, ttab, p.tcap, pref, offs, E, kBN, kEven, p.sched, tb, unit, nunits);
      const int nval = uniform((c.valid + 15) & ~15);   // the MMA's N
      const uint32_t idesc = kMx ? make_idesc_mx(kFmt == kFmtMx8, nval, kTileN * kCG)
                             : kNative ? make_idesc(false, kTileN, kBN)   // M = 128 tokens, N = 128 weight rows
                                     : make_idesc(kSparse, nval, kTileN * kCG);
      if (p.stall_ns != 0ull && j == (n_mma > 1 ? 1 : 0) &&
          !wait_warp(never_bar, 0u, abort_flag, p.status, p.stall_ns))
        break;
      if (!wait_warp(acce_bar(acc), aph ^ 1u, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + G::kColAcc + (uint32_t)(acc * G::kNT * G::kAccStride);
      bool ok = true;
      for (int kc = 0; kc < KC; kc += G::kCPS) {
        const int nch = KC - kc >= G::kCPS ? G::kCPS : KC - kc;
        if (!wait_warp2(full_bar(s), ph, tfull_bar(set), sph, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = sbase + (uint32_t)s * G::kStage;
        const uint32_t tset = tmem + (uint32_t)set * G::kSetCols;
        if constexpr (kMx) {
#pragma unroll
          for (int ch = 0; ch < G::kCPS; ++ch)
            if (ch < nch) {
#pragma unroll
              for (int t = 0; t < G::kNT; ++t)
                tc_mma_mx_chunk<kFmt == kFmtMx8, kPair, 4 * G::kSfbA>(
                    d_tmem + (uint32_t)(t * G::kAccStride),
                    smem_desc(st + G::kOffW + (t * G::kCPS + ch) * G::kCB, 16, 1024, 2),
                    smem_desc(st + ch * G::kBChunk, 16, 1024, 2), idesc, (kc | ch) != 0 ? 1u : 0u,
                    tset + G::kColSFA + 4 * (t * G::kSfps + ch * G::kSfPerChunk),
                    tset + G::kColSFB + 4 * G::kSfbA * ch * G::kSfPerChunk);
            }
        } else {
#pragma unroll
          for (int ch = 0; ch < G::kCPS; ++ch) {
            if (ch < nch) {
#pragma unroll
              for (int h = 0; h < G::kKbPerChunk; ++h) {
                const int kbi = ch * G::kSfPerChunk + h;   // scale atom
                const uint64_t bdesc = smem_desc(st + ch * G::kBChunk + G::kBStep * h, 16, 1024, 2);
                const uint32_t accum = (kc | ch | h) != 0 ? 1u : 0u;
#pragma unroll
                for (int t = 0; t < G::kNT; ++t) {
                  const uint32_t aaddr = st + G::kOffW + (t * G::kCPS + ch) * G::kCB + 4096u * h;
                  const uint64_t adesc = smem_desc(aaddr, 128, 256, 0);
                  const uint32_t d = d_tmem + (uint32_t)(t * G::kAccStride);
                  const int kt = t * G::kSfps + kbi;
                  const uint32_t sfa = tset + G::kColSFA + 4 * kt, sfb = tset + G::kColSFB + 4 * kbi;
                  if constexpr (kNative)   // tokens as A, weights as B: the operands and their scales swap
                    tc_mma_dense(d, bdesc, adesc, idesc, accum, sfb, sfa);
                  else if constexpr (kSparse && kPair)
                    tc_mma_sparse_pair(d, adesc, bdesc, idesc, accum, sfa, sfb, tset + 2 * kt);
                  else if constexpr (kSparse)
                    tc_mma_sparse(d, adesc, bdesc, idesc, accum, sfa, sfb, tset + 2 * kt);
                  else if constexpr (kPair)
                    tc_mma_dense_pair(d, adesc, bdesc, idesc, accum, sfa, sfb);
                  else
                    tc_mma_dense(d, adesc, bdesc, idesc, accum, sfa, sfb);
                }
              }
            }
          }
        }
        if constexpr (kPair) tc_commit_pair(empty_bar(s), 3);   // the stage is free in both CTAs
        else tc_commit(empty_bar(s));
        any = true;
        if (++set == kNSets) { set = 0; sph ^= 1u; }
        if (++s == S) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if constexpr (kPair) tc_commit_pair(accf_bar(acc), 3);   // both CTAs' epilogues
      else tc_commit(accf_bar(acc));
      if (++acc == NACC) { acc = 0; aph ^= 1u; }
    }
    __syncwarp();
    if (any) {
      // all MMAs issued by this warp have completed once the drain barrier fires
      if constexpr (kPair) tc_commit_pair(drain_bar, 1);
      else tc_commit(drain_bar);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
  } else {
    // =============================== epilogue (warps 3..6, and 11..14 for wide tiles -> TMEM lane
    // quadrants 3,0,1,2)
    const int q = warp & 3;
    const float sx = kMx ? 1.0f : __ldca(p.x_scale);
    int acc = 0;
    uint32_t aph = 0;
    for (int j = 0; j < n_my; ++j) {
      const TileDesc c = my_tile(j, ttab, p.tcap, pref, offs, E, kBN, kEven, p.sched, tb, unit, nunits);
      // (an n-tile past the last, in a microscaled format's wide tile at the end of N, is computed like any
      // other and not stored)
      const bool past = kMx && kWide && (2 * c.nt + (warp >= 11 ? 1 : 0)) * kCG + (int)rank >= NT;
      const int r0 = c.r0, valid = past ? 0 : c.valid;
      if (!wait_warp(accf_bar(acc), aph, abort_flag, p.status)) break;
      tc_fence_after();
      const float scale = kMx ? 1.0f : __fmul_rn(sx, wsc[c.e]);
      const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + G::kColAcc + (uint32_t)(acc * G::kNT * G::kAccStride);
      bool released = false;   // the accumulator already handed back to the MMA warp
      if constexpr (kNative) {
        // lane = token 32q + lane of the tile, columns = the n-tile's 128 features: each lane scales
        // and stores its own token's row segment (16-byte stores, 16 features at a time)
        const int tok = 32 * q + lane;
        const size_t col0 = (size_t)c.nt * kTileN;
        for (int f0 = 0; f0 < kTileN; f0 += 16) {
          float v[16];
          tc_ld_16(taddr + f0, v);
          if (tok < valid) {
            if (p.y_f32) {
              float* Yr = static_cast<float*>(p.Y) + (size_t)(r0 + tok) * p.N + col0 + f0;
#pragma unroll
              for (int w = 0; w < 4; ++w)
                *reinterpret_cast<float4*>(Yr + 4 * w) =
                    make_float4(__fmul_rn(v[4 * w], scale), __fmul_rn(v[4 * w + 1], scale),
                                __fmul_rn(v[4 * w + 2], scale), __fmul_rn(v[4 * w + 3], scale));
            } else {
              uint32_t pk[8];
#pragma unroll
              for (int w = 0; w < 8; ++w)
                pk[w] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(v[2 * w], scale))) |
                        ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(v[2 * w + 1], scale))) << 16);
              uint4* Yr = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.Y) + (size_t)(r0 + tok) * p.N + col0 + f0);
              Yr[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              Yr[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            }
          }
        }
      } else if constexpr (kGLU) {
        // SwiGLU output preparation, 32 tokens at a time: lane = feature f of this warp's
        // 32-feature block (one NVFP4 block of the down-projection's K), h = silu(gate) * up in
        // fp32; the block is transposed through shared memory so that each lane then owns one
        // token's 32 values: block max, UE4M3 scale and E2M1 codes once per token, 16-byte code
        // stores, scale bytes into the quad layout (k-block nt, position q).
        const float sh = __ldca(p.h_scale);
        const float six_sh = __fmul_rn(6.0f, sh);
        const int f0 = c.nt * kTileN + 32 * q;
        const int hrow = p.N / 4;                 // bytes of h codes per row (N/2 features)
        uint8_t* hc = static_cast<uint8_t*>(p.Y);
        const uint32_t tb = smem_u32(ostage + (size_t)(warp - 3) * kGluStageBytes);   // [32][36] fp32
        for (int c0 = 0; c0 < valid; c0 += 32) {
          float g[32], u[32];
          tc_ld_16(taddr + c0, g);
          tc_ld_16(taddr + c0 + 16, g + 16);
          tc_ld_16(taddr + G::kAccStride + c0, u);
          tc_ld_16(taddr + G::kAccStride + c0 + 16, u + 16);
#pragma unroll
          for (int t = 0; t < 32; ++t) {
            const float gs = __fmul_rn(g[t], scale), us = __fmul_rn(u[t], scale);
            const float hv = __fmul_rn(__fdividef(gs, __fadd_rn(1.0f, __expf(-gs))), us);
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(tb + (uint32_t)(t * 36 + lane) * 4u), "f"(hv) : "memory");
          }
          __syncwarp();
          float v[32];
#pragma unroll
          for (int k4 = 0; k4 < 8; ++k4) {
            uint32_t a, b, cc, d;
            lds128(tb + (uint32_t)(lane * 36 + 4 * k4) * 4u, a, b, cc, d);
            v[4 * k4] = __uint_as_float(a);
            v[4 * k4 + 1] = __uint_as_float(b);
            v[4 * k4 + 2] = __uint_as_float(cc);
            v[4 * k4 + 3] = __uint_as_float(d);
          }
          __syncwarp();
          float am = 0.0f;
#pragma unroll
          for (int k = 0; k < 32; ++k) am = fmaxf(am, fabsf(v[k]));
          const BlockScale bs = block_scale_cvt(am, six_sh, sh);
          uint32_t wd[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            float xs[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) xs[i] = __fmul_rn(v[8 * w + i], bs.inv);
            wd[w] = e2m1_encode8_cvt(xs);
          }
          const int row = r0 + c0 + lane;
          if (c0 + lane < valid) {
            *reinterpret_cast<uint4*>(hc + (size_t)row * hrow + f0 / 2) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              const int rr = row - 32 * cc;
              if (rr >= 0) p.h_scales[((size_t)c.nt * p.rcap + rr) * 16 + cc * 4 + q] = (uint8_t)bs.sc;
            }
          }
        }
      } else {
      // Each 16-token chunk: TMEM lane (= output feature) -> registers, scale, transpose through
      // the warp's shared buffer into [token][32 features], then 16-byte stores of whole row
      // segments (64 B bf16 / 128 B fp32 per token).
      uint8_t* obuf = ostage + (size_t)(warp >= 11 ? warp - 7 : warp - 3) * kOutStageBytes;
      const uint32_t obuf_s = smem_u32(obuf);
      // the tile's n-tiles: a wide pair tile's second one goes to warps 11..14
      const int u_begin = kWide ? (warp >= 11 ? 1 : 0) : 0, u_end = kWide ? u_begin + 1 : G::kNT;
      if constexpr (kBN >= 128 && G::kNT == 1 + (kWide ? 1 : 0)) {
        if (!p.y_f32 && p.perm_src == nullptr) {
          // bf16 output of a tile of 128 tokens or more (one n-tile per warp): the warp's whole accumulator
          // block in 32-column TMEM loads, held as packed bf16, and the accumulator released
          // before any store, so the MMA warp's next tile waits for the loads, not for the stores
          const uint32_t tcol = taddr + (uint32_t)(u_begin * G::kAccStride);
          const int col0 = (c.nt * kCG * G::kNT + u_begin * kCG + (int)rank) * kTileN + 32 * q;
          // tokens t0 .. t0 + 31 of the tile, h16[i] this lane's feature of tokens t0 + 2i (low half) and t0 + 2i + 1
          // (NVFP4, whose extra scaling leaves fewer registers: through the warp's buffer, sixteen tokens at a time)
          auto store32 = [&](int t0, const uint32_t* h16) {
            if constexpr (!kMx) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                if (t0 + 16 * g < valid) {
#pragma unroll
                  for (int j = 0; j < 16; j += 2) {
                    const uint32_t w = h16[8 * g + j / 2];
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(obuf_s + (uint32_t)(j * 64 + lane * 2)),
                                 "h"((unsigned short)(w & 0xffffu)) : "memory");
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(obuf_s + (uint32_t)((j + 1) * 64 + lane * 2)),
                                 "h"((unsigned short)(w >> 16)) : "memory");
                  }
                  __syncwarp();
#pragma unroll
                  for (int k = 0; k < 2; ++k) {   // 16 tokens x 4 chunks of 16 B
                    const int ci = lane + 32 * k, tok = ci >> 2, part = ci & 3;
                    if (t0 + 16 * g + tok < valid) {
                      uint32_t a, b, cc, d;
                      lds128(obuf_s + (uint32_t)(tok * 64 + part * 16), a, b, cc, d);
                      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.Y) + (size_t)(r0 + t0 + 16 * g + tok) * p.N +
                                                col0 + part * 8) = make_uint4(a, b, cc, d);
                    }
                  }
                  __syncwarp();
                }
              }
              return;
            }
            store_pairs<16>(static_cast<__nv_bfloat16*>(p.Y) + (size_t)(r0 + t0 + (lane & 1)) * p.N + col0 + (lane & ~1),
                            (size_t)p.N, valid - t0, lane, h16);
          };
          // (128 tokens are what a thread's registers hold; a 192-token tile's others are stored first)
          if constexpr (kBN > 128) {
#pragma unroll 1
            for (int t0 = 128; t0 < valid; t0 += 32) {
              uint32_t h16[16];
              tc_ld_32_bf16<!kMx>(tcol + t0, scale, h16);
              store32(t0, h16);
            }
          }
          uint32_t hb[64];
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (32 * h < valid) tc_ld_32_bf16<!kMx>(tcol + 32u * h, scale, hb + 16 * h);   // warp-uniform
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair) mbar_arrive_cluster(cluster_addr(acce_bar(acc), 0u));
            else mbar_arrive(acce_bar(acc));
          }
          released = true;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (32 * g < valid) store32(32 * g, hb + 16 * g);   // warp-uniform
        }
      }
      const bool direct = kBN >= 128 && G::kNT == 1 + (kWide ? 1 : 0) && !p.y_f32 && p.perm_src == nullptr;
      for (int u = u_begin; u < u_end && !direct; ++u) {
        // first feature of this warp
        const size_t col0 = ((size_t)c.nt * kCG * G::kNT + u * kCG + rank) * kTileN + 32 * q;
        for (int c0 = 0; c0 < valid; c0 += 16) {
          float v[16];
          tc_ld_16(taddr + (uint32_t)(u * G::kAccStride) + c0, v);
          if (p.y_f32) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(obuf_s + (uint32_t)(j * 128 + lane * 4)),
                           "f"(__fmul_rn(v[j], scale)) : "memory");
            __syncwarp();
            float* Y = static_cast<float*>(p.Y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {          // 16 tokens x 8 chunks of 16 B
              const int ci = lane + 32 * k, tok = ci >> 3, part = ci & 7;
              if (c0 + tok < valid) {
                uint32_t a, b, cc, d;
                lds128(obuf_s + (uint32_t)(tok * 128 + part * 16), a, b, cc, d);
                *reinterpret_cast<uint4*>(Y + (size_t)(r0 + c0 + tok) * p.N + col0 + part * 4) =
                    make_uint4(a, b, cc, d);
              }
            }
          } else if constexpr (kMx) {
            uint32_t h8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h8[j] = pack_bf16<false>(v[2 * j], v[2 * j + 1], 1.0f);
            store_pairs<8>(static_cast<__nv_bfloat16*>(p.Y) + (size_t)(r0 + c0 + (lane & 1)) * p.N + col0 + (lane & ~1),
                           (size_t)p.N, valid - c0, lane, h8);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const unsigned short h = __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(v[j], scale)));
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(obuf_s + (uint32_t)(j * 64 + lane * 2)), "h"(h) : "memory");
            }
            __syncwarp();
            __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(p.Y);
            // combine: lane j < 16 holds the flat index f = t*k + j of chunk row j; the row goes to
            // slot f instead of row r
            const bool comb = p.perm_src != nullptr;
            int myf = (comb && lane < 16 && c0 + lane < valid) ? __ldca(p.perm_src + r0 + c0 + lane) : 0;
            // a slot index outside [0, T*k) (corrupt routing) gets nothing stored
            const unsigned badf = __ballot_sync(0xffffffffu, comb && lane < 16 && c0 + lane < valid &&
                                                                 (myf < 0 || myf >= p.R));
            if (badf != 0u && lane == 0) set_status(p.status, GSG_ERR_BAD_ROUTING);
            if ((badf >> lane) & 1u) myf = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {          // 16 tokens x 4 chunks of 16 B
              const int ci = lane + 32 * k, tok = ci >> 2, part = ci & 3;
              const int f = __shfl_sync(0xffffffffu, myf, tok);
              if (c0 + tok < valid && !((badf >> tok) & 1u)) {
                uint32_t a, b, cc, d;
                lds128(obuf_s + (uint32_t)(tok * 64 + part * 16), a, b, cc, d);
                const size_t dst = comb ? (size_t)f : (size_t)(r0 + c0 + tok);
                *reinterpret_cast<uint4*>(Y + dst * p.N + col0 + part * 8) = make_uint4(a, b, cc, d);
              }
            }
          }
          __syncwarp();
        }
      }
      }
      if (!released) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {   // the accumulator may be overwritten (for a pair: once both CTAs read it)
          if constexpr (kPair) mbar_arrive_cluster(cluster_addr(acce_bar(acc), 0u));
          else mbar_arrive(acce_bar(acc));
        }
      }
      if (++acc == NACC) { acc = 0; aph ^= 1u; }
    }
  }

  // ---- teardown (a CTA of a pair leaves only once the other is done with its shared memory and
  // barriers: the leader's MMAs read both CTAs' stages, and both CTAs arrive on the leader's
  // barriers)
  tc_fence_before();
  if constexpr (kPair) {
    __syncwarp();          // the cluster barrier is executed by converged warps
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
  if (p.perm_src != nullptr) combine_tokens(p, abort_flag);
}

// ------------------------------------------------------------------ host side
struct GemmPlan {
  int BN, cps, stage, stages, nacc, tcap;
  size_t smem;
};

constexpr int kMaxStages = 12;
constexpr int kStageBudget128 = 192 * 1024;   // 128-token tiles: a deeper ring only adds L2 pressure
// opt-in dynamic shared memory per block minus room for static shared memory (set per device)
static int g_smem_limit = 232448 - 1024;

// tcap: capacity of the per-CTA tile table (tiles beyond it are decoded on the fly); an upper
// bound on a CTA's tiles is ceil((ceil(R/BN) + E) * NT / grid).  cg = 2: a CTA of a pair, which
// stages half of the tile's token rows (the geometry of Geo<..., 2>).
static GemmPlan make_plan(int fmt, int BN, int E, int tcap, bool glu = false, int cg = 1, bool wide = false) {
  GemmPlan g;
  g.BN = BN;
  g.tcap = tcap;
  // weight n-tiles per tile and CTA: gate + up with the SwiGLU epilogue, two n-tile pairs for a
  // wide pair tile
  const int nt = glu || wide ? 2 : 1;
  g.cps = stage_chunks(fmt, BN, glu, cg, wide);
  const int sfps = g.cps * fmt_sf_chunk(fmt);
  const int body = g.cps * (BN / cg) * 128 + nt * g.cps * fmt_w_chunk(fmt) + (fmt_mx(fmt) ? 0 : sfps * 512);
  g.stage = (body + 1023) / 1024 * 1024;
  // everything but the stage ring and the tile table, at its largest
  const int ostage = (wide ? 8 : 4) * (glu ? kGluStageBytes : kOutStageBytes);
  // the microscaled formats' scale ring and its barriers
  const int sring = fmt_mx(fmt) ? kScaleRing * ((nt + sfb_atoms(BN)) * sfps * 512 + 16) : 0;
  const int fixed = 1024 + (2 * kMaxStages + kNSets + 2 * kMaxAcc + 2) * 8 + (int)sizeof(Ctl) + (3 * E + 2) * 4 +
                    16 + (E + 1) * 8 + 16 + ostage + sring;
  int budget = g_smem_limit - fixed;
  if (BN == 128 && cg == 1 && budget > kStageBudget128) budget = kStageBudget128;
  g.stages = (budget - tcap * 16) / g.stage;
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  // the ring comes before the tile table: where the table would cost a stage, it keeps only what
  // fits beside the full ring (a CTA decodes its later tiles from the expert offsets instead)
  int ring = budget / g.stage;
  if (ring > kMaxStages) ring = kMaxStages;
  if (g.stages < ring) {
    g.stages = ring;
    g.tcap = (budget - ring * g.stage) / 16;
  }
  const int acc_stride = (BN < 32 ? 32 : BN) * nt;
  g.nacc = (int)((kTmemCols - col_acc(fmt)) / acc_stride);
  if (g.nacc > kMaxAcc) g.nacc = kMaxAcc;
  const int nbars = 2 * g.stages + kNSets + 2 * g.nacc + 2;
  g.smem = 1024 + (size_t)g.stages * g.stage + nbars * 8 + sizeof(Ctl) + (size_t)(3 * E + 2) * 4 + 16 +
           (size_t)(E + 1) * 8 + 16 +
           (size_t)g.tcap * 16 + ostage + sring;
  return g;
}

constexpr int kMaxTableTiles = 1024;

// test hook: the MMA warp's stall of GemmParams::stall_ns for the launches that follow (0 = off)
static std::atomic<unsigned long long> g_test_stall_ns{0ull};
void gemm_set_test_stall(unsigned long long ns) { g_test_stall_ns.store(ns); }
// test hook: at most this many entries of the per-CTA tile table (-1 = no limit); the tiles past
// it are decoded from the expert offsets as the roles reach them
static std::atomic<int> g_test_table_cap{-1};
void gemm_set_test_table_cap(int cap) { g_test_table_cap.store(cap); }

// Token tile: the smallest of 16/32/64 that holds the largest expert; past 64 rows, 128 only when
// experts average at least 64 rows (R / E), since a 128-row activation chunk takes shared memory
// from the weight ring that the many small experts of a skewed routing would leave unused.
int gemm_pick_bn(int max_rows, int R, int E) {
  if (max_rows > 0 && max_rows <= 16) return 16;
  if (max_rows > 0 && max_rows <= 32) return 32;
  if (max_rows > 0 && max_rows <= 64) return 64;
  return (long long)R >= 64ll * E ? 128 : 64;
}

// Token tile of the microscaled formats.  Up to 32 rows in every expert: the smallest tile that holds them,
// one CTA per tile.  Beyond: 64 tokens on one CTA, or 128 or 192 on a wide pair tile, whichever an estimate in
// SM cycles (1.9 GHz) makes cheaper for experts of R / E rows each.  `chunks` ring stages make a tile; a wide
// one takes max(620, 4 N) cycles for N tokens (4 N: the tensor pipe's time for 512 x N x one chunk; 620:
// issuing it), its single accumulator buffer costs 1500 or 2600 more between tiles, and the pair launch about
// 4000 at its ends; a 64-token stage takes 700 (470 with 8-bit activations, half as long).  Measured, 4-bit,
// 64 / 128 / 192 tokens: 32 experts x 100 rows, N = 1280, K = 2048 19.5 / 14.6 / 14.9 us; 8 x 100, N = K = 1024 5.6 /
// 7.4 / 7.4; 64 x 300, N = 768, K = 2048 44 / 30.5 / 27.7; N = 4096, K = 7168: one expert x 128 rows 13.7 / 16.7 / 17.2,
// x 1023 rows 43.9 / 18.9 / 20.6, 4 x 1100 rows 164 / 61 / 55.6, 16 x 171 rows 114 / 63 / 52, 16 x 256 rows 144 / 70 / 71.
static int mx_pick_bn(int max_rows, int R, int E, int N, int chunks, bool act8, int num_sms, int pairs) {
  if (max_rows > 0 && max_rows <= 16) return 16;
  if (max_rows > 0 && max_rows <= 32) return 32;
  if (pairs == 0) return 64;
  const int bns[3] = {64, 128, 192};
  const long long rows = ((long long)R + E - 1) / E, nt = N / kTileN;
  long long best = 0;
  int bn = 64;
  for (int i = 0; i < 3; ++i) {
    const bool wide = bns[i] > 64;
    const long long n = (rows + bns[i] - 1) / bns[i], units = wide ? pairs : num_sms;
    const long long tokens = ((rows + n - 1) / n + 15) / 16 * 16;
    const long long waves = (n * E * (wide ? (nt + 3) / 4 : nt) + units - 1) / units;
    const long long stage = !wide ? (act8 ? 470 : 700) : 4 * tokens > 620 ? 4 * tokens : 620;
    const long long cost = (wide ? 4000 : 0) + waves * (chunks * stage + (i == 0 ? 1000 : i == 1 ? 1500 : 2600));
    if (i == 0 || cost < best) { best = cost; bn = bns[i]; }
  }
  return bn;
}

bool gemm_supported(int E) { return E >= 1 && E <= kMaxE; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  return fn;
}

template <int kFmt, int kBN, bool kGLU = false, int kCG = 1, bool kNative = false, bool kWide = false>
static cudaError_t set_attr_one(int bytes) {
  return cudaFuncSetAttribute(grouped_gemm_kernel<kFmt, kBN, kGLU, kCG, kNative, kWide>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// CTA pairs the device can hold at once at one CTA per SM (the pairs' SMs must share a GPC), per
// format; 0 when the device cannot run them (then 128-token tiles run one CTA per tile).
static int g_pair_units[4] = {0, 0, 0, 0};
static int g_wide_units[4] = {0, 0, 0, 0};   // the same for the wide pair tiles

template <int kFmt, bool kWide = false>
static int max_pairs(int smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(gemm_threads(kFmt, kWide));
  cfg.dynamicSmemBytes = (size_t)smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, grouped_gemm_kernel<kFmt, 128, false, 2, false, kWide>, &cfg) !=
      cudaSuccess) {
    cudaGetLastError();   // clear the error: pairs are then simply not used
    return 0;
  }
  return n;
}

cudaError_t gemm_set_smem_attrs() {
  // every plan stays below the opt-in limit (make_plan sizes the ring from it)
  int dev = 0, maxb = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&maxb, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;
  maxb -= 1024;   // room for the kernels' static shared memory
  g_smem_limit = maxb;
  constexpr int D = kFmtDense, S = kFmtSparse, M4 = kFmtMx4, M8 = kFmtMx8;
  const cudaError_t errs[] = {
      set_attr_one<S, 16>(maxb), set_attr_one<S, 32>(maxb), set_attr_one<S, 64>(maxb), set_attr_one<S, 128>(maxb),
      set_attr_one<D, 16>(maxb), set_attr_one<D, 32>(maxb), set_attr_one<D, 64>(maxb), set_attr_one<D, 128>(maxb),
      set_attr_one<S, 16, true>(maxb), set_attr_one<S, 32, true>(maxb), set_attr_one<S, 64, true>(maxb),
      set_attr_one<S, 128, false, 2>(maxb), set_attr_one<D, 128, false, 2>(maxb),
      set_attr_one<D, 128, false, 1, true>(maxb), set_attr_one<S, 128, false, 2, false, true>(maxb),
      set_attr_one<D, 128, false, 2, false, true>(maxb),
      set_attr_one<M4, 16>(maxb), set_attr_one<M4, 32>(maxb), set_attr_one<M4, 64>(maxb),
      set_attr_one<M8, 16>(maxb), set_attr_one<M8, 32>(maxb), set_attr_one<M8, 64>(maxb),
      set_attr_one<M4, 128, false, 2, false, true>(maxb), set_attr_one<M8, 128, false, 2, false, true>(maxb),
      set_attr_one<M4, 192, false, 2, false, true>(maxb), set_attr_one<M8, 192, false, 2, false, true>(maxb)};
  for (cudaError_t x : errs)
    if (x != cudaSuccess) return x;
  g_pair_units[S] = max_pairs<S>(maxb);
  g_pair_units[D] = max_pairs<D>(maxb);
  g_wide_units[S] = max_pairs<S, true>(maxb);
  g_wide_units[D] = max_pairs<D, true>(maxb);
  g_wide_units[M4] = max_pairs<M4, true>(maxb);
  g_wide_units[M8] = max_pairs<M8, true>(maxb);
  return cudaSuccess;
}

template <int kFmt, bool kGLU = false>
static cudaError_t launch_bn(int BN, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& tb,
                             const CUtensorMap& tb64, const CUtensorMap& ts, const CUtensorMap& tw,
                             const GemmParams& p) {
  switch (BN) {
    case 16: return launch_pdl(grouped_gemm_kernel<kFmt, 16, kGLU, 1>, grid, gemm_threads(kFmt, false), smem, stream, tb, tb64, ts, tw, p);
    case 32: return launch_pdl(grouped_gemm_kernel<kFmt, 32, kGLU, 1>, grid, gemm_threads(kFmt, false), smem, stream, tb, tb64, ts, tw, p);
    default: return launch_pdl(grouped_gemm_kernel<kFmt, 64, kGLU, 1>, grid, gemm_threads(kFmt, false), smem, stream, tb, tb64, ts, tw, p);
  }
}

template <int kFmt>
static cudaError_t launch_fmt(int BN, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& tb,
                              const CUtensorMap& tb64, const CUtensorMap& ts, const CUtensorMap& tw,
                              const GemmParams& p, bool glu, bool pair, bool native, bool wide) {
  if constexpr (kFmt == kFmtSparse)
    if (glu) return launch_bn<kFmt, true>(BN, grid, smem, stream, tb, tb64, ts, tw, p);
  if constexpr (kFmt == kFmtDense)
    if (native)
      return launch_pdl(grouped_gemm_kernel<kFmt, 128, false, 1, true>, grid, gemm_threads(kFmt, false), smem, stream, tb, tb64, ts,
                        tw, p);
  if constexpr (fmt_mx(kFmt))
    if (BN == 192)
      return launch_pdl_cluster(grouped_gemm_kernel<kFmt, 192, false, 2, false, true>, grid, gemm_threads(kFmt, true), smem,
                                stream, 2u, tb, tb64, ts, tw, p);
  if (BN == 128 && pair && wide)
    return launch_pdl_cluster(grouped_gemm_kernel<kFmt, 128, false, 2, false, true>, grid, gemm_threads(kFmt, true), smem,
                              stream, 2u, tb, tb64, ts, tw, p);
  if constexpr (!fmt_mx(kFmt)) {
    if (BN == 128 && pair)
      return launch_pdl_cluster(grouped_gemm_kernel<kFmt, 128, false, 2>, grid, gemm_threads(kFmt, false), smem, stream,
                                2u, tb, tb64, ts, tw, p);
    if (BN == 128)
      return launch_pdl(grouped_gemm_kernel<kFmt, 128, false, 1>, grid, gemm_threads(kFmt, false), smem, stream, tb, tb64,
                        ts, tw, p);
  }
  return launch_bn<kFmt, false>(BN, grid, smem, stream, tb, tb64, ts, tw, p);
}

// returns 0 ok, 1 cuda error, 2 tensor map failure.  h_scales / h_scale non-null: the SwiGLU
// epilogue (sparse only; Y receives the h codes).  comb non-null: the combine epilogue (Y is the
// slot buffer, bf16 output only).
int launch_gemm(int fmt, const uint8_t* a_codes, const uint8_t* a_scales, const float* x_scale,
                const uint8_t* w_packed, const float* w_scale, const int32_t* off, int E, int N, int K, int R,
                int max_rows, void* Y, int y_f32, int* status, int num_sms, cudaStream_t stream,
                uint8_t* h_scales, const float* h_scale, const CombineArgs* comb, bool native) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return 2;
  const bool glu = h_scales != nullptr;
  if (native && (fmt != kFmtDense || glu || comb != nullptr)) return 1;
  if ((glu || comb != nullptr) && fmt != kFmtSparse) return 1;
  const int mx_pairs = g_wide_units[fmt] < num_sms / 2 ? g_wide_units[fmt] : num_sms / 2;
  int BN = native        ? 128   // the native orientation: 128-token tiles (MMA M)
           : fmt_mx(fmt) ? mx_pick_bn(max_rows, R, E, N, K / fmt_chunk_k(fmt), fmt == kFmtMx8, num_sms, mx_pairs)
                         : gemm_pick_bn(max_rows, R, E);
  if (glu && BN > 64) BN = 64;   // two accumulators per tile: 64-token tiles at most
  // 128-token tiles run as CTA pairs (256 weight rows per tile) when N holds whole n-tile pairs
  // and the device can co-schedule pairs
  // a wide pair tile (no combine epilogue, N a multiple of 512; the microscaled formats: any N) holds two
  // n-tile pairs, 512 weight rows, and reads its tokens' activations once for both
  const bool wide = BN >= 128 && !glu && !native && comb == nullptr && (fmt_mx(fmt) || (N / kTileN) % 4 == 0) &&
                    g_wide_units[fmt] > 0;
  const int pair_units = wide ? g_wide_units[fmt] : g_pair_units[fmt];
  const bool pair = wide || (BN == 128 && !glu && !native && (N / kTileN) % 2 == 0 && pair_units > 0);
  const int cg = pair ? 2 : 1;
  const int units = pair ? (pair_units < num_sms / 2 ? pair_units : num_sms / 2) : num_sms;   // pairs or CTAs
  const int grid = units * cg;
  const int ntt = glu || (pair && wide) ? 2 : 1;   // weight n-tiles per tile and CTA
  const int NTt = ceil_div_i(N / kTileN, ntt * cg);
  const long long bound = (((long long)R + BN - 1) / BN + E) * NTt;
  // schedule: contiguous byte-balanced runs when every expert fits one token tile (max_rows known)
  // and the CTAs can hold at least 32 tiles each (at most min(E, R) experts are touched), else
  // round-robin
  const long long touched_max = R < E ? R : E;
  const int sched = (!pair && max_rows > 0 && max_rows <= BN && touched_max * NTt >= 32LL * units) ? kSchedRuns
                                                                                                  : kSchedRoundRobin;
  long long tcap;
  if (sched == kSchedRuns) {
    // a CTA's share of the bytes holds at most (wc + BN ac) / (wc + ac) times the average tile count
    const long long wc = (glu ? 2LL : 1LL) * kTileN * K * fmt_w_bytes32(fmt) / 32;
    const long long ac = fmt_act_row(fmt, K) + (glu ? 2LL : 1LL) * kTileN * (y_f32 ? 4 : 2);
    tcap = (bound * (wc + BN * ac) / (wc + ac) + units - 1) / units + 2;
  } else {
    tcap = (bound + units - 1) / units;
  }
  if (tcap > kMaxTableTiles) tcap = kMaxTableTiles;
  const int tcap_test = g_test_table_cap.load();
  if (tcap_test >= 0 && tcap > tcap_test) tcap = tcap_test;
  const GemmPlan g = make_plan(fmt, BN, E, (int)tcap, glu, cg, pair && wide);
  if (g.stages < kNSets || g.smem > (size_t)g_smem_limit) return 1;   // ring too shallow: refuse, launch nothing
  const int box_h = g.BN / cg < 32 ? g.BN / cg : 32;
  const int sfps = g.cps * fmt_sf_chunk(fmt);
  const int rcap = R + (fmt_mx(fmt) ? 0 : kActScalePadRows);   // (TMA boxes past the last row read zeros)
  const int KBa = K / fmt_chunk_k(fmt) * fmt_sf_chunk(fmt);
  const cuuint64_t row_bytes = (cuuint64_t)(K / fmt_chunk_k(fmt)) * 128;
  CUtensorMap tb, tb64, ts, tw;
  // activation codes [R][K/2] ([R][K] for 8-bit activations): boxes of 128 bytes x box_h rows, and (token tiles >= 64) x 64 rows
  for (int m = 0; m < 2; ++m) {
    if (m == 1 && g.BN / cg < 64) { tb64 = tb; break; }
    cuuint64_t dims[2] = {row_bytes, (cuuint64_t)R};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {128u, (cuuint32_t)(m == 0 ? box_h : 64)};
    cuuint32_t estr[2] = {1u, 1u};
    if (enc(m == 0 ? &tb : &tb64, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a_codes), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return 2;
  }
  {
    // activation scale quad entries as a [KBa][rcap * 2] tensor of 64-bit words (an entry is two; coordinates
    // stay within 31 bits for R <= 2^30); one box = the stage's atoms, 32 entries to a row
    cuuint64_t dims[2] = {(cuuint64_t)rcap * 2u, (cuuint64_t)KBa};
    cuuint64_t strides[1] = {(cuuint64_t)rcap * 16u};
    cuuint32_t box[2] = {64u, (cuuint32_t)sfps};
    cuuint32_t estr[2] = {1u, 1u};
    if (enc(&ts, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, const_cast<uint8_t*>(a_scales), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return 2;
  }
  if (fmt_mx(fmt)) {
    // microscaled weights as rows of 128 bytes (256 codes): a chunk block is 128 rows of codes and 8 of
    // scales (copied separately); one box = the codes of a block, or for 8-bit activations half of each
    // row, which the copy widens to 16 bytes per 16 codes
    const bool m8 = fmt == kFmtMx8;
    cuuint64_t dims[2] = {m8 ? 256u : 128u, (cuuint64_t)E * (N / kTileN) * (K / kChunkK) * kMxChunkRows};
    cuuint64_t strides[1] = {128u};
    cuuint32_t box[2] = {128u, 128u};
    cuuint32_t estr[2] = {1u, 1u};
    if (enc(&tw, m8 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<uint8_t*>(w_packed), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return 2;
  } else {
    tw = ts;   // not read
  }
  GemmParams p;
  p.a_scales = a_scales; p.x_scale = x_scale; p.w_packed = w_packed;
  p.w_scale = w_scale; p.off = off; p.Y = Y; p.status = status;
  p.E = E; p.N = N; p.K = K; p.R = R; p.y_f32 = y_f32; p.rcap = rcap;
  p.stages = g.stages; p.nacc = g.nacc; p.tcap = g.tcap; p.sched = sched;
  p.h_scales = h_scales; p.h_scale = h_scale;
  p.perm_src = comb ? comb->perm_src : nullptr;
  p.gates = comb ? comb->gates : nullptr;
  p.counters = comb ? comb->counters : nullptr;
  p.out = comb ? comb->out : nullptr;
  p.k = comb ? comb->k : 1;
  p.stall_ns = g_test_stall_ns.load();
  cudaError_t e = cudaErrorInvalidValue;
  switch (fmt) {
    case kFmtDense: e = launch_fmt<kFmtDense>(g.BN, grid, g.smem, stream, tb, tb64, ts, tw, p, glu, pair, native, wide); break;
    case kFmtSparse: e = launch_fmt<kFmtSparse>(g.BN, grid, g.smem, stream, tb, tb64, ts, tw, p, glu, pair, native, wide); break;
    case kFmtMx4: e = launch_fmt<kFmtMx4>(g.BN, grid, g.smem, stream, tb, tb64, ts, tw, p, glu, pair, native, wide); break;
    case kFmtMx8: e = launch_fmt<kFmtMx8>(g.BN, grid, g.smem, stream, tb, tb64, ts, tw, p, glu, pair, native, wide); break;
  }
  return e == cudaSuccess ? 0 : 1;
}

}  // namespace gsg
