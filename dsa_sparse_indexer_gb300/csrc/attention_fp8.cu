// Sparse MLA decode attention over an 8-bit cache with a scale for each block
// of slots (sm_103a).
//
// Per (shard s, row r, head h), over the valid slots j of the row's list:
// x_j = scale t_j (q . c_j), t_j the scale of the slot's block and c_j its 576
// e4m3 codes; O = sum_j 2^(x_j log2 e) t_j c_j[0..512) / sum_j 2^(x_j log2 e).
//
// The codes go to the tensor cores as they are stored (kind::f8f6f4); nothing
// is widened in shared memory.  What multiplies them is held in two 8-bit
// floats instead: the query (bf16, 8 significant bits) as e4m3 + e4m3 after a
// power of two per head that brings its largest value to [2^7, 2^8), exact but
// for values below 2^-10 of that one; a weight as e4m3 plus what that leaves as
// e5m2 (7 bits and more, down to 2^-17).  Two products with 8-bit operands cost
// what one with 16-bit ones does.  The scale of a token's block multiplies its
// scores, and its weight before that is split.
//
// A CTA takes 64 heads of one (row, shard), tiles of 128 tokens:
//  * S^T[token][head]: A = the tile (M = 128 tokens, K-major), B = the query
//    (N = 128: 64 heads' first parts, then their second parts), 18 MMAs of
//    K = 32.  The two halves of N are added by the softmax.  A score's thread
//    is its token's, so the token's scale is a register.
//  * O[head][dim]: A = the weights (M = 64 heads, MN-major: a thread stores its
//    token's weights side by side), B = the same tile as values (MN-major,
//    N = 256 dimensions), weight-stationary MMAs (tcgen05.mma.ws): 64 rows by
//    256 columns in 83 cycles, where M = 128 forms would take 128 for the same
//    heads (measured; shared-memory bandwidth: 2 + 8 KB an MMA).
// Tensor memory: O 256 columns, two score buffers of 128.  Shared memory: two
// stages of a tile (72 KB each), the query 72 KB, and 8 KB of weights; the
// other 8 KB of weights take the tile's rope block, which only the scores read.
//
//  warps 0-7   the query's two parts, then the softmax: a token and 32 heads a
//              thread, the running reference of a head moving only when a
//              tile's maximum is 2^5.75 above the last, and the outputs
//  warps 8-11  gather the selected rows, two warps a stage, 16-byte cp.async
//              into the swizzled layouts; a stage is filled and freed in two
//              parts (dimensions 0-255, the rest), as the value products that
//              read them end
//  warp 12     one thread issues the MMAs, whichever is ready first
// Every wait is bounded; one that runs out raises DSA_FLAG_TIMEOUT and stops
// the CTA's roles, which drain their copies and MMAs in flight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kDqk = DSA_MLA_DQK, kDv = DSA_MLA_DV;
constexpr int kTile = 128;                   // tokens of a tile: the scores' M
constexpr int kHeads = 64;                   // heads of a CTA
constexpr int kStages = 2;
constexpr int kBlocks = kDv / 128;           // latent blocks of 128 codes
constexpr int kKvBlock = kTile * 128;        // bytes of a tile's block
constexpr int kKvRope = kTile * 64;          // and of its rope block
constexpr int kQBlock = 2 * kHeads * 128;    // bytes of a query block, both parts
constexpr int kQRope = 2 * kHeads * 64;
constexpr int kSoftmaxWarps = 8, kGatherWarps = 4;
constexpr int kGather0 = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + kGatherWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
// Tensor-memory columns.
constexpr int kOCol = 0, kSCol = 256, kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
// A head's weights, with their token's scale, are t 2^(x - ref): a new reference
// puts the largest at 2^3, and they may grow to 2^8.75 (448 is the largest
// e4m3) before the next.
constexpr float kTop = 3.f, kGap = 8.75f;
// Scales for which neither the sums nor the weights leave fp32.
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p100f;

struct alignas(1024) Smem {
  uint8_t kv[kStages][kBlocks][kKvBlock];    // 131072
  uint8_t q[kBlocks][kQBlock];               // 65536
  uint8_t rope[kStages][kKvRope];            // 16384; then the weights' first parts
  uint8_t qrope[kQRope];                     // 8192
  uint8_t plo[kKvRope];                      // 8192: the weights' second parts
  float part[2][4][kHeads];                  // per 32 tokens: a tile's maxima, then the sums
  float ref[2][kHeads];                      // a tile's references
  float fq[kHeads];                          // scale log2(e) / the query's power of two; at the
                                             // end the outputs' factors
  uint64_t group[2], final, qfull, fullA[kStages], fullB[kStages], emptyA[kStages], emptyB[kStages];
  uint64_t sfull[2], sfree[2], pfull, pvdone, drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Smem) <= 232448, "shared memory of a CTA");

struct MlaFp8Args {
  const __nv_bfloat16* q;        // [rows][H][kDqk]
  const uint8_t* cache;          // [S][n_slots][kDqk]
  const float* scales;           // [S][n_blocks]
  const int32_t* slots;          // [S][rows][K]
  const int32_t* counts;         // [S][rows]
  int64_t n_slots, n_blocks;
  int rows, H, K, hgroups;
  float c2;                      // scale * log2(e)
  __nv_bfloat16* out;            // [S][rows][H][kDv]
  float* lse2;                   // [S][rows][H]
  uint32_t* flags;
  FastDiv fblock;
};

// Shared-memory matrix descriptor: start address >> 4 (bits 0-13), leading
// offset >> 4 (bits 16-29), stride >> 4 (bits 32-45), version 1 (bits 46-47),
// swizzle (bits 61-63: 2 = 128-byte, 4 = 64-byte).  K-major: the stride steps
// between 8-row groups.  MN-major: the stride steps between groups of 8 along
// K, the leading offset between swizzle atoms along M or N.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride,
                                              uint32_t swizzle) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((stride >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)swizzle << 61);
}

// Instruction descriptor of kind::f8f6f4: D fp32 (bits 4-5 = 1), A's type
// (bits 7-9) and B's (10-12) 0 = e4m3, 1 = e5m2, MN-major A (bit 15) and B
// (bit 16), N >> 3 (bits 17-22), M >> 4 (bits 24-28).
constexpr uint32_t idesc_f8(int m, int n, int a_type, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_type << 7) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ void mma_f8_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.ws.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive1(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ bool aborted(const Smem& sm) {
  return *reinterpret_cast<const volatile int*>(&sm.abort) != 0;
}

// Bounded wait that also gives up once another role of the CTA has aborted.
__device__ __forceinline__ bool wait_or_abort(Smem& sm, uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (aborted(sm)) return false;
    if (i > 64) __nanosleep(64);
  }
  return false;
}

__device__ __forceinline__ void abort_cta(Smem& sm, uint32_t* flags) {
  raise_flag(flags, DSA_FLAG_TIMEOUT);
  *reinterpret_cast<volatile int*>(&sm.abort) = 1;
}

// 32 columns of this warp's 32 tensor-memory lanes; tmem_wait names the
// registers so that no use of them is scheduled before it.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

// 2^x (ex2.approx.ftz.f32: relative error about 2^-22, 2^-inf = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest of the warp's values (a NaN loses to a number).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Two values as e4m3 codes, and as the half floats that those stand for.
__device__ __forceinline__ uint32_t to_e4m3x2(__half2 v) {
  return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t to_e5m2x2(__half2 v) {
  return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(v), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ __half2 of_e4m3x2(uint32_t c) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3));
}
__device__ __forceinline__ __half2 of_e5m2x2(uint32_t c) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E5M2));
}

// ---- gathering: the selected rows into the stages --------------------------
// Warps g and g + 2 serve stage g, rows 0-63 and 64-127 of each tile.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void landed(uint64_t* bar) {   // this lane's copies, for the MMAs
  proxy_fence();
  mbar_arrive1(bar);
}

__device__ __forceinline__ void gather_tiles(const MlaFp8Args& a, Smem& sm, int64_t shard_slots,
                                             int count, int ntiles, const int32_t* list) {
  const int lane = threadIdx.x & 31, g = (threadIdx.x >> 5) - kGather0;
  const int st = g & 1, row0 = (g >> 1) * 64;
  const uint8_t* cache = a.cache + shard_slots * kDqk;
  const uint32_t kv = smem_u32(sm.kv[st][0]), rope = smem_u32(sm.rope[st]);
  bool bad = false, ok = true;
  for (int t = st, k = 0; t < ntiles; t += kStages, ++k) {
    // Two tokens a lane; one left out, or past the list, becomes a zero row.
    int y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = t * kTile + row0 + 32 * i + lane;
      const int slot = j < count ? __ldg(list + j) : -1;
      const bool in = slot >= 0 && slot < a.n_slots;
      bad |= j < count && !in;
      y[i] = in ? slot : -1;
    }
    // The value products read whole groups of 32 tokens; a group past the list
    // is not read by any, and its scores are masked.
    const int groups = min(2, (count - t * kTile - row0 + 31) / 32);
    if (k >= 1) ok = wait_or_abort(sm, &sm.emptyA[st], (uint32_t)(k - 1) & 1u);
    if (!__all_sync(kFull, ok)) break;
    for (int i = 0; i < groups; ++i)
#pragma unroll 2
      for (int rq = 0; rq < 8; ++rq) {
        const int jr = 4 * rq + (lane >> 3), c = lane & 7;
        const int slot = __shfl_sync(kFull, i ? y[1] : y[0], jr);
        const uint8_t* src = cache + (int64_t)max(slot, 0) * kDqk + c * 16;
        const uint32_t dst = kv + (uint32_t)((row0 + 32 * i + jr) * 128 + ((c ^ (jr & 7)) << 4));
        copy16(dst, src, slot >= 0);
        copy16(dst + kKvBlock, src + 128, slot >= 0);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // Part B at once where its stage is free already, so that both are in
    // flight; else part A is handed over before the wait.
    const bool both = k == 0 || __all_sync(kFull, mbar_test(&sm.emptyB[st], (uint32_t)(k - 1) & 1u));
    if (!both) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      landed(&sm.fullA[st]);
      ok = wait_or_abort(sm, &sm.emptyB[st], (uint32_t)(k - 1) & 1u);
      if (!__all_sync(kFull, ok)) break;
    }
    for (int i = 0; i < groups; ++i) {
#pragma unroll 2
      for (int rq = 0; rq < 8; ++rq) {
        const int jr = 4 * rq + (lane >> 3), c = lane & 7;
        const int slot = __shfl_sync(kFull, i ? y[1] : y[0], jr);
        const uint8_t* src = cache + (int64_t)max(slot, 0) * kDqk + 256 + c * 16;
        const uint32_t dst =
            kv + 2 * kKvBlock + (uint32_t)((row0 + 32 * i + jr) * 128 + ((c ^ (jr & 7)) << 4));
        copy16(dst, src, slot >= 0);
        copy16(dst + kKvBlock, src + 128, slot >= 0);
      }
#pragma unroll 2
      for (int rq = 0; rq < 4; ++rq) {
        const int jr = 8 * rq + (lane >> 2), c = lane & 3;
        const int slot = __shfl_sync(kFull, i ? y[1] : y[0], jr);
        copy16(rope + (uint32_t)((row0 + 32 * i + jr) * 64 + ((c ^ ((jr >> 1) & 3)) << 4)),
               cache + (int64_t)max(slot, 0) * kDqk + kDv + c * 16, slot >= 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (both) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      landed(&sm.fullA[st]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    landed(&sm.fullB[st]);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");   // none outlives the CTA
  if (!__all_sync(kFull, ok) && lane == 0 && !aborted(sm)) abort_cta(sm, a.flags);
  if (bad) raise_flag(a.flags, DSA_FLAG_BOUNDS);
}

// ---- one thread: the MMAs ----------------------------------------------------
__device__ __forceinline__ void issue_mmas(const MlaFp8Args& a, Smem& sm, uint32_t tmem, int count,
                                           int ntiles) {
  constexpr uint32_t kIdS = idesc_f8(kTile, 2 * kHeads, 0, 0, 0);
  constexpr uint32_t kIdHi = idesc_f8(kHeads, 256, 0, 1, 1), kIdLo = idesc_f8(kHeads, 256, 1, 1, 1);
  bool ok = wait_or_abort(sm, &sm.qfull, 0);
  tc_fence_after();
  const uint64_t qd = smem_desc(smem_u32(sm.q[0]), 16, 1024, 2);
  const uint64_t qrd = smem_desc(smem_u32(sm.qrope), 16, 512, 4);
  const uint64_t lod = smem_desc(smem_u32(sm.plo), 16, 512, 4);
  int na = 0, nb = 0;                        // tiles whose score parts A and B are issued
  uint32_t idle = 0;
  for (int t = 0; ok && t < ntiles;) {
    const int st = t & 1;
    if (nb > t && mbar_test(&sm.pfull, (uint32_t)t & 1u)) {
      tc_fence_after();
      // Groups of 32 tokens that the tile has; the two halves of the
      // dimensions one after the other, so that the first one's blocks free
      // early.
      const int steps = min(kTile / 32, (count - t * kTile + 31) / 32);
      const uint64_t hid = smem_desc(smem_u32(sm.rope[st]), 16, 512, 4);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint64_t vd = smem_desc(smem_u32(sm.kv[st][2 * half]), kKvBlock, 1024, 2);
        const uint32_t d = tmem + kOCol + half * 128;
        for (int k = 0; k < steps; ++k) {
          const uint64_t v = vd + (uint64_t)(k * (4096 >> 4)), p = (uint64_t)(k * (2048 >> 4));
          mma_f8_ws(d, lod + p, v, kIdLo, (t > 0 || k > 0) ? 1u : 0u);
          mma_f8_ws(d, hid + p, v, kIdHi, 1u);
        }
        mma_commit(half == 0 ? &sm.emptyA[st] : &sm.emptyB[st]);
      }
      mma_commit(&sm.pvdone);
      ++t;
      idle = 0;
      continue;
    }
    const int sb = nb & 1;
    if (na > nb && mbar_test(&sm.fullB[sb], (uint32_t)(nb >> 1) & 1u)) {
      tc_fence_after();
      const uint32_t d = tmem + kSCol + sb * 128;
#pragma unroll
      for (int b = 2; b < kBlocks; ++b) {
        const uint64_t kd = smem_desc(smem_u32(sm.kv[sb][b]), 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(d, kd + k * 2, qd + (uint64_t)(b * (kQBlock >> 4) + k * 2), kIdS, 1u);
      }
      const uint64_t rd = smem_desc(smem_u32(sm.rope[sb]), 16, 512, 4);
#pragma unroll
      for (int k = 0; k < 2; ++k) mma_f8(d, rd + k * 2, qrd + k * 2, kIdS, 1u);
      mma_commit(&sm.sfull[sb]);
      ++nb;
      idle = 0;
      continue;
    }
    const int sa = na & 1;
    if (na == nb && na < ntiles && mbar_test(&sm.fullA[sa], (uint32_t)(na >> 1) & 1u) &&
        (na < 2 || mbar_test(&sm.sfree[sa], (uint32_t)((na >> 1) - 1) & 1u))) {
      tc_fence_after();
      const uint32_t d = tmem + kSCol + sa * 128;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint64_t kd = smem_desc(smem_u32(sm.kv[sa][b]), 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(d, kd + k * 2, qd + (uint64_t)(b * (kQBlock >> 4) + k * 2), kIdS,
                 (b > 0 || k > 0) ? 1u : 0u);
      }
      ++na;
      idle = 0;
      continue;
    }
    if (++idle >= 4 * kWaitPolls || aborted(sm)) {
      ok = false;
      break;
    }
    if (idle > 64) __nanosleep(32);
  }
  if (!ok && !aborted(sm)) abort_cta(sm, a.flags);
  mma_commit(&sm.drain);                     // every MMA issued ends before the memory is freed
  if (!mbar_wait(&sm.drain, 0)) abort_cta(sm, a.flags);
}

// ---- the query's two parts -----------------------------------------------------
// A warp takes eight heads; a head's 576 values are 72 chunks of 8, lanes
// 0-31 three times (the last for eight lanes).
__device__ __forceinline__ void split_query(const MlaFp8Args& a, Smem& sm, int r, int hg) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 2
  for (int i = 0; i < kHeads / kSoftmaxWarps; ++i) {
    const int h = warp * (kHeads / kSoftmaxWarps) + i, gh = hg * kHeads + h;
    const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)r * a.H + gh) * kDqk);
    uint4 v[3];
#pragma unroll
    for (int c = 0; c < 3; ++c)
      v[c] = gh < a.H && (c < 2 || lane < 8) ? __ldg(src + c * 32 + lane) : make_uint4(0, 0, 0, 0);
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) m = max(m, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
    }
    m = __reduce_max_sync(kFull, m);
    // 2^up brings the largest value to [2^7, 2^8).
    const int up = m ? min(7 - ((int)(m >> 7) - 127), 120) : 0;
    const float f = __uint_as_float((uint32_t)(up + 127) << 23);
    if (lane == 0)
      sm.fq[h] = m >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                              : a.c2 * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = make_float2(__uint_as_float(w[k] << 16) * f,
                                     __uint_as_float(w[k] & 0xFFFF0000u) * f);
        const __half2 xh = __float22half2_rn(x);
        hi[k] = to_e4m3x2(xh);
        lo[k] = to_e4m3x2(__hsub2(xh, of_e4m3x2(hi[k])));
      }
      const uint2 ph = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      const uint2 pl = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      const int d = (c * 32 + lane) * 8;     // first dimension of the chunk
      if (d < kDv) {
        uint8_t* blk = sm.q[d >> 7] + (d & 8);
        const int at = (((d & 127) >> 4) ^ (h & 7)) << 4;      // heads and 64 + heads alike
        *reinterpret_cast<uint2*>(blk + h * 128 + at) = ph;
        *reinterpret_cast<uint2*>(blk + (kHeads + h) * 128 + at) = pl;
      } else if (d < kDqk) {
        uint8_t* blk = sm.qrope + (d & 8);
        const int at = (((d & 63) >> 4) ^ ((h >> 1) & 3)) << 4;
        *reinterpret_cast<uint2*>(blk + h * 64 + at) = ph;
        *reinterpret_cast<uint2*>(blk + (kHeads + h) * 64 + at) = pl;
      }
    }
  }
  proxy_fence();
  __syncwarp();
  if (lane == 0) mbar_arrive1(&sm.qfull);
}

// Sums of 32 registers over the warp: lane h gets register h's.
__device__ __forceinline__ float transpose_sum(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < o) {
        const bool up = lane & o;
        const float mine = up ? v[i + o] : v[i], other = up ? v[i] : v[i + o];
        v[i] = mine + __shfl_xor_sync(kFull, other, o);
      }
  return v[0];
}

// ---- the softmax and the outputs ---------------------------------------------------
// Warp w reads the scores of tokens 32 (w % 4) .. + 31 (its tensor-memory
// lanes) for 32 of the 64 heads: half `hh`, chosen so that warps 0-3 handle the
// heads whose outputs lie in their lanes (head h with dimensions 0-127 of each
// 256 in lane h, with dimensions 128-255 in lane 64 + h).  The four warps of a
// half exchange their maxima and take the same decisions from them.
__device__ __forceinline__ void softmax_and_store(const MlaFp8Args& a, Smem& sm, uint32_t tmem,
                                                  int s, int count, int ntiles,
                                                  const int32_t* list, int64_t head0, int nheads) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3;
  const int hh = warp < 4 ? (quad & 1) : ((quad & 1) ^ 1);
  const int token = quad * 32 + lane, col = hh * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  const float* scales = a.scales + (int64_t)s * a.n_blocks;
  // The scale of this thread's token of tile t; `in` false for one left out.
  auto token_scale = [&](int t, bool* in) {
    const int j = t * kTile + token;
    const int slot = j < count ? __ldg(list + j) : -1;
    *in = slot >= 0 && slot < a.n_slots;
    return *in ? __ldg(scales + fdiv((uint32_t)slot, a.fblock)) : 0.f;
  };
  bool in_next, odd = false;
  float ts_next = token_scale(0, &in_next);
  float ref = -INFINITY;                     // of head `col`
  float l[32], gone[32];                     // weights; weights less their two parts
#pragma unroll
  for (int i = 0; i < 32; ++i) l[i] = gone[i] = 0.f;
  bool ok = wait_or_abort(sm, &sm.qfull, 0);   // fq is there
  for (int t = 0; __all_sync(kFull, ok) && t < ntiles; ++t) {
    const int sb = t & 1;
    const float ts = ts_next;
    const bool in = in_next;
    if (t + 1 < ntiles) ts_next = token_scale(t + 1, &in_next);
    odd |= in && !(ts == 0.f || (ts >= kMinScale && ts <= kMaxScale));
    const float rts = ts > 0.f ? __frcp_rn(ts) : 0.f;
    const float lt = ts > 0.f ? __log2f(ts) : 0.f;
    ok = wait_or_abort(sm, &sm.sfull[sb], (uint32_t)(t >> 1) & 1u);
    if (!__all_sync(kFull, ok)) break;
    tc_fence_after();
    float y[32];
    {
      uint32_t hi[32], lo[32];
      tmem_ld32(lanes + kSCol + sb * 128 + hh * 32, hi);
      tmem_ld32(lanes + kSCol + sb * 128 + kHeads + hh * 32, lo);
      tmem_wait(hi);
      tmem_wait(lo);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.sfree[sb]);
      const float4* fq = reinterpret_cast<const float4*>(sm.fq + hh * 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = fq[i];
        const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = (__uint_as_float(hi[4 * i + k]) + __uint_as_float(lo[4 * i + k])) * ts;
          y[4 * i + k] = in ? x * ff[k] : -INFINITY;
        }
      }
    }
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float m = warp_max(y[i] + lt);
      if (lane == i) mine = m;
    }
    sm.part[sb][quad][col] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.group[hh]);
    ok = wait_or_abort(sm, &sm.group[hh], (uint32_t)t & 1u);
    if (!__all_sync(kFull, ok)) break;
    const float mx = fmaxf(fmaxf(sm.part[sb][0][col], sm.part[sb][1][col]),
                           fmaxf(sm.part[sb][2][col], sm.part[sb][3][col]));
    const bool move = mx > ref + kGap || (ref == -INFINITY && mx > -INFINITY);
    const float now = move ? mx - kTop : ref;
    const float alpha = move && ref > -INFINITY ? fast_exp2(ref - now) : 1.f;
    const unsigned moved = __ballot_sync(kFull, alpha != 1.f);
    ref = now;
    sm.ref[sb][col] = now == -INFINITY ? 0.f : now;   // the half's four warps alike
    __syncwarp();
    if (moved) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float f = __shfl_sync(kFull, alpha, i);
        l[i] *= f;
        gone[i] *= f;
      }
    }
    uint32_t phi[8], plo[8];
    const float4* rf = reinterpret_cast<const float4*>(sm.ref[sb] + hh * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 r = rf[i];
      const float rr[4] = {r.x, r.y, r.z, r.w};
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = 4 * i + 2 * k;
        const float p0 = fast_exp2(y[e] - rr[2 * k]), p1 = fast_exp2(y[e + 1] - rr[2 * k + 1]);
        l[e] += p0;
        l[e + 1] += p1;
        const __half2 p = __floats2half2_rn(p0 * ts, p1 * ts);
        hi[k] = to_e4m3x2(p);
        const __half2 rest = __hsub2(p, of_e4m3x2(hi[k]));
        lo[k] = to_e5m2x2(rest);
        const float2 lost = __half22float2(__hsub2(rest, of_e5m2x2(lo[k])));
        gone[e] = fmaf(lost.x, rts, gone[e]);
        gone[e + 1] = fmaf(lost.y, rts, gone[e + 1]);
      }
      phi[i] = hi[0] | (hi[1] << 16);
      plo[i] = lo[0] | (lo[1] << 16);
    }
    // The last tile's value products are done: its weights' space is free and
    // O holds every earlier tile.
    if (t > 0) ok = wait_or_abort(sm, &sm.pvdone, (uint32_t)(t - 1) & 1u);
    if (!__all_sync(kFull, ok)) break;
    if (moved && warp < 4 && t > 0) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t o[32];
        tmem_ld32(lanes + kOCol + c, o);
        tmem_wait(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        tmem_st32(lanes + kOCol + c, o);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
    uint8_t* dh = sm.rope[sb] + token * 64;
    uint8_t* dl = sm.plo + token * 64;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int at = ((2 * hh + c) ^ ((token >> 1) & 3)) << 4;
      *reinterpret_cast<uint4*>(dh + at) =
          make_uint4(phi[4 * c], phi[4 * c + 1], phi[4 * c + 2], phi[4 * c + 3]);
      *reinterpret_cast<uint4*>(dl + at) =
          make_uint4(plo[4 * c], plo[4 * c + 1], plo[4 * c + 2], plo[4 * c + 3]);
    }
    proxy_fence();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.pfull);
  }
  if (odd) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  // The sums over all tokens: 32 lanes, then the half's four warps.
  auto half_sum = [&](float mine, int phase) {
    sm.part[phase & 1][quad][col] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.group[hh]);
    ok = wait_or_abort(sm, &sm.group[hh], (uint32_t)phase & 1u);
    const float(*p)[kHeads] = sm.part[phase & 1];
    return (p[0][col] + p[1][col]) + (p[2][col] + p[3][col]);
  };
  if (__all_sync(kFull, ok)) {
    const float sum = half_sum(transpose_sum(l), ntiles);
    const float less = __all_sync(kFull, ok) ? half_sum(transpose_sum(gone), ntiles + 1) : 0.f;
    if (warp < 2) {                          // warp = hh
      sm.fq[col] = sum == 0.f ? 0.f : 1.f / (sum - less);
      if (__all_sync(kFull, ok) && col < nheads)
        a.lse2[head0 + col] = sum == 0.f ? -INFINITY : ref + log2f(sum);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.final);
    ok = __all_sync(kFull, ok) && wait_or_abort(sm, &sm.final, 0) &&
         wait_or_abort(sm, &sm.pvdone, (uint32_t)(ntiles - 1) & 1u);
  }
  if (!__all_sync(kFull, ok)) {
    if (lane == 0 && !aborted(sm)) abort_cta(sm, a.flags);
    return;
  }
  tc_fence_after();
  const int h = (quad & 1) * 32 + lane, group = warp >> 2;
  const float inv = sm.fq[h];
  __nv_bfloat16* orow = a.out + (head0 + h) * kDv + group * 256 + (quad >> 1) * 128;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    uint32_t o[32];
    tmem_ld32(lanes + kOCol + group * 128 + c, o);
    tmem_wait(o);
    if (h < nheads) {
      uint4* dst = reinterpret_cast<uint4*>(orow + c);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x =
              __floats2bfloat162_rn(__uint_as_float(o[8 * v + 2 * i]) * inv,
                                    __uint_as_float(o[8 * v + 2 * i + 1]) * inv);
          b[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        dst[v] = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) sparse_mla_decode_fp8_kernel(const MlaFp8Args a) {
  extern __shared__ __align__(1024) unsigned char mla_fp8_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(mla_fp8_smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int hg = blockIdx.x % a.hgroups, pair = blockIdx.x / a.hgroups;
  const int s = pair / a.rows, r = pair - s * a.rows;
  int count = __ldg(a.counts + pair);
  if ((count < 0 || count > a.K) && tid == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  count = min(max(count, 0), a.K);
  const int ntiles = (count + kTile - 1) / kTile;
  const int64_t head0 = (int64_t)pair * a.H + hg * kHeads;   // first head of the group
  const int nheads = min(kHeads, a.H - hg * kHeads);
  const int32_t* list = a.slots + (int64_t)pair * a.K;

  if (count == 0) {
    // Nothing selected on this shard: O = 0, lse2 = -inf.
    for (int i = tid; i < nheads * (kDv / 8); i += kThreads)
      reinterpret_cast<uint4*>(a.out + head0 * kDv)[i] = make_uint4(0, 0, 0, 0);
    if (tid < nheads) a.lse2[head0 + tid] = -INFINITY;
    return;
  }

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.group[i], 4);
      mbar_init(&sm.fullA[i], 64);           // every lane of the stage's two gathering warps
      mbar_init(&sm.fullB[i], 64);
      mbar_init(&sm.emptyA[i], 1);
      mbar_init(&sm.emptyB[i], 1);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sfree[i], kSoftmaxWarps);
    }
    mbar_init(&sm.qfull, kSoftmaxWarps);
    mbar_init(&sm.pfull, kSoftmaxWarps);
    mbar_init(&sm.final, kSoftmaxWarps);
    mbar_init(&sm.pvdone, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < kSoftmaxWarps) {
    split_query(a, sm, r, hg);
    softmax_and_store(a, sm, tmem, s, count, ntiles, list, head0, nheads);
  } else if (warp < kMmaWarp) {
    gather_tiles(a, sm, (int64_t)s * a.n_slots, count, ntiles, list);
  } else {
    if ((tid & 31) == 0) issue_mmas(a, sm, tmem, count, ntiles);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_sparse_mla_decode_fp8(const uint16_t* q, const uint8_t* kv_cache,
                                                const float* block_scales, int64_t n_slots,
                                                int block_tokens, const int32_t* slots,
                                                const int32_t* counts, int rows, int S, int H,
                                                int K, float scale, uint16_t* out, float* lse2,
                                                uint32_t* err_flags, cudaStream_t stream) {
  if (rows < 0 || K < 1 || H < 1 || n_slots < 1 || block_tokens < 1 || n_slots % block_tokens ||
      !std::isfinite(scale))
    return DSA_ERR_INVALID_ARG;
  if (S < 1 || S > DSA_MAX_SHARDS || n_slots > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (rows == 0) return DSA_OK;
  if (!q || !kv_cache || !block_scales || !slots || !counts || !out || !lse2)
    return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  const int hgroups = (H + kHeads - 1) / kHeads;
  const int64_t blocks = (int64_t)rows * S * hgroups;
  if (blocks > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  const int smem = (int)sizeof(Smem);
  if (cudaFuncSetAttribute(sparse_mla_decode_fp8_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const MlaFp8Args a{reinterpret_cast<const __nv_bfloat16*>(q),
                     kv_cache,
                     block_scales,
                     slots,
                     counts,
                     n_slots,
                     n_slots / block_tokens,
                     rows,
                     H,
                     K,
                     hgroups,
                     scale * kLog2e,
                     reinterpret_cast<__nv_bfloat16*>(out),
                     lse2,
                     err_flags,
                     FastDiv((uint32_t)block_tokens)};
  const cudaError_t e = launch_kernel(sparse_mla_decode_fp8_kernel, dim3((unsigned)blocks),
                                      dim3(kThreads), (size_t)smem, stream, 0u, a);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
