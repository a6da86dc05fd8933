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
// for values below 2^-9 of that one; a weight, times its token's scale, as e4m3
// plus what that leaves as e5m2 (to 2^-7; below 2^-9 of the largest to 2^-16 of
// that one).  Two products with 8-bit operands cost what one with 16-bit ones
// does.  The scale of a token's block multiplies its scores, and its weight
// before that is split.
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
//  warps 0-15  the softmax: a token and 16 heads a thread, the running
//              reference of a head moving only when a weight would pass its
//              bound; the outputs (with few heads warps 8-15 write them); and a
//              row's query in its two parts, the next one's while this one's last
//              value products run
//  warps 16-19 gather the selected rows, 32 of each tile a warp, 16-byte
//              cp.async into the swizzled layouts; a stage is filled and freed
//              in two parts (dimensions 0-255, the rest), as the value products
//              that read them end
//  warps 20-21 a thread each issues the scores and the value products
// The kernel is persistent: one CTA an SM, each with a run of (row, shard)
// pairs in row order, so that a row's shards share the query on chip and a
// pair's start and end overlap its neighbours' tiles.  Few pairs are split over
// clusters of CTAs.
// Measured, 128 heads: 512 rows of 2048 tokens in 325 us (0.90 PFLOP/s of 16-bit
// work, 0.48 of a measured bf16 GEMM), 275 with one scale for all blocks, where
// fewer references move after a list's first tile; 64 rows, 4 shards of 400 to
// 640 tokens 75 (69); 16 heads, 128 rows, 8 shards of 200 to 312 tokens 53 (52); a
// row of 2048 tokens 19.2 (18.0).  Bound by the chain gather, scores, softmax,
// values over two stages, about 4030 cycles a tile where the MMAs take 2840 and no
// reference moves, and by a pair's end: 6 thousand cycles, 13 when a new row's
// query has to be split.
// Every wait is bounded; one that runs out raises DSA_FLAG_TIMEOUT and stops
// the CTA's roles, which drain their copies and MMAs in flight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
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
constexpr int kSoftmaxWarps = 16, kGatherWarps = 4;
constexpr int kGroups = kSoftmaxWarps / 4;   // of four warps, 16 heads each
constexpr int kGroupHeads = kHeads / kGroups;
constexpr int kGather0 = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + kGatherWarps;
constexpr int kThreads = 768;                // six warpgroups; warps 22-23 only make up the last
// Registers a thread of the softmax's four warpgroups, the gathering one and
// the MMA's: 128 (4 x 96 + 48 + 48) = the 768 x 80 the CTA is launched with.  A
// few registers spilled in any role's loop cost 3 to 6 %, so the roles' loops are
// kept within these.
constexpr int kRegsSoftmax = 96, kRegsGather = 48, kRegsMma = 48;
// With few heads: two warpgroups of the softmax, two that write outputs.
constexpr int kWriter0 = 8, kRegsFew = 120, kRegsWriter = 72;
static_assert(128 * (2 * kRegsFew + 2 * kRegsWriter + kRegsGather + kRegsMma) <= kThreads * 80, "registers");
static_assert(128 * (4 * kRegsSoftmax + kRegsGather + kRegsMma) <= kThreads * 80, "registers");
// Tensor-memory columns.
constexpr int kOCol = 0, kSCol = 256, kTmemCols = 512;
constexpr int kCounts = 20;                  // pairs whose counts are kept on chip
constexpr int kSms = 152;                     // of a GB300
constexpr int kMaxList = 1 << 30;            // tokens of a list
constexpr float kLog2e = 1.4426950408889634f;
// A head's weights, with their token's scale, are t 2^(x - ref): a new reference
// puts the largest at 2^3, and they may grow to 2^8.75 (448 is the largest
// e4m3) before the next.
constexpr float kTop = 3.f, kGap = 8.75f;
#ifdef DSA_TEST_STALLED_COPY
// The test-only build (never libdsa.so): part A of every stage expects one
// arrival that nothing makes, so the scores' wait runs out (every copy still
// lands) and the kernel returns with DSA_FLAG_TIMEOUT.
constexpr uint32_t kStalledArrivals = 1;
#else
constexpr uint32_t kStalledArrivals = 0;
#endif
// Scales for which neither the sums nor the weights leave fp32: a weight is at
// most 2^kGap over the scale, so a list's sum holds 2^18 tokens of the least.
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p100f, kLog2MinScale = -100.f;

struct alignas(1024) Smem {
  uint8_t kv[kStages][kBlocks][kKvBlock];    // 131072
  uint8_t q[kBlocks][kQBlock];               // 65536
  uint8_t rope[kStages][kKvRope];            // 16384; then the weights' first parts
  uint8_t qrope[kQRope];                     // 8192
  uint8_t plo[kKvRope];                      // 8192: the weights' second parts
  float part[4][kHeads];                     // per 32 tokens: a tile's maxima
  float ref[2][kHeads];                      // a tile's references
  float fq[kHeads];                          // scale log2(e) / the query's power of two
  float tok[kStages][kTile];                 // the tokens' scales; -1: left out
  int counts[kCounts];                       // of the CTA's first pairs
  int first;                                 // the CTA's first token of its pair (split pairs)
  uint64_t qfull, fullA[kStages], fullB[kStages], emptyA[kStages], emptyB[kStages];
  uint64_t sfull[2], sfree[2], pfull, pvdone, ofree, drain[2];
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
  int rows, S, H, K, hgroups;
  float c2;                      // scale * log2(e)
  __nv_bfloat16* out;            // [S][rows][H][kDv]
  float* lse2;                   // [S][rows][H]
  float* work;                   // a slot for every CTA of split pairs
  uint32_t* flags;
  FastDiv fblock, fS;
};

// Pair p = row * S + shard.
__device__ __forceinline__ int row_of(const MlaFp8Args& a, int p) { return (int)fdiv((uint32_t)p, a.fS); }
__device__ __forceinline__ int64_t list_of(const MlaFp8Args& a, int p, int* shard) {
  uint32_t s;
  const int row = (int)fdivmod((uint32_t)p, a.fS, &s);
  *shard = (int)s;
  return (int64_t)s * a.rows + row;          // index of the pair's list, count and outputs
}

// Steps over the tiles of the CTA's pairs [p0, p1), those with no token left out.
struct Cursor {
  int p, t, count;
  __device__ __forceinline__ bool valid(int p1) const { return p < p1; }
  // The first pair with tokens from p on.
  __device__ __forceinline__ void settle(const MlaFp8Args& a, const Smem& sm, int p0, int p1) {
    for (t = 0, count = 0; p < p1; ++p) {
      int s;
      count = p - p0 < kCounts ? sm.counts[p - p0]
                               : min(max(__ldg(a.counts + list_of(a, p, &s)), 0), a.K);
      if (count > 0) break;
    }
  }
  __device__ __forceinline__ Cursor(const MlaFp8Args& a, const Smem& sm, int p0, int p1) : p(p0) {
    settle(a, sm, p0, p1);
  }
  __device__ __forceinline__ void next_pair(const MlaFp8Args& a, const Smem& sm, int p0, int p1) {
    ++p;
    settle(a, sm, p0, p1);
  }
  __device__ __forceinline__ void advance(const MlaFp8Args& a, const Smem& sm, int p0, int p1) {
    if (++t * kTile >= count) next_pair(a, sm, p0, p1);
  }
};

// Shared-memory matrix descriptor: start address >> 4 (bits 0-13), leading
// offset >> 4 (bits 16-29), stride >> 4 (bits 32-45), version 1 (bits 46-47),
// swizzle (bits 61-63: 2 = 128-byte, 4 = 64-byte).  K-major: the stride steps
// between 8-row groups.  MN-major: the stride steps between groups of 8 along
// K, the leading offset between swizzle atoms along M or N.
// In two words: the upper ones are constants.
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | (((lead >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t smem_desc_up(uint32_t stride, uint32_t swizzle) {
  return ((stride >> 4) & 0x3FFFu) | (1u << 14) | (swizzle << 29);
}

// Instruction descriptor of kind::f8f6f4: D fp32 (bits 4-5 = 1), A's type
// (bits 7-9) and B's (10-12) 0 = e4m3, 1 = e5m2, MN-major A (bit 15) and B
// (bit 16), N >> 3 (bits 17-22), M >> 4 (bits 24-28).
constexpr uint32_t idesc_f8(int m, int n, int a_type, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_type << 7) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <uint32_t kA, uint32_t kB, uint32_t kIdesc>
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %6, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(accum), "n"(kA), "n"(kB), "r"(kIdesc)
      : "memory");
}

template <uint32_t kA, uint32_t kB, uint32_t kIdesc>
__device__ __forceinline__ void mma_f8_ws(uint32_t d, uint32_t a, uint32_t b, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.ws.cta_group::1.kind::f8f6f4 [%0], x, y, %6, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(accum), "n"(kA), "n"(kB), "r"(kIdesc)
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
// Named hardware barriers of the softmax's warps, which run the same sequence
// of them whatever happens: a failed wait does not end their loops, so that no
// warp is left behind.
__device__ __forceinline__ bool barrier_or(int id, int threads, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"((uint32_t)mine)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void barrier(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void barrier_arrive(int id, int threads) {
  asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- clusters: a pair split over several CTAs ------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster's CTAs that has not exited.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ bool aborted(const Smem& sm) {
  return *reinterpret_cast<const volatile int*>(&sm.abort) != 0;
}

// Bounded wait that also gives up once another role of the CTA has aborted.  A
// try may suspend the thread for up to kSuspendNs.
constexpr uint32_t kSuspendNs = 1000;
__device__ __forceinline__ bool wait_or_abort(Smem& sm, uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (done) return true;
    if (aborted(sm)) return false;
  }
  return false;
}

__device__ __forceinline__ void abort_cta(Smem& sm, uint32_t* flags) {
  raise_flag(flags, DSA_FLAG_TIMEOUT);
  *reinterpret_cast<volatile int*>(&sm.abort) = 1;
}

// 16 columns of this warp's 32 tensor-memory lanes; or 32 columns of 16 lanes,
// a thread then holding of each 8 columns two of lane (id / 4) and two
// of lane 8 + id / 4.  tmem_wait names the registers so that no use of them is
// scheduled before it.
#define DSA_R16(o)                                                                             \
  "+r"(r[o + 0]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]),              \
      "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7]), "+r"(r[o + 8]), "+r"(r[o + 9]),          \
      "+r"(r[o + 10]), "+r"(r[o + 11]), "+r"(r[o + 12]), "+r"(r[o + 13]), "+r"(r[o + 14]),     \
      "+r"(r[o + 15])
#define DSA_W16(o)                                                                             \
  "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]),              \
      "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]),          \
      "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]), "=r"(r[o + 13]), "=r"(r[o + 14]),     \
      "=r"(r[o + 15])
#define DSA_L16 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {" DSA_L16 "}, [%16];"
               : DSA_W16(0)
               : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32_of16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {" DSA_L16 "}, [%16];"
               : DSA_W16(0)
               : "r"(addr));
}
__device__ __forceinline__ void tmem_st32_of16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {" DSA_L16 "};"
               : DSA_R16(0)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : DSA_R16(0));
}
#undef DSA_R16
#undef DSA_W16
#undef DSA_L16

// 2^x (ex2.approx.ftz.f32: relative error about 2^-22, 2^-inf = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two products, sums or fused multiply-adds in one instruction, each rounded as
// the scalar operation would be.
#define DSA_F32X2(name, op)                                                              \
  __device__ __forceinline__ float2 name(float2 a, float2 b) {                           \
    uint64_t r;                                                                          \
    asm(op " %0, %1, %2;"                                                                \
        : "=l"(r)                                                                        \
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b))); \
    return *reinterpret_cast<float2*>(&r);                                               \
  }
DSA_F32X2(fmul2, "mul.rn.f32x2")
DSA_F32X2(fadd2, "add.rn.f32x2")
#undef DSA_F32X2
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
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
// Warp g takes rows 32 g .. + 31 of every tile.  Eight lanes copy a row's
// 128-byte segment of a block, so lane l serves rows l / 8 + 4 i, and keeps
// their offsets in registers: the copies of a part are issued back to back.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
// An arrival once this lane's copies so far have landed; the thread that then
// issues MMAs on them fences them to the async proxy.
__device__ __forceinline__ void arrive_landed(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void gather_tiles(const MlaFp8Args& a, Smem& sm, int p0, int p1) {
  const int lane = threadIdx.x & 31, row0 = ((threadIdx.x >> 5) - kGather0) * 32;
  const int sub = lane >> 3, c = lane & 7;
  // A row's chunk c lies at c ^ (row & 7): rows 4 i + sub alternate between
  // two places.  The rope block's rows have four chunks, at c ^ (row / 2 & 3);
  // lanes 0-3 of eight copy row 4 i + sub, lanes 4-7 the same plus 16.
  const uint32_t kv0 = smem_u32(sm.kv[0][0]) + (uint32_t)(row0 + sub) * 128;
  const uint32_t even = (uint32_t)(c ^ sub) << 4, odd = (uint32_t)(c ^ (sub + 4)) << 4;
  const uint32_t rope0 = smem_u32(sm.rope[0]) + (uint32_t)(row0 + sub + (c >> 2) * 16) * 64;
  bool bad = false, ok = true;
  Cursor cur(a, sm, p0, p1);
  const int32_t* slots = a.slots + sm.first;
  int shard = 0;
  int32_t mine = -1;                         // the slot of row0 + lane, the next tile's
  auto fetch_mine = [&]() {
    const int32_t* list = slots + list_of(a, cur.p, &shard) * a.K;   // every lane's shard
    const int j = cur.t * kTile + row0 + lane;
    mine = j < cur.count ? __ldg(list + j) : -1;
  };
  if (cur.valid(p1)) fetch_mine();
  // A part may be filled once the value products of its last tile are done.
  auto room = [&](uint64_t* empty, int k) {
    if (k >= 1) ok = wait_or_abort(sm, empty, (uint32_t)(k - 1) & 1u);
    return __all_sync(kFull, ok) != 0;
  };
  for (int n = 0; cur.valid(p1); ++n) {
    const int st = n & 1, k = n >> 1, left = cur.count - cur.t * kTile - row0;
    const uint8_t* cache = a.cache + (int64_t)shard * a.n_slots * kDqk + c * 16;
    // One left out, or past the list, becomes a zero row.  The value products
    // read whole groups of 32 tokens; a group past the list is not read by any,
    // and its scores are masked: it is not filled.
    int32_t y[8];
    const bool in = mine >= 0 && mine < a.n_slots;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(kFull, in ? mine : -1, 4 * i + sub);
    // The scale of row0 + lane's token, for the softmax.
    bad |= !in && lane < left;
    float ts = -1.f;
    if (in) ts = __ldg(a.scales + shard * a.n_blocks + fdiv((uint32_t)mine, a.fblock));
    cur.advance(a, sm, p0, p1);
    if (cur.valid(p1)) fetch_mine();
    const uint32_t kv = kv0 + (uint32_t)st * (kBlocks * kKvBlock);
    auto copy_pair = [&](int block) {        // blocks `block` and block + 1
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint8_t* src = cache + (int64_t)max(y[i], 0) * kDqk + block * 128;
        const uint32_t dst = kv + block * kKvBlock + i * 512 + ((i & 1) ? odd : even);
        copy16(dst, src, y[i] >= 0);
        copy16(dst + kKvBlock, src + 128, y[i] >= 0);
      }
    };
    if (!room(&sm.emptyA[st], k)) break;
    if (left > 0) copy_pair(0);
    arrive_landed(&sm.fullA[st]);
    if (!room(&sm.emptyB[st], k)) break;
    bad |= in && !(ts == 0.f || (ts >= kMinScale && ts <= kMaxScale));
    sm.tok[st][row0 + lane] = !in ? -1.f : ts > 0.f ? ts : 0.f;
    if (left > 0) {
      copy_pair(2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t row = c < 4 ? y[i] : y[i + 4];
        copy16(rope0 + (uint32_t)st * kKvRope + i * 256 + (((c & 3) ^ ((2 * i + (sub >> 1)) & 3)) << 4),
               cache + (int64_t)max(row, 0) * kDqk + kDv - (c & 4) * 16, row >= 0);
      }
    }
    arrive_landed(&sm.fullB[st]);
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.fullB[st]);   // the scales
  }
  asm volatile("cp.async.wait_all;" ::: "memory");   // none outlives the CTA
  if (!__all_sync(kFull, ok) && lane == 0 && !aborted(sm)) abort_cta(sm, a.flags);
  if (bad) raise_flag(a.flags, DSA_FLAG_BOUNDS);
}

// ---- the MMAs: a thread for the scores, a thread for the value products ------
// Scores run up to two tiles ahead of the value products, across pairs; a new
// row's wait for its query.
__device__ __forceinline__ bool issue_scores(const MlaFp8Args& a, Smem& sm, uint32_t tmem, int p0,
                                             int p1) {
  constexpr uint32_t kId = idesc_f8(kTile, 2 * kHeads, 0, 0, 0);
  constexpr uint32_t k128 = smem_desc_up(1024, 2), k64 = smem_desc_up(512, 4);
  const uint32_t qd = smem_desc(smem_u32(sm.q[0]), 16), qrd = smem_desc(smem_u32(sm.qrope), 16);
  auto block = [&](uint32_t d, int st, int b) {
    const uint32_t kd = smem_desc(smem_u32(sm.kv[st][b]), 16);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_f8<k128, k128, kId>(d, kd + k * 2, qd + (uint32_t)(b * (kQBlock >> 4) + k * 2),
                              b + k > 0 ? 1u : 0u);
  };
  Cursor cur(a, sm, p0, p1);
  int row = -1, run = -1;                    // the row at hand; rows begun
  for (int n = 0; cur.valid(p1); ++n) {
    const int st = n & 1;
    const uint32_t parity = (uint32_t)(n >> 1) & 1u, d = tmem + kSCol + st * 128;
    if (row_of(a, cur.p) != row) {
      row = row_of(a, cur.p);
      if (!wait_or_abort(sm, &sm.qfull, (uint32_t)++run & 1u)) return false;
    }
    if ((n >= 2 && !wait_or_abort(sm, &sm.sfree[st], parity ^ 1u)) ||
        !wait_or_abort(sm, &sm.fullA[st], parity))
      return false;
    proxy_fence();
    tc_fence_after();
    block(d, st, 0);
    block(d, st, 1);
    if (!wait_or_abort(sm, &sm.fullB[st], parity)) return false;
    proxy_fence();
    tc_fence_after();
    block(d, st, 2);
    block(d, st, 3);
    const uint32_t rd = smem_desc(smem_u32(sm.rope[st]), 16);
#pragma unroll
    for (int k = 0; k < 2; ++k) mma_f8<k64, k64, kId>(d, rd + k * 2, qrd + k * 2, 1u);
    mma_commit(&sm.sfull[st]);
    cur.advance(a, sm, p0, p1);
  }
  return true;
}

__device__ __forceinline__ bool issue_values(const MlaFp8Args& a, Smem& sm, uint32_t tmem, int p0,
                                             int p1, bool handed) {
  constexpr uint32_t kIdHi = idesc_f8(kHeads, 256, 0, 1, 1), kIdLo = idesc_f8(kHeads, 256, 1, 1, 1);
  constexpr uint32_t kP = smem_desc_up(512, 4), kV = smem_desc_up(1024, 2);
  const uint32_t lod = smem_desc(smem_u32(sm.plo), 16);
  Cursor cur(a, sm, p0, p1);
  int pair = -1;                             // pairs begun, less one
  for (int n = 0; cur.valid(p1); ++n) {
    // Groups of 32 tokens that the tile has; the two halves of the dimensions
    // one after the other, so that the first one's blocks free early.
    const int st = n & 1, steps = min(kTile / 32, (cur.count - cur.t * kTile + 31) / 32);
    const uint32_t hid = smem_desc(smem_u32(sm.rope[st]), 16);
    if (!wait_or_abort(sm, &sm.pfull, (uint32_t)n & 1u)) return false;
    // Where others write a pair's outputs, they have read the last pair's O.
    if (handed && cur.t == 0 && ++pair > 0 &&
        !wait_or_abort(sm, &sm.ofree, (uint32_t)(pair - 1) & 1u))
      return false;
    tc_fence_after();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t vd = smem_desc(smem_u32(sm.kv[st][2 * half]), kKvBlock);
      const uint32_t d = tmem + kOCol + half * 128;
      for (int k = 0; k < steps; ++k) {
        const uint32_t v = vd + (uint32_t)(k * (4096 >> 4)), p = (uint32_t)(k * (2048 >> 4));
        mma_f8_ws<kP, kV, kIdLo>(d, lod + p, v, (cur.t > 0 || k > 0) ? 1u : 0u);
        mma_f8_ws<kP, kV, kIdHi>(d, hid + p, v, 1u);
      }
      mma_commit(half == 0 ? &sm.emptyA[st] : &sm.emptyB[st]);
    }
    mma_commit(&sm.pvdone);
    cur.advance(a, sm, p0, p1);
  }
  return true;
}

// Every MMA issued ends before the tensor memory is freed.
__device__ __forceinline__ void drain_mmas(const MlaFp8Args& a, Smem& sm, uint64_t* bar, bool ok) {
  if (!ok && !aborted(sm)) abort_cta(sm, a.flags);
  mma_commit(bar);
  if (!mbar_wait(bar, 0)) abort_cta(sm, a.flags);
}

// ---- the query's two parts -----------------------------------------------------
// Warp w takes heads 4 w .. + 3.  A head's 512 latent values are 64 chunks of 8,
// two a lane; the four rope parts, 32 chunks, one a lane.  Returns the factor of
// head 4 w + lane (lanes 0-3).
__device__ __forceinline__ void split_chunk(const uint4& v, float f, uint8_t* hi_at, uint8_t* lo_at) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = fmul2(make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)),
                           make_float2(f, f));
    const __half2 x = __floats2half2_rn(y.x, y.y);
    hi[k] = to_e4m3x2(x);
    lo[k] = to_e4m3x2(__hsub2(x, of_e4m3x2(hi[k])));
  }
  *reinterpret_cast<uint2*>(hi_at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
  *reinterpret_cast<uint2*>(lo_at) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
}
__device__ __forceinline__ uint32_t chunk_amax(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;                            // two at a time: bits order magnitudes
#pragma unroll
  for (int k = 0; k < 4; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}
// 2^up brings a head's largest value (bf16 bits m) to [2^7, 2^8).
__device__ __forceinline__ int query_up(uint32_t m) {
  return m ? min(7 - ((int)(m >> 7) - 127), 120) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float split_query(const MlaFp8Args& a, Smem& sm, int r, int hg) {
  constexpr int kEach = kHeads / kSoftmaxWarps;
  const int lane = threadIdx.x & 31, h0 = (threadIdx.x >> 5) * kEach, gh0 = hg * kHeads + h0;
  const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)r * a.H + gh0) * kDqk);
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 v[kEach][2];
  const int ri = lane >> 3;                  // this lane's rope chunk: its head, and place
  const uint4 rope = gh0 + ri < a.H ? __ldcs(src + ri * (kDqk / 8) + kDv / 8 + (lane & 7)) : none;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      v[i][c] = gh0 + i < a.H ? __ldcs(src + i * (kDqk / 8) + c * 32 + lane) : none;
  uint32_t mr = chunk_amax(rope);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mr = max(mr, __shfl_xor_sync(kFull, mr, o));
  int rope_up = 0;
  float factor = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int h = h0 + i;
    const uint32_t m = max(__reduce_max_sync(kFull, max(chunk_amax(v[i][0]), chunk_amax(v[i][1]))),
                           __shfl_sync(kFull, mr, 8 * i));
    const int up = query_up(m);
    if (ri == i) rope_up = up;
    if (lane == i) factor = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : a.c2 * pow2(-up);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // Heads h and 64 + h (the second parts) share a swizzle phase.
      const int chunk = c * 32 + lane;       // of 8 values; two make 16 codes
      uint8_t* at = sm.q[chunk >> 4] + h * 128 + ((((chunk >> 1) & 7) ^ (h & 7)) << 4) + (chunk & 1) * 8;
      split_chunk(v[i][c], pow2(up), at, at + kHeads * 128);
    }
  }
  const int h = h0 + ri;
  uint8_t* at = sm.qrope + h * 64 + ((((lane & 7) >> 1) ^ ((h >> 1) & 3)) << 4) + (lane & 1) * 8;
  split_chunk(rope, pow2(rope_up), at, at + kHeads * 64);
  proxy_fence();
  __syncwarp();
  if (lane == 0) mbar_arrive1(&sm.qfull);
  return factor;
}

// 16 values of every lane joined over the warp, by halves: lanes i and 16 + i get
// value i's.  16 shuffles, where one value after another takes 80.
template <typename Join>
__device__ __forceinline__ float transpose_join(const float2 (&v2)[8], Join join) {
  const int lane = threadIdx.x & 31;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = i & 1 ? v2[i / 2].y : v2[i / 2].x;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < o) {
        const bool up = lane & o;
        const float mine = up ? v[i + o] : v[i], other = up ? v[i] : v[i + o];
        v[i] = join(mine, __shfl_xor_sync(kFull, other, o));
      }
  return join(v[0], __shfl_xor_sync(kFull, v[0], 16));
}
__device__ __forceinline__ float transpose_sum(const float2 (&v)[8]) {
  return transpose_join(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float transpose_max(const float2 (&v)[8]) {
  return transpose_join(v, [](float a, float b) { return fmaxf(a, b); });
}

// ---- the softmax and the outputs ---------------------------------------------------
// Warp 4 g + q reads the scores of tokens 32 q .. + 31 (its tensor-memory lanes)
// for the 16 heads of group g.  The four warps of a group exchange what they
// need and take the same decisions from it.  O holds head h with dimensions
// 0-127 of each 256 in lane h, with dimensions 128-255 in lane 64 + h.
// The sums of a pair, in the weights' space: of each head 4 partial sums of the
// weights, 4 of what rounding took from the larger ones, and the reference.
__device__ __forceinline__ float head_sum(const float* w, int h, float* off) {
  const float* y = w + h;
  *off = (y[4 * kHeads] + y[5 * kHeads]) + (y[6 * kHeads] + y[7 * kHeads]);
  return (y[0] + y[kHeads]) + (y[2 * kHeads] + y[3 * kHeads]);
}

// log2 of a head's sum of weights: the sum's own exponent meets the reference
// first, so that a large one (all scales 0 or small) costs no bits.
__device__ __forceinline__ float lse2_of(float ref, float sum) {
  const int e = min(max((int)(__float_as_uint(sum) >> 23) - 127, -126), 126);
  return (ref + (float)e) + log2f(sum * pow2(-e));
}

// Softmax warps with a head; the others leave, and what they would hold (scores,
// weights and outputs of no head) stays as it is.
__device__ __forceinline__ int active_warps(int nheads) {
  return (nheads + kGroupHeads - 1) / kGroupHeads * 4;
}

// Outputs of a pair by warp `quad` of `groups` groups; `of_h` is the factor of
// head (quad & 1) 32 + lane.  The warp's 32 tensor-memory lanes hold heads
// (quad & 1) 32 + lane, 64 columns a group.  16 lanes and 32 columns at a time; a
// thread holds two columns of each 8 of two heads, and swaps with its neighbour
// so that four threads store 32 contiguous bytes of a head, a whole sector: 4.8
// thousand cycles a pair of 64 heads, 2.1 of them the stores.  (More with a head
// a thread and 32-byte stores, and with 16 bytes a thread after two exchanges.
// From the last stage's space by bulk copies it is 1.3, but the stage then comes
// back later: the same time in all, and 12 % more where pairs have two tiles.)
__device__ __forceinline__ void write_outputs(const MlaFp8Args& a, uint32_t lanes, int64_t head0,
                                              int nheads, int grp, int groups, float of_h,
                                              bool good) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  float inv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) inv[i] = __shfl_sync(kFull, of_h, 8 * i + (lane >> 2));
  const int j = lane & 3;
  for (int cg = grp; cg < 4; cg += groups) {
    __nv_bfloat16* orow = a.out + (head0 + (quad & 1) * 32 + (lane >> 2)) * kDv + (cg >> 1) * 256 +
                          (quad >> 1) * 128 + (cg & 1) * 64 + (j & 1) * 8 + (j >> 1) * 4;
#pragma unroll
    for (int up16 = 0; up16 < 2; ++up16) {
      if ((quad & 1) * 32 + up16 * 16 >= nheads) break;
      uint32_t o0[16], o1[16];             // columns 0-31 and 32-63
      tmem_ld32_of16(lanes + ((uint32_t)up16 << 20) + kOCol + cg * 64, o0);
      tmem_ld32_of16(lanes + ((uint32_t)up16 << 20) + kOCol + cg * 64 + 32, o1);
      tmem_wait(o0);
      tmem_wait(o1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {        // 32 columns; heads lane / 4, then 8 + lane / 4
        const int c = (q >> 1) * 32, half = q & 1;
        const uint32_t(&o)[16] = q < 2 ? o0 : o1;
        const float f = inv[2 * up16 + half];
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 y =
              __floats2bfloat162_rn(__uint_as_float(o[4 * i + 2 * half]) * f,
                                    __uint_as_float(o[4 * i + 2 * half + 1]) * f);
          b[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
        const int h = up16 * 16 + half * 8;
        const bool there = good && (quad & 1) * 32 + h + (lane >> 2) < nheads;
#pragma unroll
        for (int k = 0; k < 2; ++k) {      // columns 16 k .. + 15: 8-column groups 2 k, 2 k + 1
          const uint32_t give = j & 1 ? b[2 * k] : b[2 * k + 1];
          const uint32_t got = __shfl_xor_sync(kFull, give, 1);
          const uint2 v = j & 1 ? make_uint2(got, b[2 * k + 1]) : make_uint2(b[2 * k], got);
          if (there) *reinterpret_cast<uint2*>(orow + (int64_t)h * kDv + c + 16 * k) = v;
        }
      }
    }
  }
}

// With up to 32 heads (kFew), half of the softmax's warps or more have none:
// two warpgroups write the outputs, while the softmax goes on with the next
// pair, with more registers a thread (one scale for all blocks, 256 tokens a pair,
// 16 heads: 49.5 -> 46.4 us; 32 heads 53.2 -> 48.7; in longer pairs the same).  A pair's
// sums reach the writers in those parts of the weights' space that belong to no
// head, alternately in two: the softmax cannot end a pair before the outputs of
// the one before the last are written, as its first value product waits for
// them.
constexpr int kHanded = 32;                  // heads
__device__ __forceinline__ float* handed_over(Smem& sm, int which, int i) {
  const int t = i >> 2;                      // 16 bytes of a token's 64, swizzled as the weights are
  return reinterpret_cast<float*>(sm.plo + t * 64 + (((2 + which) ^ ((t >> 1) & 3)) << 4)) + (i & 3);
}

__device__ __forceinline__ void write_handed(const MlaFp8Args& a, Smem& sm, uint32_t tmem, int hg,
                                             int p0, int p1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3;
  const int nheads = min(kHeads, a.H - hg * kHeads), active = active_warps(nheads);
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  bool ok = true;
  Cursor cur(a, sm, p0, p1);
  for (int n = 0, pair = 0; cur.valid(p1); ++pair) {
    const int p = cur.p, which = pair & 1;
    n += (cur.count + kTile - 1) / kTile;
    cur.next_pair(a, sm, p0, p1);
    barrier(2 + kGroups + which, (active + kSoftmaxWarps - kWriter0) * 32);
    bool good = true;
    for (int i = 0; i < active; ++i) good = good && *handed_over(sm, which, 9 * kHanded + i) != 0.f;
    float off = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum += *handed_over(sm, which, i * kHanded + lane);
      off += *handed_over(sm, which, (4 + i) * kHanded + lane);
    }
    const float ref = *handed_over(sm, which, 8 * kHanded + lane);
    if (!wait_or_abort(sm, &sm.pvdone, (uint32_t)(n - 1) & 1u)) ok = false;
    good = __all_sync(kFull, good && ok);
    tc_fence_after();
    int shard;
    const int64_t head0 = list_of(a, p, &shard) * a.H + hg * kHeads;
    if (warp == kWriter0 && lane < nheads && good)
      a.lse2[head0 + lane] = sum == 0.f ? -INFINITY : lse2_of(ref, sum);
    write_outputs(a, lanes, head0, nheads, (warp - kWriter0) >> 2, (kSoftmaxWarps - kWriter0) / 4,
                  sum == 0.f ? 0.f : 1.f / (sum - off), good);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.ofree);
  }
  if (!__all_sync(kFull, ok) && lane == 0 && !aborted(sm)) abort_cta(sm, a.flags);
}

template <bool kSplit, bool kFew>
__device__ __forceinline__ void softmax_and_store(const MlaFp8Args& a, Smem& sm, uint32_t tmem,
                                                  int hg, int p0, int p1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, grp = warp >> 2;
  const int token = quad * 32 + lane, col0 = grp * kGroupHeads, col = col0 + (lane & 15);
  const int nheads = min(kHeads, a.H - hg * kHeads);
  const int active = active_warps(nheads);
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  bool ok = true;
  // A wait that fails leaves `ok` false; nothing is written out then.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!wait_or_abort(sm, bar, parity)) ok = false;
    __syncwarp();
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive1(bar);
  };
  // Nothing selected on a shard: O = 0, lse2 = -inf.
  for (int p = p0 + warp; !kSplit && p < p1; p += active) {
    int shard;
    const int64_t at = list_of(a, p, &shard);
    if (__ldg(a.counts + at) > 0) continue;
    const int64_t head0 = at * a.H + hg * kHeads;
    for (int i = lane; i < nheads * (kDv / 8); i += 32)
      reinterpret_cast<uint4*>(a.out + head0 * kDv)[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < nheads; i += 32) a.lse2[head0 + i] = -INFINITY;
  }
  Cursor cur(a, sm, p0, p1);
  if (cur.valid(p1)) {
    const float f = split_query(a, sm, row_of(a, cur.p), hg);
    if (lane < 4) sm.fq[4 * warp + lane] = f;
    barrier(1 + kGroups, active * 32);
  }
  int n = 0, which = 0;                      // tiles done; the parity of pairs
#pragma unroll 1
  while (cur.valid(p1)) {
    const int p = cur.p, ntiles = (cur.count + kTile - 1) / kTile;
    cur.next_pair(a, sm, p0, p1);
    const bool first = cur.valid(p1) && row_of(a, cur.p) != row_of(a, p);   // of its row
    // The last pair's sums have been read, and a new row's factors are there.
    if (n > 0 && !kFew) barrier(1 + kGroups, active * 32);
    const float4* fq = reinterpret_cast<const float4*>(sm.fq + col0);
    float ref = 0.f;                         // of head `col`
    bool fresh = true;                       // every token so far left out: no reference yet
    float2 l[8], gone[8];                    // weights; weights less their two parts
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = gone[i] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int t = 0; t < ntiles; ++t, ++n) {
      const int sb = n & 1;
      if (first && t + 1 == ntiles) {
        // The next row's query on its way to L2, 128 bytes a thread.
        const char* q = reinterpret_cast<const char*>(
            a.q + ((int64_t)row_of(a, cur.p) * a.H + hg * kHeads) * kDqk);
        for (int i = threadIdx.x; i < nheads * kDqk / 64; i += active * 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i * 128));
      }
      wait(&sm.fullB[sb], (uint32_t)(n >> 1) & 1u);   // the token's scale is there
      const float held = sm.tok[sb][token], ts = fmaxf(held, 0.f);
      const bool in = held >= 0.f;
      // A token of scale 0 has no product whose precision the reference would
      // serve: it only keeps its weight within fp32, as the least scale does.
      const float lt = ts > 0.f ? __log2f(ts) : kLog2MinScale;
      wait(&sm.sfull[sb], (uint32_t)(n >> 1) & 1u);
      tc_fence_after();
      // Exponents of 16 heads relative to their references: the query's parts
      // added, times the token's scale and the head's factor.
      float2 x[8];
      {
        uint32_t hi[16], lo[16];
        tmem_ld16(lanes + kSCol + sb * 128 + col0, hi);
        tmem_ld16(lanes + kSCol + sb * 128 + kHeads + col0, lo);
        const float4* rf = reinterpret_cast<const float4*>(sm.ref[sb ^ 1] + col0);
        const float2 t2 = make_float2(ts, ts);
        tmem_wait(hi);
        tmem_wait(lo);
        tc_fence_before();
        arrive(&sm.sfree[sb]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = fq[i], r = t > 0 ? rf[i] : make_float4(0.f, 0.f, 0.f, 0.f);
          const float2 u = fadd2(
              make_float2(__uint_as_float(hi[4 * i]), __uint_as_float(hi[4 * i + 1])),
              make_float2(__uint_as_float(lo[4 * i]), __uint_as_float(lo[4 * i + 1])));
          const float2 v = fadd2(
              make_float2(__uint_as_float(hi[4 * i + 2]), __uint_as_float(hi[4 * i + 3])),
              make_float2(__uint_as_float(lo[4 * i + 2]), __uint_as_float(lo[4 * i + 3])));
          x[2 * i] = ffma2(fmul2(u, t2), make_float2(f.x, f.y), make_float2(-r.x, -r.y));
          x[2 * i + 1] = ffma2(fmul2(v, t2), make_float2(f.z, f.w), make_float2(-r.z, -r.w));
        }
      }
      if (!__all_sync(kFull, in)) {          // a last tile, or a token left out
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!in) x[i] = make_float2(-INFINITY, -INFINITY);
      }
      // The references stay unless some weight of the group's heads would pass
      // its bound: then, as for a pair's first tile, the heads' maxima decide
      // the new ones.
      bool moves = fresh;
      if (!fresh) {
        float2 top = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          top.x = fmaxf(top.x, x[i].x);
          top.y = fmaxf(top.y, x[i].y);
        }
        moves = barrier_or(1 + grp, 128, fmaxf(top.x, top.y) + lt > kGap);
      }
      float alpha = 1.f;
      if (moves) {
        float2 xt[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) xt[i] = fadd2(x[i], make_float2(lt, lt));
        sm.part[quad][col] = transpose_max(xt);
        barrier(1 + grp, 128);
        // Relative to `ref`; -inf where the tile has no token.
        const float mx = fmaxf(fmaxf(sm.part[0][col], sm.part[1][col]),
                               fmaxf(sm.part[2][col], sm.part[3][col]));
        const bool move = fresh ? mx > -INFINITY : mx > kGap;
        const float up = move ? mx - kTop : 0.f;
        // The sums take the factor in two steps: before it they may be as far
        // above 1 as it is below (with scales at both ends of their range).
        float step = 1.f;
        if (!fresh) step = fast_exp2(-0.5f * up);
        alpha = step * step;
        const bool first_tile = fresh;
        fresh = fresh && !__any_sync(kFull, move);
        ref += up;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 d = make_float2(__shfl_sync(kFull, up, 2 * i), __shfl_sync(kFull, up, 2 * i + 1));
          x[i] = fadd2(x[i], make_float2(-d.x, -d.y));
          if (!first_tile) {
            const float2 f = make_float2(__shfl_sync(kFull, step, 2 * i),
                                         __shfl_sync(kFull, step, 2 * i + 1));
            l[i] = fmul2(fmul2(l[i], f), f);
            gone[i] = fmul2(fmul2(gone[i], f), f);
          }
        }
        // The maxima have been read before another tile's are written.
        barrier(1 + grp, 128);
      }
      sm.ref[sb][col] = ref;                 // the group's four warps alike
      const float rts = ts > 0.f ? __frcp_rn(ts) : 0.f;
      uint32_t phi[4], plo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = 2 * i + k;
          const float2 w = make_float2(fast_exp2(x[e].x), fast_exp2(x[e].y));
          l[e] = fadd2(l[e], w);
          // The token's scale goes with its weight into the value product.
          const float2 wt = fmul2(w, make_float2(ts, ts));
          const __half2 pw = __floats2half2_rn(wt.x, wt.y);
          hi[k] = to_e4m3x2(pw);
          const __half2 rest = __hsub2(pw, of_e4m3x2(hi[k]));
          lo[k] = to_e5m2x2(rest);
          // Only a relative loss (to 2^-7) is taken from the normaliser: below
          // e4m3's normal range, 2^-6, a product may round away whole, however
          // much of the normaliser its weight is where its scale is small.
          const __half2 counts = __hge2(pw, __floats2half2_rn(0x1p-6f, 0x1p-6f));
          const float2 lost = __half22float2(__hmul2(__hsub2(rest, of_e5m2x2(lo[k])), counts));
          gone[e] = ffma2(lost, make_float2(rts, rts), gone[e]);
        }
        phi[i] = hi[0] | (hi[1] << 16);
        plo[i] = lo[0] | (lo[1] << 16);
      }
      // The last tile's value products are done (its weights' space is free and
      // O holds every earlier tile).
      if (n > 0) wait(&sm.pvdone, (uint32_t)(n - 1) & 1u);
      // A reference has moved: the group's heads of O, 16 lanes of two quads.
      if (__any_sync(kFull, alpha != 1.f) && (quad & 1) == (grp >> 1)) {
        tc_fence_after();
        const float up = __shfl_sync(kFull, alpha, lane >> 2);
        const float down = __shfl_sync(kFull, alpha, 8 + (lane >> 2));
        const uint32_t o16 = lanes + ((uint32_t)(grp & 1) << 20) + kOCol;
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t o[16];
          tmem_ld32_of16(o16 + c, o);
          tmem_wait(o);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * (i & 2 ? down : up));
          tmem_st32_of16(o16 + c, o);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      const int at = token * 64 + ((grp ^ ((token >> 1) & 3)) << 4);
      *reinterpret_cast<uint4*>(sm.rope[sb] + at) = make_uint4(phi[0], phi[1], phi[2], phi[3]);
      *reinterpret_cast<uint4*>(sm.plo + at) = make_uint4(plo[0], plo[1], plo[2], plo[3]);
      proxy_fence();
      tc_fence_before();
      arrive(&sm.pfull);
    }
    // The sums over all tokens: 32 lanes, then the group's four warps, exchanged
    // in the weights' space once the value products have read it.
    const float all = transpose_sum(l), less = transpose_sum(gone);
    if (kFew) {
      *handed_over(sm, which, quad * kHanded + col) = all;
      *handed_over(sm, which, (4 + quad) * kHanded + col) = less;
      if (quad == 0) *handed_over(sm, which, 8 * kHanded + col) = ref;
      const bool good = __all_sync(kFull, ok);
      if (lane == 0) *handed_over(sm, which, 9 * kHanded + warp) = good ? 1.f : 0.f;
      __threadfence_block();
      barrier_arrive(2 + kGroups + which, (active + kSoftmaxWarps - kWriter0) * 32);
      which ^= 1;
      if (first) {
        const float factor = split_query(a, sm, row_of(a, cur.p), hg);
        barrier(1 + kGroups, active * 32);
        if (lane < 4) sm.fq[4 * warp + lane] = factor;
        barrier(1 + kGroups, active * 32);
      }
      continue;
    }
    // This row's scores are done: the next row's query takes the place of this
    // one's while the last value products run.
    float factor = 0.f;
    if (first) factor = split_query(a, sm, row_of(a, cur.p), hg);
    wait(&sm.pvdone, (uint32_t)(n - 1) & 1u);
    float* w = reinterpret_cast<float*>(sm.plo);
    w[quad * kHeads + col] = all;
    w[(4 + quad) * kHeads + col] = less;
    if (quad == 0) w[8 * kHeads + col] = ref;
    barrier(1 + kGroups, active * 32);
    if (first && lane < 4) sm.fq[4 * warp + lane] = factor;   // read after the next such barrier
    tc_fence_after();
    const bool good = __all_sync(kFull, ok);
    if (kSplit) break;                       // merged with the cluster's other parts
    int shard;
    const int64_t head0 = list_of(a, p, &shard) * a.H + hg * kHeads;   // first head of the CTA's
    if (warp < 2) {
      const int h = warp * 32 + lane;
      float off;
      const float sum = head_sum(w, h, &off);
      sm.part[0][h] = sum == 0.f ? 0.f : 1.f / (sum - off);
      if (h < nheads && good)
        a.lse2[head0 + h] = sum == 0.f ? -INFINITY : lse2_of(w[8 * kHeads + h], sum);
    }
    barrier(1 + kGroups, active * 32);
    write_outputs(a, lanes, head0, nheads, grp, active / 4, sm.part[0][(quad & 1) * 32 + lane], good);
  }
  if (!__all_sync(kFull, ok) && lane == 0 && !aborted(sm)) abort_cta(sm, a.flags);
}

// ---- a split pair's parts together ---------------------------------------------
// Every CTA of the cluster writes the O of its part of the list, unscaled, and
// its sums to its slot of the workspace: through shared memory and bulk copies,
// 16 dimensions of 32 heads at a time ([dims / 16][head][16] fp32, the 16-byte
// chunks of a head swizzled by it against bank conflicts, and so they stay).
// After one cluster barrier each reads all parts of the 512 / C dimensions that
// are its own, from L2, and adds them in rank order.
// (The same exchange through distributed shared memory, written or read 16
// bytes a lane, moved about 5 bytes a cycle: 13 us of a 26 us call.)
constexpr int kSlotFloats = kHeads * kDv + 4 * kHeads;   // O; sum, loss, reference, failed

__device__ __forceinline__ void merge_parts(const MlaFp8Args& a, Smem& sm, uint32_t tmem, int hg, int p,
                                            bool mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, grp = warp >> 2;
  const uint32_t rank = cluster_rank(), parts = cluster_size();
  const int nheads = min(kHeads, a.H - hg * kHeads), active = active_warps(nheads);
  float* slots = a.work + (int64_t)(blockIdx.x - rank) * kSlotFloats;   // of the cluster's CTAs
  float* slot = slots + (int64_t)rank * kSlotFloats;
  for (int h = threadIdx.x; h < nheads; h += active * 32) {
    const float* w = reinterpret_cast<const float*>(sm.plo);
    float off = 0.f;
    float* to = slot + kHeads * kDv + h;
    to[0] = mine ? head_sum(w, h, &off) : 0.f;
    to[kHeads] = off;
    to[2 * kHeads] = mine ? w[8 * kHeads + h] : 0.f;
    to[3 * kHeads] = aborted(sm) ? 1.f : 0.f;
  }
  if (mine) {
    const int h = (quad & 1) * 32 + lane;    // this thread's head, 64 columns a group
    float4* space = reinterpret_cast<float4*>(sm.kv[0][0]);
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    tc_fence_after();
    for (int cg = grp; cg < 4 && (quad & 1) * 32 < nheads; cg += active / 4) {
      const int d0 = (cg >> 1) * 256 + (quad >> 1) * 128 + (cg & 1) * 64;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t o[16];
        tmem_ld16(lanes + kOCol + cg * 64 + c, o);
        tmem_wait(o);
        const int at = ((d0 + c) / 16 * kHeads + h) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          space[at + (i ^ ((h >> 1) & 3))] =
              make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                          __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        proxy_fence();
        __syncwarp();
        if (lane == 0)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                           reinterpret_cast<float4*>(slot) + at),
                       "r"(smem_u32(space + at)), "r"(32 * 64)
                       : "memory");
      }
    }
    if (lane == 0) {
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      asm volatile("fence.proxy.async.global;" ::: "memory");
    }
    __syncwarp();
  }
  cluster_sync();                            // releases and acquires what was written
  int shard;
  const int64_t head0 = list_of(a, p, &shard) * a.H + hg * kHeads;
  float* factor = reinterpret_cast<float*>(sm.plo);   // [C][64]
  bool good = true;
  if ((int)threadIdx.x < nheads) {
    const int h = threadIdx.x;
    float sum[8], off[8], ref[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      sum[c] = off[c] = ref[c] = 0.f;
      if (c < (int)parts) {
        const float* at = slots + (int64_t)c * kSlotFloats + kHeads * kDv + h;
        sum[c] = __ldcg(at);
        off[c] = __ldcg(at + kHeads);
        ref[c] = __ldcg(at + 2 * kHeads);
        good &= __ldcg(at + 3 * kHeads) == 0.f;
      }
    }
    float top = -INFINITY, all = 0.f, less = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (sum[c] != 0.f) top = fmaxf(top, ref[c]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      // (In two steps, as above.)
      const float step = sum[c] != 0.f ? fast_exp2(0.5f * (ref[c] - top)) : 0.f;
      all = fmaf(sum[c] * step, step, all);
      less = fmaf(off[c] * step, step, less);
      ref[c] = step * step;
    }
    const float inv = all == 0.f ? 0.f : 1.f / (all - less);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < (int)parts) factor[c * kHeads + h] = ref[c] * inv;
    if (rank == 0 && good)
      a.lse2[head0 + h] = all == 0.f ? -INFINITY : lse2_of(top, all);
  }
  good = !barrier_or(1 + kGroups, active * 32, !good);
  const int groups = kDv / 16 / (int)parts;  // of 16 dimensions; a thread takes 8 of a head
  for (int i = threadIdx.x; i < 2 * nheads * groups; i += active * 32) {
    const int gi = (i >> 1) / nheads, h = (i >> 1) - gi * nheads, d16 = (int)rank * groups + gi;
    uint32_t b[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float4* at = reinterpret_cast<const float4*>(slots) + (d16 * kHeads + h) * 4 +
                         ((2 * (i & 1) + half) ^ ((h >> 1) & 3));
      float4 u[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < (int)parts) u[c] = __ldcg(at + (int64_t)c * (kSlotFloats / 4));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float f = c < (int)parts ? factor[c * kHeads + h] : 0.f;
        if (f != 0.f)                        // a part without tokens has written nothing
          x = make_float4(fmaf(u[c].x, f, x.x), fmaf(u[c].y, f, x.y), fmaf(u[c].z, f, x.z),
                          fmaf(u[c].w, f, x.w));
      }
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(x.x, x.y), y1 = __floats2bfloat162_rn(x.z, x.w);
      b[2 * half] = *reinterpret_cast<const uint32_t*>(&y0);
      b[2 * half + 1] = *reinterpret_cast<const uint32_t*>(&y1);
    }
    if (good)
      *reinterpret_cast<uint4*>(a.out + (head0 + h) * kDv + d16 * 16 + (i & 1) * 8) =
          make_uint4(b[0], b[1], b[2], b[3]);
  }
}

template <bool kSplit, bool kFew>
__global__ void __launch_bounds__(kThreads, 1) sparse_mla_decode_fp8_kernel(const MlaFp8Args a) {
  extern __shared__ __align__(1024) unsigned char mla_fp8_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(mla_fp8_smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  // Neighbouring CTAs (clusters) take the head groups of the same pairs, whose
  // rows the second finds in L2.
  const int parts = kSplit ? (int)cluster_size() : 1;
  const int unit = blockIdx.x / parts, units = gridDim.x / parts;
  const int hg = unit % a.hgroups, g = unit / a.hgroups, groups = units / a.hgroups;
  const int64_t pairs = (int64_t)a.rows * a.S;
  const int p0 = (int)(pairs * g / groups), p1 = (int)(pairs * (g + 1) / groups);
  const int nheads = min(kHeads, a.H - hg * kHeads), active = active_warps(nheads);

  int total = 0;                             // tokens of a split pair, over the cluster
  for (int p = p0 + (kSplit ? 0 : tid); p < p1; p += kThreads) {
    int shard;
    int count = __ldg(a.counts + list_of(a, p, &shard));
    if ((count < 0 || count > a.K) && (!kSplit || tid == 0)) raise_flag(a.flags, DSA_FLAG_BOUNDS);
    count = min(max(count, 0), a.K);
    if (kSplit) {                            // the one pair: this CTA's tiles of it
      total = count;
      const int tiles = (count + kTile - 1) / kTile, rank = (int)cluster_rank();
      const int lo = tiles * rank / parts * kTile, hi = tiles * (rank + 1) / parts * kTile;
      if (tid == 0) {
        sm.first = lo;
        sm.counts[0] = min(count, hi) - min(count, lo);
      }
    } else if (p - p0 < kCounts) {
      sm.counts[p - p0] = count;
    }
  }
  if (kSplit && total == 0) {
    // Nothing selected on this shard: O = 0, lse2 = -inf.
    int shard;
    const int64_t head0 = list_of(a, p0, &shard) * a.H + hg * kHeads;
    for (int i = tid; i < nheads * (kDv / 8) && cluster_rank() == 0; i += kThreads)
      reinterpret_cast<uint4*>(a.out + head0 * kDv)[i] = make_uint4(0, 0, 0, 0);
    if (cluster_rank() == 0 && tid < nheads) a.lse2[head0 + tid] = -INFINITY;
    return;                                  // the whole cluster alike
  }
  if (!kSplit && tid == 0) sm.first = 0;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.fullA[i], 32 * kGatherWarps + kStalledArrivals);   // every gathering lane
      mbar_init(&sm.fullB[i], 33 * kGatherWarps);
      mbar_init(&sm.emptyA[i], 1);
      mbar_init(&sm.emptyB[i], 1);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sfree[i], active);
    }
    mbar_init(&sm.qfull, active);
    mbar_init(&sm.pfull, active);
    mbar_init(&sm.pvdone, 1);
    mbar_init(&sm.ofree, kSoftmaxWarps - kWriter0);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (kFew && warp < kWriter0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp < active) softmax_and_store<kSplit, kFew>(a, sm, tmem, hg, p0, p1);
  } else if (kFew && warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWriter));
    write_handed(a, sm, tmem, hg, p0, p1);
  } else if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    if (warp < active) {
      softmax_and_store<kSplit, kFew>(a, sm, tmem, hg, p0, p1);
      if (kSplit) merge_parts(a, sm, tmem, hg, p0, sm.counts[0] > 0);
    } else if (kSplit) {
      cluster_sync();                        // the merge's barrier
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsGather));
    gather_tiles(a, sm, p0, p1);
    if (kSplit) cluster_sync();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (tid == kMmaWarp * 32)
      drain_mmas(a, sm, &sm.drain[0], issue_scores(a, sm, tmem, p0, p1));
    else if (tid == (kMmaWarp + 1) * 32)
      drain_mmas(a, sm, &sm.drain[1], issue_values(a, sm, tmem, p0, p1, kFew));
    __syncwarp();
    if (kSplit) cluster_sync();
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

// Clusters of `parts` CTAs of the split kernel that the device runs at the same
// time; 0 if that cannot be told.
int clusters_at_once(unsigned parts, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  const auto e = cudaOccupancyMaxActiveClusters(&n, sparse_mla_decode_fp8_kernel<true, false>, &cfg);
  return e == cudaSuccess ? n : 0;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace dsa

using namespace dsa;

// Few pairs are split, each over a cluster of at most as many CTAs (up to 8) as
// the SMs hold, with four tiles or more a CTA before the last doubling: two
// tiles cost about what the merge does.  A launch takes fewer where that many
// clusters do not run at once (a cluster lies within a group of SMs, and not
// every group is a multiple of it: 15 of 8, 36 of 4 and 76 of 2 do), as the ones
// left over would be a second round: 9 rows of 128 heads and 2048 tokens took
// 37.6 us over 8, 24.6 over 4; 19 rows 46.8 over 4, 34.7 over 2.
static int split_parts(int64_t pairs, int64_t hgroups, int K) {
  const int tiles = (K + kTile - 1) / kTile;
  int parts = 1;
  if (pairs > kSms || hgroups > kSms) return parts;
  while (parts < 8 && pairs * hgroups * parts * 2 <= kSms && parts * 4 <= tiles) parts *= 2;
  return parts;
}

extern "C" int64_t dsa_sparse_mla_decode_fp8_work(int rows, int S, int H, int K) {
  if (rows < 1 || S < 1 || S > DSA_MAX_SHARDS || H < 1 || K < 1 || K > kMaxList) return 0;
  const int64_t pairs = (int64_t)rows * S, hgroups = ((int64_t)H + kHeads - 1) / kHeads;
  const int parts = split_parts(pairs, hgroups, K);
  return parts > 1 ? pairs * hgroups * parts * kSlotFloats * 4 : 0;
}

extern "C" dsa_status dsa_sparse_mla_decode_fp8(const uint16_t* q, const uint8_t* kv_cache,
                                                const float* block_scales, int64_t n_slots,
                                                int block_tokens, const int32_t* slots,
                                                const int32_t* counts, int rows, int S, int H,
                                                int K, float scale, uint16_t* out, float* lse2,
                                                float* work, uint32_t* err_flags,
                                                cudaStream_t stream) {
  if (rows < 0 || K < 1 || H < 1 || n_slots < 1 || block_tokens < 1 || n_slots % block_tokens ||
      !std::isfinite(scale))
    return DSA_ERR_INVALID_ARG;
  if (S < 1 || S > DSA_MAX_SHARDS || n_slots > INT32_MAX || K > kMaxList)
    return DSA_ERR_UNSUPPORTED;
  if (rows == 0) return DSA_OK;
  if (!q || !kv_cache || !block_scales || !slots || !counts || !out || !lse2)
    return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out) || !aligned16(work))
    return DSA_ERR_INVALID_ARG;
  const int64_t hgroups = ((int64_t)H + kHeads - 1) / kHeads, pairs = (int64_t)rows * S;
  if (pairs > INT32_MAX || hgroups > INT32_MAX / kSms) return DSA_ERR_UNSUPPORTED;
  // One CTA an SM: as many groups of pairs as all SMs hold with each head group.
  const int64_t groups = std::min<int64_t>(pairs, std::max<int64_t>(1, kSms / hgroups));
  unsigned parts = work ? (unsigned)split_parts(pairs, hgroups, K) : 1u;
  const int smem = (int)sizeof(Smem);
  if (parts > 1 &&
      cudaFuncSetAttribute(sparse_mla_decode_fp8_kernel<true, false>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  while (parts > 1 && pairs * hgroups > clusters_at_once(parts, (size_t)smem)) parts /= 2;   // (0.3 us each)
  const auto kernel =
      parts > 1       ? sparse_mla_decode_fp8_kernel<true, false>
      : H <= kHanded ? sparse_mla_decode_fp8_kernel<false, true>
                     : sparse_mla_decode_fp8_kernel<false, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const MlaFp8Args a{reinterpret_cast<const __nv_bfloat16*>(q),
                     kv_cache,
                     block_scales,
                     slots,
                     counts,
                     n_slots,
                     n_slots / block_tokens,
                     rows,
                     S,
                     H,
                     K,
                     (int)hgroups,
                     scale * kLog2e,
                     reinterpret_cast<__nv_bfloat16*>(out),
                     lse2,
                     work,
                     err_flags,
                     FastDiv((uint32_t)block_tokens),
                     FastDiv((uint32_t)S)};
  const cudaError_t e =
      launch_kernel(kernel, dim3((unsigned)(groups * hgroups * parts)), dim3(kThreads),
                    (size_t)smem, stream, parts > 1 ? parts : 0u, a);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
