// Helpers of the latent-attention kernels over whole contexts: matrix
// descriptors, tcgen05 instructions, tensor-map copies, bounded waits.
//
// CG is the tcgen05 CTA group of a kernel (1, or 2 for a pair of CTAs that
// share one product): every tcgen05 instruction of a kernel has the same one.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "common.cuh"

namespace dsa {

constexpr float kLog2e = 1.4426950408889634f;
// SMs of a GB300, for which calls are cut.  (A constant: the size of a workspace and the
// launch that uses it go by the same number, whatever device is current at either.)
constexpr int kSms = 152;
// A softmax's reference moves when a tile's maximum exceeds it by this much in
// binades: weights stay below 2^8, and accumulators are rescaled rarely.
constexpr float kRescaleGap = 8.f;

// Shared-memory matrix descriptor with the 128-byte swizzle: start address >> 4
// (bits 0-13), leading byte offset >> 4 (bits 16-29), stride byte offset >> 4
// (bits 32-45), version 1 (bits 46-47), swizzle mode 2 (bits 61-63).  K-major:
// the stride is that of 8-row groups, the leading offset unused.  MN-major: the
// leading offset steps between 64-element atoms along M or N, the stride
// between 8-row groups along K.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The same value in every lane, made known as such: what follows from it stays in
// uniform registers, and branches on it are the warp's.
__device__ __forceinline__ int uni(int v) { return __shfl_sync(kFull, v, 0); }
__device__ __forceinline__ uint32_t uni(uint32_t v) { return __shfl_sync(kFull, v, 0); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B of one
// type (bits 7-9, 10-12: 0 fp16, 1 bf16), A K-major, B K-major or MN-major (bit
// 16), N >> 3 (bits 17-22), M >> 4 (bits 24-28).
constexpr uint32_t idesc_f16(int m, int n, bool bf16, bool b_mn_major) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

constexpr uint32_t kNegateA = 1u << 13;      // descriptor bit: D = or += -A B
constexpr uint32_t kAcrossA = 1u << 15;      // descriptor bit: A MN-major

// D (tensor memory) = or += A B: A from shared memory (_ss) or tensor memory (_ts).
template <int CG>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accum) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accum) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}

// One arrival on `bar` once every MMA issued so far has completed (a pair: on
// the barrier of both CTAs).
template <int CG>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// Tensor memory of a CTA (a pair: of both, by one warp of each).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(where)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(where)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// This thread's writes to shared memory, read next by a product (of a pair: that
// the first CTA issues).
template <int CG>
__device__ __forceinline__ void fence_for_products() {
  fence_async_smem();
  if constexpr (CG == 2) asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive1(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A CTA's word that one role sets when a wait of its ran out; the others stop
// at their next wait.
__device__ __forceinline__ bool cta_aborted(const int* abort) {
  return *reinterpret_cast<const volatile int*>(abort) != 0;
}
__device__ __forceinline__ void cta_abort(int* abort, uint32_t* flags) {
  raise_flag(flags, DSA_FLAG_TIMEOUT);
  *reinterpret_cast<volatile int*>(abort) = 1;
}
// Bounded wait (a few seconds) that also gives up once another role has aborted.
__device__ __forceinline__ bool wait_or_abort(const int* abort, uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitPolls / 4; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && cta_aborted(abort)) return false;
  }
  return false;
}
// The same for what lands before a CTA may end: it waits on when others have aborted.
__device__ __forceinline__ bool wait_landed(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitPolls / 4; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
// wait_or_abort for a converged warp, all lanes alike.  All of them poll: a branch for
// one lane costs every wait its divergence (8192 queries of 128 heads, expanded:
// 2992 us with one polling lane, 2180 so).
__device__ __forceinline__ bool warp_wait(const int* abort, uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, wait_or_abort(abort, bar, parity));
}

// ---- pairs of CTAs ----------------------------------------------------------
__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of the same object in the pair's first CTA.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// A box into this CTA's memory, its bytes counted by `bar` (a shared::cluster address).
template <int CG>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, int z,
                                         uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// One arrival on the barrier of the pair's first CTA.  What it announces lies in
// tensor memory (waited for and fenced by tcgen05 instructions): released to the
// CTA's scope alone.  With .cluster it waits for every memory access of the thread
// before, and a hand-over of weights took 1400 cycles instead of 150.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
// Every thread of both CTAs.
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- items of work, shared out while the kernel runs -------------------------
// The grid has a cluster of CG CTAs for every item; those that the device has not
// started yet are cancelled by running ones, which take their items over (cluster
// launch control), so that CTAs end together whatever their items' lengths, and
// the next item's first copies run under the last one's end.  One warp of each
// CTA claims items and works out what they are; the others read that from two
// slots in shared memory.
template <typename Item>
struct WorkSlots {
  uint4 claimed;              // the launch control's answer (of a pair: to both CTAs)
  uint64_t answer, ready;     // it has come; both CTAs are ready for the next one
  uint64_t full[2], empty[2];
  Item item[2];
  int last[2];                // nothing here: no more items
};
template <typename Item>
__device__ __forceinline__ void init_slots(WorkSlots<Item>& s, int cg, int readers) {
  mbar_init(&s.answer, 1);
  mbar_init(&s.ready, cg);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&s.full[i], 1);
    mbar_init(&s.empty[i], readers);
  }
}

// The claiming warp.  `find` (warp-wide) says what item `index` < total is.
template <int CG, typename Item, typename Find>
__device__ __forceinline__ void share_out(WorkSlots<Item>& s, int* abort, uint32_t* flags,
                                          int64_t total, uint32_t rank, Find&& find) {
  const int lane = threadIdx.x & 31;
  int64_t index = blockIdx.x / CG;
  uint32_t claims = 0;
  bool ok = true;
  for (uint32_t n = 0; ok; ++n) {
    const uint32_t slot = n & 1u;
    const bool last = index >= total;
    Item it{};
    if (!last) it = find(index);
    if (n >= 2) ok = warp_wait(abort, &s.empty[slot], ((n >> 1) - 1) & 1u);
    if (!ok) break;
    if (lane == 0) {
      s.item[slot] = it;
      s.last[slot] = last;
      mbar_arrive1(&s.full[slot]);
    }
    if (last) return;
    bool got;
    do {                                     // clusters past the last item are only cancelled
      if (lane == 0) {
        mbar_expect_tx(&s.answer, 16);
        if (CG == 1) mbar_arrive1(&s.ready);
        else mbar_arrive_leader(&s.ready);
        if (rank == 0) {
          ok = wait_or_abort(abort, &s.ready, claims & 1u);
          if (ok) {
            if constexpr (CG == 1)
              asm volatile(
                  "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
                  " [%0], [%1];" ::"r"(smem_u32(&s.claimed)), "r"(smem_u32(&s.answer))
                  : "memory");
            else
              asm volatile(
                  "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
                  ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_u32(&s.claimed)),
                  "r"(smem_u32(&s.answer))
                  : "memory");
          }
        }
      }
      const bool asked = __shfl_sync(kFull, (int)ok, 0) != 0;
      ok = asked && warp_wait(abort, &s.answer, claims & 1u);
      // An answer under way is not left to land in memory of the CTA that comes next.  (A
      // pair's second CTA does not know whether the first has asked: at worst it waits
      // until the bound.)
      if (!ok && asked) wait_landed(&s.answer, claims & 1u);
      __syncwarp();
      ++claims;
      uint32_t x = 0, yes = 0;
      if (ok)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
            "ld.shared.b128 r, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
            "selp.u32 %1, 1, 0, p;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
            : "+r"(x), "=r"(yes)
            : "r"(smem_u32(&s.claimed))
            : "memory");
      got = ok && yes != 0;
      index = got ? (int64_t)(x / CG) : total;
      fence_async_smem();                    // read before the next answer is written
      __syncwarp();
    } while (got && index >= total);
  }
  if (lane == 0 && !cta_aborted(abort)) cta_abort(abort, flags);
  __syncwarp();
}

// Sequences by length, the longest first, so that CTAs, which claim items in this
// order, end alike.  A rank is found by comparing with all, a thread a sequence, by
// all threads of the CTA; `i` is taken as it is where the call is not to order.
constexpr int kOrder = 128;
struct Order {
  int length[kOrder];
  uint8_t at[kOrder];
};
template <typename Len>
__device__ __forceinline__ void longest_first(Order& o, int n, int tid, Len&& len) {
  if (tid < n) o.length[tid] = len(tid);
  __syncthreads();
  if (tid >= n) return;
  const int mine = o.length[tid];
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) rank += o.length[j] > mine || (o.length[j] == mine && j < tid);
  o.at[rank] = (uint8_t)tid;
}
__device__ __forceinline__ int in_order(const Order& o, bool ordered, int i) {
  return ordered ? o.at[min(i, kOrder - 1)] : i;
}
// Whether to: items a CTA, so that the last ones' ends matter, in us, in the batch's
// order against this: 64 requests of 8192 to 16384 tokens on 4 shards 388 / 358 (512
// items on 152 CTAs), 128 of 2048 to 8192 on 8 shards 166 / 163 (1024 on 152), ten
// prompts of 1 to 2048 tokens 84 / 78 (272 on 76 pairs); but trees of eight for those
// 64 requests 1525 / 1540 (2048 on 76).  Ranks cost 1 us for 128 sequences.
inline bool order_pays(int n, int64_t items, int64_t ctas) { return n > 1 && n <= kOrder && items <= 16 * ctas; }

// A reading warp's n-th item; false at the end (or where a wait ran out).
template <typename Item>
__device__ __forceinline__ bool next_item(const WorkSlots<Item>& s, const int* abort, uint32_t n,
                                          bool& ok) {
  const uint32_t slot = n & 1u;
  ok = ok && warp_wait(abort, const_cast<uint64_t*>(&s.full[slot]), (n >> 1) & 1u);
  return ok && !s.last[slot];
}
template <typename Item>
__device__ __forceinline__ bool next_item(const WorkSlots<Item>& s, const int* abort, uint32_t n,
                                          bool& ok, Item& it) {
  const bool more = next_item(s, abort, n, ok);
  if (more) {
    static_assert(sizeof(Item) % 4 == 0, "an item is words");
    int w[sizeof(Item) / 4];
#pragma unroll
    for (unsigned i = 0; i < sizeof(Item) / 4; ++i) w[i] = uni(reinterpret_cast<const int*>(&s.item[n & 1u])[i]);
    memcpy(&it, w, sizeof(Item));
  }
  return more;
}
template <typename Item>
__device__ __forceinline__ void item_done(WorkSlots<Item>& s, uint32_t n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive1(&s.empty[n & 1u]);
}

// Entries i and i + 1 of ascending bounds cu[0 .. n] of T rows; of others (`bad`) each
// taken as the nearest inside the rows that is not below one before it, so that no row
// is in two sequences.
__device__ __forceinline__ void bounds_of(const int32_t* cu, int i, int T, bool bad, int& first, int& end) {
  first = min(max(__ldg(cu + i), 0), T);
  if (bad)
    for (int j = 0; j < i; ++j) first = max(first, min(__ldg(cu + j), T));
  end = min(max(__ldg(cu + i + 1), first), T);
}
// Warp-wide: how many blocks of up to `size` the rows of n sequences make, `times` of
// them a row; whether bounds (cu's, or those of `more`) are bad, flagged once a call.
__device__ __forceinline__ int count_blocks(const int32_t* cu, int T, const int32_t* more, int T_more, int n,
                                            int times, int size, uint32_t* flags, bool& bad) {
  const int lane = threadIdx.x & 31;
  int blocks = 0;
  bad = false;
  for (int i = lane; i < n; i += 32) {
    int first, end;
    bounds_of(cu, i, T, false, first, end);
    bad |= first != __ldg(cu + i) || end != __ldg(cu + i + 1);
    blocks += ((end - first) * times + size - 1) / size;
    if (more) {
      bounds_of(more, i, T_more, false, first, end);
      bad |= first != __ldg(more + i) || end != __ldg(more + i + 1);
    }
  }
  bad = __any_sync(kFull, bad);
  if (bad) {
    if (blockIdx.x == 0 && lane == 0) raise_flag(flags, DSA_FLAG_BOUNDS);
    blocks = 0;
    for (int i = lane; i < n; i += 32) {
      int first, end;
      bounds_of(cu, i, T, true, first, end);
      blocks += ((end - first) * times + size - 1) / size;
    }
  }
  return __reduce_add_sync(kFull, blocks);
}

// Sixteen registers' uses are not scheduled before the wait for a load of them: empty
// statements name them as read and written.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// Sixteen columns of a warp's 32 lanes, a thread a lane.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
               "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                 "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, "
               "%8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
               "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
               "r"(r[15])
               : "memory");
}

// Sixteen lanes as fragments: of 8 fp32 columns a thread has, in registers 4 i to 4
// i + 3, columns 8 i + 2 (lane % 4) and the next of row lane / 4, then of row lane /
// 4 + 8; of 4 columns of 16-bit pairs, in registers 2 i and 2 i + 1, column 4 i +
// lane % 4 of either row: where the same thread's fp32 columns go as pairs.
__device__ __forceinline__ void tmem_load_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
               "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                 "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_store_frag(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, "
               "%8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
               "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
               "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_store_pairs(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, "
               "%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The largest of a warp's values that is no NaN.
__device__ __forceinline__ float warp_max(float v) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// In a branch rarely taken: keeps it one (as predicated instructions, a pass of
// 128 compares and selects cost every tile 300 cycles).
__device__ __forceinline__ void keep_branch() { asm volatile("" ::: "memory"); }

// 2^x (ex2.approx.ftz.f32: relative error about 2^-22, results below 2^-126
// flushed to zero; 2^-inf = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fused multiply-adds or additions in one instruction, each
// rounded as the scalar operation would be.
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
// Two values as 16-bit floats in one word, each rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

// A row's 32 columns as fragments hold them (row k of the lane's two: o[4 i + 2 k],
// o[4 i + 2 k + 1] are columns 8 i + 2 (lane % 4) and the next), as 16-bit floats to
// `row`: neighbouring lanes swap words, so that each stores eight bytes and the four
// lanes of a row whole sectors.
template <bool BF16>
__device__ __forceinline__ void store_row(const uint32_t (&o)[16], int k, int lane, bool active, uint16_t* row) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack16<BF16>(__uint_as_float(o[4 * i + 2 * k]), __uint_as_float(o[4 * i + 2 * k + 1]));
  const bool odd = (lane & 1) != 0;          // has i = 1, 3 in the end, an even lane i = 0, 2
  const uint32_t a = __shfl_xor_sync(kFull, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(kFull, odd ? w[2] : w[3], 1);
  if (active) {
    uint16_t* at = row + (odd ? 8 : 0) + (lane & 2 ? 4 : 0);
    *reinterpret_cast<uint2*>(at) = odd ? make_uint2(a, w[1]) : make_uint2(w[0], a);
    *reinterpret_cast<uint2*>(at + 16) = odd ? make_uint2(b, w[3]) : make_uint2(w[2], b);
  }
}

// ---- host ------------------------------------------------------------------
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Boxes of 64 values (128 bytes, 128-byte swizzle) by rows1 of dimension 1 by
// rows2 of dimension 2 of a [dim2][dim1][dim0] array of 16-bit values; strides
// in bytes, outside reads as zero.
inline bool encode_map16(CUtensorMap* map, const void* base, bool bf16, uint64_t dim0,
                         uint64_t dim1, uint64_t dim2, uint64_t stride1, uint64_t stride2,
                         uint32_t rows1, uint32_t rows2) {
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {dim0, dim1, dim2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {64, rows1, rows2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dsa
