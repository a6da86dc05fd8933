// Latent attention in its expanded form over a ragged batch (sm_103a).
//
// Per query i of a sequence and head h, over its visible keys j: x_j = scale *
// (q_i[0..128) . k_nope_j + q_i[128..192) . k_pe_j), k_pe shared by all heads,
// out = sum_j 2^(x_j log2 e) v_j / sum_j 2^(x_j log2 e) and lse2 = log2 sum_j
// exp(x_j), so that outputs over parts of a context are merged as a shard's are.
//
// Compute-bound: 640 operations a visible (query, key) pair, and the exponent
// of each.  A CTA is persistent over items (a head's block of 256 queries, or
// a part of its keys) and holds two tiles of 128 queries, so that one's softmax
// runs under the other's products.  Keys go in tiles of 128, the last first:
// the masked ones.  The scores' and values' products have M = N = 128, the
// smallest whose instructions run at the full rate.
//  * tensor memory: two score tiles (128 columns each; the weights take the
//    first half of the same columns as 16-bit pairs) and two outputs (128 each);
//  * shared memory: the queries (96 KB) and a ring of eight 16 KB blocks: a
//    tile's keys as three of [128 keys][64 values], its values as two of [64
//    keys][128 values], freed one by one, so that copies run about one and a
//    half tiles ahead;
//  * one warp copies (tensor maps, 128-byte swizzle), one thread issues the
//    products: values of tile t + 1, scores of tile t for the first query tile,
//    then for the second; the order alone keeps a score tile from being
//    overwritten while its weights are read;
//  * four warps a query tile, a thread a row: maximum, weights relative to a
//    reference that moves when exceeded by 2^8, their sum, the outputs.
// The weights' sum is of the fp32 weights; a weight enters the value product
// rounded to 16 bits (2^-8 of itself at most in bf16, 2^-11 in fp16), the
// reference's own weight is 1 and exact.
// Every wait is bounded and raises DSA_FLAG_TIMEOUT when it runs out.
#include <algorithm>

#include "split_merge.cuh"

namespace dsa {
namespace {

constexpr int kDn = DSA_MLA_DN, kDr = DSA_MLA_DR, kDv = DSA_MLA_DVH;
constexpr int kTileQ = 128, kBlockQ = 2 * kTileQ;   // queries of a tile, of an item
constexpr int kTileK = 128;                         // keys of a tile
constexpr int kBlock = 16384;                       // bytes of a block
constexpr int kQBlocks = (kDn + kDr) / 64;          // 3
constexpr int kKBlocks = kQBlocks, kVBlocks = 2, kTileBlocks = kKBlocks + kVBlocks;
constexpr int kRing = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 9;          // warps 0-3, 4-7: softmax of tile 0, 1
constexpr int kThreads = 384;
// Registers: 168 a thread at launch; the two softmax warpgroups take 208, the
// third (copies, products) keeps 88 of them: 2 x 208 + 88 = 3 x 168.
constexpr int kTmemCols = 512;
__device__ __forceinline__ constexpr int s_col(int g) { return g * 128; }
__device__ __forceinline__ constexpr int o_col(int g) { return 256 + g * 128; }
#ifdef DSA_TEST_STALLED_COPY
// The test-only build (never libdsa.so): the first key block's barrier expects
// one arrival that nothing makes (its copy still lands).
constexpr uint32_t kStalledArrivals = 1;
#else
constexpr uint32_t kStalledArrivals = 0;
#endif

struct alignas(1024) PrefillSmem {
  uint8_t q[2][kQBlocks][kBlock];
  uint8_t ring[kRing][kBlock];
  uint64_t qfull[2], qempty[2], full[kRing], empty[kRing], sfull[2], pfull[2], ofull[2], drain;
  uint32_t tmem;
  int blocks;                 // query blocks of all sequences
  int abort;
};

struct PrefillArgs {
  const int32_t *cu_q, *cu_k; // [n + 1]
  void* out;                  // [Tq][H][kDv]
  float* lse2;                // [Tq][H]
  float *part_o, *part_l;     // [splits][Tq][H][kDv], [splits][Tq][H]
  uint32_t* flags;
  int n, Tq, Tk, H, group, splits, causal;
  float c2;                   // scale * log2(e)
};

// Sequence i's rows of an array of T rows, kept inside it.
__device__ __forceinline__ void bounds_of(const int32_t* cu, int i, int T, int& first, int& end) {
  first = min(max(__ldg(cu + i), 0), T);
  end = min(max(__ldg(cu + i + 1), first), T);
}

// What an item is; the same in every warp.
struct Item {
  int head, split;
  int row0, rows;             // its queries: first row, how many
  int key0, lk;               // its sequence's keys
  int shift;                  // causal: row r of the block sees shift + r + 1 keys
  int t0, t1;                 // its key tiles
  int end[2];                 // each query tile's: [t0, end)
};

struct Cursor {               // where the last item's sequence was found
  int seq = 0, before = 0;    // query blocks before it
};

// Warp-wide: item `index` of a.H * blocks * splits.  Heads go in groups whose
// keys and values stay in L2 together; within one, a sequence's longest blocks
// (its last) come first, so that CTAs taking every gridDim-th item end alike.
__device__ __forceinline__ Item find_item(const PrefillArgs& a, int blocks, int64_t index,
                                          Cursor& c) {
  const int lane = threadIdx.x & 31;
  Item it;
  const int64_t group_items = (int64_t)blocks * a.group * a.splits;
  const int hg = (int)(index / group_items);
  const int rem = (int)(index - hg * group_items);
  const int heads = min(a.group, a.H - hg * a.group);
  it.split = rem % a.splits;
  const int x = rem / a.splits;
  const int qb = x / heads;
  it.head = hg * a.group + x % heads;
  if (qb < c.before) c = Cursor{};
  int local = 0, nb = 0;
  for (int base = c.seq;; base += 32) {
    const int i = base + lane;
    int first = 0, end = 0;
    if (i < a.n) bounds_of(a.cu_q, i, a.Tq, first, end);
    const int mine = (end - first + kBlockQ - 1) / kBlockQ;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(kFull, c.before + incl > qb);
    if (past) {
      const int l = __ffs(past) - 1;
      nb = __shfl_sync(kFull, mine, l);
      c.before += __shfl_sync(kFull, incl, l) - nb;
      c.seq = base + l;
      local = qb - c.before;
      break;
    }
    c.before += __shfl_sync(kFull, incl, 31);
    if (base + 32 >= a.n) break;             // not reached: qb < blocks
  }
  int q0, q1, k0, k1;
  bounds_of(a.cu_q, c.seq, a.Tq, q0, q1);
  bounds_of(a.cu_k, c.seq, a.Tk, k0, k1);
  const int at = (nb - 1 - local) * kBlockQ;
  it.row0 = q0 + at;
  it.rows = min(kBlockQ, q1 - it.row0);
  it.key0 = k0;
  it.lk = k1 - k0;
  it.shift = it.lk - (q1 - q0) + at;
  int nt = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int r = min(max(it.rows - g * kTileQ, 0), kTileQ);
    const int seen = r == 0 ? 0 : !a.causal ? it.lk : min(max(it.shift + g * kTileQ + r, 0), it.lk);
    it.end[g] = (seen + kTileK - 1) / kTileK;
    nt = max(nt, it.end[g]);
  }
  const int per = (nt + a.splits - 1) / a.splits;
  it.t0 = min(it.split * per, nt);
  it.t1 = min(it.t0 + per, nt);
#pragma unroll
  for (int g = 0; g < 2; ++g) it.end[g] = max(min(it.end[g], it.t1), it.t0);
  return it;
}

// Steps of 16 keys that tile t's value product takes for query tile g.
__device__ __forceinline__ int value_steps(const PrefillArgs& a, const Item& it, int g, int t) {
  int keys = min(it.lk - t * kTileK, kTileK);
  if (a.causal) {
    const int r = min(it.rows - g * kTileQ, kTileQ);
    keys = min(keys, it.shift + g * kTileQ + r - t * kTileK);
  }
  return (keys + 15) / 16;
}

// ---- warp 9: the copies ------------------------------------------------------
__device__ __forceinline__ void load_tiles(const PrefillArgs& a, PrefillSmem& sm,
                                           const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                           const CUtensorMap* tm_pe, const CUtensorMap* tm_v,
                                           int blocks, int64_t items) {
  const int lane = threadIdx.x & 31;
  Cursor cur;
  uint32_t seq = 0, loads[2] = {0, 0};       // ring blocks and query tiles copied so far
  bool ok = true;
  auto next_blocks = [&](int n, auto&& copy) {   // of kBlock bytes each
    for (int b = 0; ok && b < n; ++b, ++seq) {
      const uint32_t slot = seq % kRing, use = seq / kRing;
      if (use > 0) ok = wait_or_abort(&sm.abort, &sm.empty[slot], (use - 1) & 1u);
      if (!ok) break;
      mbar_expect_tx(&sm.full[slot], kBlock);
      copy(b, sm.ring[slot], &sm.full[slot]);
    }
  };
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item it = find_item(a, blocks, i, cur);
    if (lane == 0 && ok) {
      for (int t = it.t1 - 1; ok && t >= it.t0; --t) {
        for (int g = 0; ok && g < 2; ++g) {
          if (t != it.end[g] - 1) continue;  // the tile's first key tile: its queries
          if (loads[g] > 0) ok = wait_or_abort(&sm.abort, &sm.qempty[g], (loads[g] - 1) & 1u);
          if (!ok) break;
          mbar_expect_tx(&sm.qfull[g], kQBlocks * kBlock);
          for (int b = 0; b < kQBlocks; ++b)
            tma_load_3d(sm.q[g][b], tm_q, b * 64, it.head, it.row0 + g * kTileQ, &sm.qfull[g]);
          ++loads[g];
        }
        const int key = it.key0 + t * kTileK;
        next_blocks(kKBlocks, [&](int b, uint8_t* dst, uint64_t* bar) {
          if (b < kDn / 64) tma_load_3d(dst, tm_k, b * 64, it.head, key, bar);
          else tma_load_3d(dst, tm_pe, b * 64 - kDn, key, 0, bar);
        });
        next_blocks(kVBlocks, [&](int b, uint8_t* dst, uint64_t* bar) {
          tma_load_3d(dst, tm_v, 0, it.head, key + b * 64, bar);
          tma_load_3d(dst + kBlock / 2, tm_v, 64, it.head, key + b * 64, bar);
        });
      }
    }
    ok = __shfl_sync(kFull, (int)ok, 0) != 0;
    if (!ok) break;
  }
  if (lane == 0 && !ok) {
    if (!cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
    // Every copy issued lands before the CTA ends.
    for (int g = 0; g < 2; ++g)
      if (loads[g] > 0) mbar_wait(&sm.qfull[g], (loads[g] - 1) & 1u);
    for (uint32_t b = seq > kRing ? seq - kRing : 0; b < seq; ++b)
      mbar_wait(&sm.full[b % kRing], (b / kRing) & 1u);
  }
}

// ---- warp 8, one thread: the products ---------------------------------------
template <bool BF16>
__device__ __forceinline__ void issue_products(const PrefillArgs& a, PrefillSmem& sm, uint32_t tmem,
                                               int blocks, int64_t items) {
  constexpr uint32_t kIdS = idesc_f16(kTileQ, kTileK, BF16, false);
  constexpr uint32_t kIdO = idesc_f16(kTileQ, kDv, BF16, true);
  const int lane = threadIdx.x & 31;
  const uint32_t ring0 = smem_u32(sm.ring[0]);
  Cursor cur;
  uint32_t seq = 0;                          // ring block of the item's tile k: seq + k * kTileBlocks
  uint32_t np[2] = {0, 0}, nq[2] = {0, 0};   // weights and query tiles waited for so far
  bool ok = true;
  auto landed = [&](uint32_t b) {
    return wait_or_abort(&sm.abort, &sm.full[b % kRing], (b / kRing) & 1u);
  };
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item it = find_item(a, blocks, i, cur);
    const int tiles = it.t1 - it.t0;
    if (lane == 0 && ok && tiles > 0) {
      for (int k = 0; ok && k <= tiles; ++k) {
        const int t = it.t1 - 1 - k;         // scores of tile t, values of tile t + 1
        const uint32_t kb = seq + (uint32_t)k * kTileBlocks, vb = kb - kTileBlocks + kKBlocks;
        bool waited_v = false, waited_k = false;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (ok && k > 0 && t + 1 < it.end[g]) {
            ok = wait_or_abort(&sm.abort, &sm.pfull[g], np[g] & 1u);
            ++np[g];
            if (ok && !waited_v) {
              ok = landed(vb) && landed(vb + 1);
              waited_v = true;
            }
            if (!ok) break;
            tc_fence_after();
            const int steps = value_steps(a, it, g, t + 1);
            for (int s = 0; s < steps; ++s) {
              const uint32_t blk = ring0 + ((vb + (uint32_t)(s >> 2)) % kRing) * kBlock;
              mma_ts<1>(tmem + o_col(g), tmem + s_col(g) + s * 8,
                        smem_desc_sw128(blk + (s & 3) * 2048, kBlock / 2, 1024), kIdO,
                        (t + 1 < it.end[g] - 1 || s > 0) ? 1u : 0u);
            }
            if (k == tiles) tc_commit<1>(&sm.ofull[g]);   // the output is complete
          }
          if (ok && g == 1 && k > 0) {
            tc_commit<1>(&sm.empty[vb % kRing]);
            tc_commit<1>(&sm.empty[(vb + 1) % kRing]);
          }
          if (ok && k < tiles && t < it.end[g]) {
            if (t == it.end[g] - 1) {
              ok = wait_or_abort(&sm.abort, &sm.qfull[g], nq[g] & 1u);
              ++nq[g];
            }
            for (int b = 0; ok && b < kKBlocks; ++b) {
              if (!waited_k) ok = landed(kb + b);
              if (!ok) break;
              tc_fence_after();
              const uint64_t qd = smem_desc_sw128(smem_u32(sm.q[g][b]), 16, 1024);
              const uint64_t kd = smem_desc_sw128(ring0 + ((kb + b) % kRing) * kBlock, 16, 1024);
#pragma unroll
              for (int s = 0; s < 4; ++s)
                mma_ss<1>(tmem + s_col(g), qd + s * 2, kd + s * 2, kIdS, (b > 0 || s > 0) ? 1u : 0u);
            }
            if (!ok) break;
            waited_k = true;
            tc_commit<1>(&sm.sfull[g]);
            if (t == it.t0) tc_commit<1>(&sm.qempty[g]);
          }
        }
        if (ok && k < tiles)
          for (int b = 0; b < kKBlocks; ++b) tc_commit<1>(&sm.empty[(kb + b) % kRing]);
      }
    }
    if (tiles > 0) seq += (uint32_t)tiles * kTileBlocks;
    ok = __shfl_sync(kFull, (int)ok, 0) != 0;
    if (!ok) break;
  }
  if (lane == 0) {
    if (!ok && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
    // Every product issued completes before the tensor memory is freed.
    tc_commit<1>(&sm.drain);
    if (!mbar_wait(&sm.drain, 0)) cta_abort(&sm.abort, a.flags);
  }
  __syncwarp();
}

// ---- warps 0-3 and 4-7: softmax and outputs of query tile g -------------------
template <bool BF16>
__device__ __forceinline__ void softmax_tiles(const PrefillArgs& a, PrefillSmem& sm, uint32_t tmem,
                                              int g, int blocks, int64_t items) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int r = quad * 32 + lane;            // this thread's row of the tile
  const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
  // A negative scale takes the scores' negatives, 0 their products with it, so
  // that a masked score is -inf under every scale.
  const float sign = a.c2 < 0.f ? -1.f : 0.f, c2 = a.c2 == 0.f ? 1.f : fabsf(a.c2);
  Cursor cur;
  uint32_t seq = 0, ns = 0, no = 0;          // ring blocks of earlier items; scores, outputs waited for
  bool ok = true;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item it = find_item(a, blocks, i, cur);
    const int row = it.row0 + g * kTileQ + r;
    const bool active = g * kTileQ + r < it.rows;
    const int seen = a.causal ? min(it.shift + g * kTileQ + r + 1, it.lk) : it.lk;
    float m = -INFINITY, l = 0.f;
    for (int t = it.end[g] - 1; t >= it.t0; --t) {
      ok = wait_or_abort(&sm.abort, &sm.sfull[g], ns & 1u);
      ++ns;
      if (!__all_sync(kFull, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t x[kTileK];
      tmem_load(trow + s_col(g), x);
      tmem_wait_ld(x);
      if (a.c2 <= 0.f) {
#pragma unroll
        for (int j = 0; j < kTileK; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * sign);
      }
      const int limit = seen - t * kTileK;   // keys of this tile that the row sees
      if (__any_sync(kFull, limit < kTileK)) {
#pragma unroll
        for (int j = 0; j < kTileK; ++j)
          if (j >= limit) x[j] = 0xff800000u;
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kTileK; j += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          m4[k] = fmaxf(fmaxf(m4[k], __uint_as_float(x[j + 2 * k])), __uint_as_float(x[j + 2 * k + 1]));
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
      const float mn = mx > m + kRescaleGap ? mx : m;   // m = -inf takes any finite maximum
      const float alpha = m == -INFINITY ? 1.f : fast_exp2(m - mn);
      const float ref = mn == -INFINITY ? 0.f : mn;
      m = mn;
      // The scores of tile t were issued after the values of tile t + 1: O is at rest.
      if (__any_sync(kFull, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < kDv; c += 32) {
          uint32_t o[32];
          tmem_load(trow + (uint32_t)(o_col(g) + c), o);
          tmem_wait_ld(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
          tmem_store(trow + (uint32_t)(o_col(g) + c), o);
        }
      }
      const float2 c2v = make_float2(c2, c2), nref = make_float2(-ref, -ref);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < kTileK; c += 32) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 e = ffma2(make_float2(__uint_as_float(x[c + 2 * j]),
                                             __uint_as_float(x[c + 2 * j + 1])), c2v, nref);
          const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
          p[j] = pack16<BF16>(e0, e1);
          sum[j & 1] = fadd2(sum[j & 1], make_float2(e0, e1));
        }
        tmem_store(trow + (uint32_t)(s_col(g) + c / 2), p);
      }
      l = l * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
      // Values behind the sequence's end (another's rows, or anything) count as
      // zeros, whatever they are: those that the last step of 16 keys reads.
      const int past = it.lk - t * kTileK, to = 16 * value_steps(a, it, g, t);
      if (past < to) {
        const uint32_t vb = seq + (uint32_t)(it.t1 - 1 - t) * kTileBlocks + kKBlocks;
        ok = wait_or_abort(&sm.abort, &sm.full[vb % kRing], (vb / kRing) & 1u) &&
             wait_or_abort(&sm.abort, &sm.full[(vb + 1) % kRing], ((vb + 1) / kRing) & 1u);
        if (!__all_sync(kFull, ok)) {
          ok = false;
          break;
        }
        for (int z = r; z < (to - past) * 16; z += kTileQ) {
          const int key = past + z / 16;
          uint8_t* blk = sm.ring[(vb + (uint32_t)(key >> 6)) % kRing] + (z & 8 ? kBlock / 2 : 0);
          *reinterpret_cast<uint4*>(blk + (key & 63) * 128 + (z & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();                  // before this warp hands its weights over
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.pfull[g]);
    }
    if (ok && it.end[g] > it.t0) {
      ok = wait_or_abort(&sm.abort, &sm.ofull[g], no & 1u);
      ++no;
    }
    if (!__all_sync(kFull, ok)) {
      ok = false;
      break;
    }
    seq += (uint32_t)(it.t1 - it.t0) * kTileBlocks;
    const int64_t to = (int64_t)row * a.H + it.head;
    const float lse = l == 0.f ? -INFINITY : m + log2f(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.splits > 1) {
      if (active) a.part_l[(int64_t)it.split * a.Tq * a.H + to] = lse;
    } else if (active) {
      a.lse2[to] = lse;
    }
    const bool some = it.end[g] > it.t0;
    if (some) tc_fence_after();
    if (!some && a.splits > 1) continue;     // the merge does not read this part
#pragma unroll 1
    for (int c = 0; c < kDv; c += 32) {
      uint32_t o[32];
      if (some) {
        tmem_load(trow + (uint32_t)(o_col(g) + c), o);
        tmem_wait_ld(o);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j)
        o[j] = some && l != 0.f ? __float_as_uint(__uint_as_float(o[j]) * inv) : 0u;
      if (active && a.splits > 1) {
        uint4* dst = reinterpret_cast<uint4*>(a.part_o + ((int64_t)it.split * a.Tq * a.H + to) * kDv + c);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
      } else if (active) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to * kDv + c);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t b[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            b[k] = pack16<BF16>(__uint_as_float(o[8 * v + 2 * k]), __uint_as_float(o[8 * v + 2 * k + 1]));
          dst[v] = make_uint4(b[0], b[1], b[2], b[3]);
        }
      }
      __syncwarp();                          // the next columns' load takes the whole warp
    }
  }
  if (!ok && lane == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_pe,
                       const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a) {
  extern __shared__ unsigned char prefill_smem_raw[];
  PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(
      (reinterpret_cast<uintptr_t>(prefill_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == kMmaWarp) {
    tmem_alloc<1>(&sm.tmem, kTmemCols);
  } else if (warp == kLoadWarp) {
    // Query blocks of all sequences; bad bounds are flagged once a call.
    const int lane = tid & 31;
    int blocks = 0;
    bool bad = false;
    for (int i = lane; i < a.n; i += 32) {
      int q0, q1, k0, k1;
      bounds_of(a.cu_q, i, a.Tq, q0, q1);
      bounds_of(a.cu_k, i, a.Tk, k0, k1);
      bad |= q0 != a.cu_q[i] || q1 != a.cu_q[i + 1] || k0 != a.cu_k[i] || k1 != a.cu_k[i + 1];
      blocks += (q1 - q0 + kBlockQ - 1) / kBlockQ;
    }
    blocks = __reduce_add_sync(kFull, blocks);
    if (bad && blockIdx.x == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
    if (lane == 0) sm.blocks = blocks;
  } else if (tid == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sm.qfull[g], 1);
      mbar_init(&sm.qempty[g], 1);
      mbar_init(&sm.sfull[g], 1);
      mbar_init(&sm.pfull[g], 4);
      mbar_init(&sm.ofull[g], 1);
    }
    for (int b = 0; b < kRing; ++b) {
      mbar_init(&sm.full[b], 1 + (b == 0 ? kStalledArrivals : 0));
      mbar_init(&sm.empty[b], 1);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int blocks = sm.blocks;
  const int64_t items = (int64_t)blocks * a.H * a.splits;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kLoadWarp) load_tiles(a, sm, &tm_q, &tm_k, &tm_pe, &tm_v, blocks, items);
    else if (warp == kMmaWarp) issue_products<BF16>(a, sm, tmem, blocks, items);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_tiles<BF16>(a, sm, tmem, warp >> 2, blocks, items);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free<1>(tmem, kTmemCols);
  }
}

// Parts that an item's keys are split into: as many as SMs are left idle
// otherwise, but eight key tiles each at least.
int splits_for(int Tq, int Tk, int n, int H) {
  const int64_t items = ((int64_t)Tq / kBlockQ + n) * H;
  const int64_t most = std::min<int64_t>(device_sms() / std::max<int64_t>(items, 1), Tk / (8 * kTileK));
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, 16));
}

bool strides_fit(int64_t token, int64_t head, int T, int H, int width) {
  return (T <= 1 || (token >= 1 && token % 8 == 0)) && (H <= 1 || (head >= width && head % 8 == 0)) &&
         token < ((int64_t)1 << 38) && head < ((int64_t)1 << 38);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int64_t dsa_mla_prefill_work(int Tq, int Tk, int n, int H) {
  if (Tq < 1 || Tk < 1 || n < 1 || H < 1) return 0;
  const int parts = splits_for(Tq, Tk, n, H);
  return parts == 1 ? 0 : (int64_t)parts * Tq * H * (kDv + 1) * 4;
}

extern "C" dsa_status dsa_mla_prefill(const void* q, int64_t q_token, int64_t q_head,
                                      const void* k_nope, int64_t k_token, int64_t k_head,
                                      const void* k_pe, int64_t pe_token, const void* v,
                                      int64_t v_token, int64_t v_head, const int32_t* cu_q,
                                      const int32_t* cu_k, int n, int Tq, int Tk, int H, int dtype,
                                      float scale, int causal, void* out, float* lse2, float* work,
                                      uint32_t* err_flags, cudaStream_t stream) {
  if (n < 0 || Tq < 0 || Tk < 0 || H < 1 || !(scale == scale) || isinf(scale))
    return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_FP16) return DSA_ERR_INVALID_ARG;
  if (n == 0 || Tq == 0) return DSA_OK;
  if (!q || !cu_q || !cu_k || !out || !lse2 || (Tk > 0 && (!k_nope || !k_pe || !v)))
    return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(work) || (Tk > 0 && (!aligned16(k_nope) ||
      !aligned16(k_pe) || !aligned16(v))))
    return DSA_ERR_INVALID_ARG;
  if (!strides_fit(q_token, q_head, Tq, H, kDn + kDr) || !strides_fit(k_token, k_head, Tk, H, kDn) ||
      !strides_fit(pe_token, kDr, Tk, 1, kDr) || !strides_fit(v_token, v_head, Tk, H, kDv))
    return DSA_ERR_INVALID_ARG;
  if (((int64_t)Tq / kBlockQ + n) * H > ((int64_t)1 << 26)) return DSA_ERR_UNSUPPORTED;
  const bool bf16 = dtype == DSA_BF16;
  if (Tk == 0) k_nope = k_pe = v = q;        // never read
  // A dimension of one row has no stride of its own.
  auto map = [&](CUtensorMap* m, const void* p, int width, int heads, int T, int64_t token,
                 int64_t head, uint32_t rows) {
    const uint64_t hs = heads > 1 ? (uint64_t)head * 2 : (uint64_t)width * 2;
    const uint64_t ts = T > 1 ? (uint64_t)token * 2 : hs * heads;
    return encode_map16(m, p, bf16, width, heads, std::max(T, 1), hs, ts, 1, rows);
  };
  CUtensorMap tm_q, tm_k, tm_pe, tm_v;
  if (!map(&tm_q, q, kDn + kDr, H, Tq, q_token, q_head, kTileQ) ||
      !map(&tm_k, k_nope, kDn, H, Tk, k_token, k_head, kTileK) ||
      !encode_map16(&tm_pe, k_pe, bf16, kDr, std::max(Tk, 1), 1, (uint64_t)(Tk > 1 ? pe_token : kDr) * 2,
                    (uint64_t)(Tk > 1 ? pe_token : kDr) * 2 * std::max(Tk, 1), kTileK, 1) ||
      !map(&tm_v, v, kDv, H, Tk, v_token, v_head, 64))
    return DSA_ERR_CUDA;
  const int smem = (int)sizeof(PrefillSmem) + 1024;
  const auto kernel = bf16 ? mla_prefill_kernel<true> : mla_prefill_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const int splits = work ? splits_for(Tq, Tk, n, H) : 1;
  // Heads whose keys and values (512 bytes a token and head) fit half of L2.
  const int64_t fit = ((int64_t)48 << 20) / (512 * (int64_t)std::max(Tk, 1));
  PrefillArgs a{cu_q, cu_k, out, lse2, nullptr, nullptr, err_flags, n, Tq, Tk, H,
                (int)std::max<int64_t>(1, std::min<int64_t>(fit, H)), splits, causal != 0,
                scale * kLog2e};
  if (splits > 1) {
    a.part_o = work;
    a.part_l = work + (int64_t)splits * Tq * H * kDv;
  }
  const int64_t most = ((int64_t)Tq / kBlockQ + n) * H * splits;
  const unsigned grid = (unsigned)std::min<int64_t>(most, device_sms());
  if (launch_kernel(kernel, dim3(grid), dim3(kThreads), (size_t)smem, stream, 0, tm_q, tm_k, tm_pe,
                    tm_v, a) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (splits > 1) {
    const MergeArgs m{a.part_o, a.part_l, splits, (int64_t)Tq * H, cu_q, n, Tq, H, out, lse2};
    const cudaError_t e = bf16 ? launch_merge<kDv, true>(m, stream) : launch_merge<kDv, false>(m, stream);
    if (e != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}
