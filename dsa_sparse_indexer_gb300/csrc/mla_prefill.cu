// Latent attention in its expanded form over a ragged batch (sm_103a).
//
// Per query i of a sequence and head h, over its visible keys j: x_j = scale *
// (q_i[0..128) . k_nope_j + q_i[128..192) . k_pe_j), k_pe shared by all heads,
// out = sum_j 2^(x_j log2 e) v_j / sum_j 2^(x_j log2 e) and lse2 = log2 sum_j
// exp(x_j), so that outputs over parts of a context are merged as a shard's are.
//
// Compute-bound: 640 operations a visible (query, key) pair, and the exponent
// of each.  An item is a head's block of 256 queries (or a part of its keys), or,
// where sequences are longer than that, of 512 for a pair of CTAs that issues one
// product of M = 256 and either of which copies half of a tile's keys and values.
// A CTA holds two tiles of 128 queries, so that one's softmax runs under the
// other's products.  Keys go in tiles of 128, the last first: the masked ones.
// Scores' and values' products have N = 128, the smallest N that runs at the full
// rate (64 cycles a step of 16): 2560 cycles a key tile and CTA.
//  * tensor memory: two score tiles (128 columns each; the weights take the
//    first half of the same columns as 16-bit pairs) and two outputs (128 each);
//  * shared memory: the queries (96 KB) and a ring of 120 KB: a tile's keys as
//    three blocks of 64 values, its values as two of 64 keys, freed as units;
//  * one warp claims items while the kernel runs, one copies (tensor maps,
//    128-byte swizzle), one a query tile issues its products, eight a query tile
//    run its softmax: maximum, weights relative to a reference that moves when
//    exceeded by 2^8, their sum, the outputs.
// The weights' sum is of the fp32 weights; a weight enters the value product
// rounded to 16 bits: by 2^-8 of itself at most in bf16; in fp16, whose weights are
// 2^7 larger so that few are subnormal, by 2^-11 of itself or 2^-32 of the
// reference's weight.  That is 1 or 2^7, and exact.
// Every wait is bounded and raises DSA_FLAG_TIMEOUT when it runs out.
// Measured, one sequence of 8192, 128 heads, causal: 1740 us after a pause (2070 MHz),
// 1.58 PFLOP/s of the 1.96 that a library product reaches, 1840 to 1900 one after
// another at the power limit (1867 to 1912 MHz); 3753 with one CTA an item, a warp
// issuing for both query tiles and a thread a row in the softmax.  16 heads, 500
// queries of 16384 keys: 80 us, 1.03 PFLOP/s, its keys in parts.
#include <algorithm>

#include "regions.h"
#include "split_merge.cuh"

namespace dsa {
namespace {

constexpr int kDn = DSA_MLA_DN, kDr = DSA_MLA_DR, kDv = DSA_MLA_DVH;
constexpr int kTileQ = 128;                         // queries of a CTA's tile
constexpr int kTileK = 128;                         // keys of a tile
constexpr int kQBlock = 16384;                      // bytes of 128 queries' 64 values
constexpr int kQBlocks = (kDn + kDr) / 64;          // 3
constexpr int kKBlocks = kQBlocks, kVBlocks = 2, kTileBlocks = kKBlocks + kVBlocks;
constexpr int kVKeys = kTileK / kVBlocks;
constexpr int kRingBytes = 122880;
constexpr int kUnits = 8;                           // barriers of the ring: a tile's keys or values each
// Warps: 16 of the softmax (g * 8 + sub * 4 + quad: query tile g, rows quad * 32 +
// sub * 16 to + 15), two issuing products, one copying, one claiming.
constexpr int kSoftmaxWarps = 16, kMmaWarp = 16, kLoadWarp = 18, kClaimWarp = 19;
constexpr int kThreads = 640;
// Registers: 96 a thread at launch; the four softmax warpgroups take 104, the
// fifth keeps 64 of them: 4 x 104 + 64 = 5 x 96.
constexpr int kTmemCols = 512;
__device__ __forceinline__ constexpr int s_col(int g) { return g * 128; }
__device__ __forceinline__ constexpr int o_col(int g) { return 256 + g * 128; }

template <int CG>
struct Shape {
  static constexpr int kGroup = CG * kTileQ;        // queries of one product
  static constexpr int kBlockQ = 2 * kGroup;        // of an item
  static constexpr int kKeys = kTileK / CG;         // keys of a tile that a CTA holds
  static constexpr int kBlock = kKeys * 128;        // bytes of a ring block
  static constexpr int kRing = kRingBytes / kBlock; // 7 or 15
  static constexpr int kAtoms = kDv / CG / 64;      // 64-value columns of its values
  static constexpr int kAtom = kVKeys * 128;        // bytes of one in a value block
  static_assert(kRing <= kUnits / 2 * kTileBlocks, "a unit's barriers are not used twice in the ring");
  static_assert(kAtoms * kAtom == kBlock, "value blocks are as large as key blocks");
};
#ifdef DSA_TEST_STALLED_COPY
// The test-only build (never libdsa.so): the first key block's barrier expects
// one arrival that nothing makes (its copy still lands).
constexpr uint32_t kStalledArrivals = 1;
#else
constexpr uint32_t kStalledArrivals = 0;
#endif

// What an item is.
struct Item {
  int head, split;
  int row0, rows;             // its queries: first row, how many
  int key0, lk;               // its sequence's keys
  int shift;                  // causal: row r of the block sees shift + r + 1 keys
  int t0, t1;                 // its key tiles
  int end[2];                 // each query tile's: [t0, end)
};

struct alignas(1024) PrefillSmem {
  uint8_t q[2][kQBlocks][kQBlock];
  uint8_t ring[kRingBytes];
  WorkSlots<Item> work;
  uint64_t qfull[2], qempty[2], full[kUnits], empty[kUnits], sfull[2], phalf[2], pfull[2], ofull[2], vtail[2],
      drain[2];
  Order order;
  uint32_t tmem;
  int blocks;                                // query blocks of all sequences
  int bad;                                   // cu_q or cu_k is not ascending inside its rows
  int abort;
};
static_assert(sizeof(PrefillSmem) + 1024 <= 232448, "shared memory of a CTA");

struct PrefillArgs {
  const int32_t *cu_q, *cu_k; // [n + 1]
  void* out;                  // [Tq][H][kDv]
  float* lse2;                // [Tq][H]
  float *part_o, *part_l;     // [splits][Tq][H][kDv], [splits][Tq][H]
  uint32_t* flags;
  int n, Tq, Tk, H, group, splits, causal, ordered;   // items in the sequences' order by length
  // |scale| log2(e), and the score product's descriptor bit that negates A for a
  // negative scale.  A scale of 0 is taken as 2^-100: finite scores then count
  // alike, masked ones are -inf as ever.
  float c2;
  uint32_t negate;
};

__device__ __forceinline__ int end_of(const Item& it, int g) { return g == 0 ? it.end[0] : it.end[1]; }

struct Cursor {               // where the last item's sequence was found
  int seq = 0, before = 0;    // its place in the order, query blocks before it
};

// Warp-wide: item `index` of a.H * blocks * splits.  Heads go in groups whose
// keys and values stay in L2 together; within one, a sequence's longest blocks
// (its last) come first, so that the CTAs, which claim items, end alike.
template <int CG>
__device__ __forceinline__ Item find_item(const PrefillArgs& a, const Order& order, int blocks, bool bad,
                                          int64_t index, Cursor& c) {
  constexpr int kGroup = Shape<CG>::kGroup, kBlockQ = Shape<CG>::kBlockQ;
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
    if (i < a.n) bounds_of(a.cu_q, in_order(order, a.ordered, i), a.Tq, bad, first, end);
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
  const int seq = in_order(order, a.ordered, c.seq);
  bounds_of(a.cu_q, seq, a.Tq, bad, q0, q1);
  bounds_of(a.cu_k, seq, a.Tk, bad, k0, k1);
  const int at = (nb - 1 - local) * kBlockQ;
  it.row0 = q0 + at;
  it.rows = min(kBlockQ, q1 - it.row0);
  it.key0 = k0;
  it.lk = k1 - k0;
  it.shift = it.lk - (q1 - q0) + at;
  int nt = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int r = min(max(it.rows - g * kGroup, 0), kGroup);
    const int seen = r == 0 ? 0 : !a.causal ? it.lk : min(max(it.shift + g * kGroup + r, 0), it.lk);
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
template <int CG>
__device__ __forceinline__ int value_steps(const PrefillArgs& a, const Item& it, int g, int t) {
  constexpr int kGroup = Shape<CG>::kGroup;
  int keys = min(it.lk - t * kTileK, kTileK);
  if (a.causal) {
    const int r = min(it.rows - g * kGroup, kGroup);
    keys = min(keys, it.shift + g * kGroup + r - t * kTileK);
  }
  return (keys + 15) / 16;
}
// Whether a step may read values behind the sequence's end: the softmax warps
// zero these in shared memory.
__device__ __forceinline__ bool has_tail(int lk, int t) {
  return lk - t * kTileK < kTileK && (lk & 15) != 0;
}

// ---- the copying warp ------------------------------------------------------
// Of a pair, either CTA copies its own queries, half of a tile's keys and half of
// its values' columns; the first CTA's barriers count both's bytes.
template <int CG>
__device__ __forceinline__ void load_tiles(const PrefillArgs& a, PrefillSmem& sm,
                                           const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                           const CUtensorMap* tm_pe, const CUtensorMap* tm_v,
                                           uint32_t rank) {
  using Sh = Shape<CG>;
  const int lane = threadIdx.x & 31;
  Item it;
  bool half_tile = false;                    // the last tile's values were not copied
  uint32_t tile = 0, loads[2] = {0, 0}, tails = 0;   // key tiles, query tiles, tails copied so far
  bool ok = true;
  // Ring block b is block b % kTileBlocks of tile b / kTileBlocks; unit 2 t is tile
  // t's keys, 2 t + 1 its values.  Units are copied and freed in this order:
  // blocks up to `end` fit once the unit of block end - 1 - kRing is free.  The
  // barrier of unit u then expects its bytes (or, values with a tail, an arrival
  // alone: they are counted elsewhere).
  auto open_unit = [&](uint32_t u, uint32_t end, uint32_t bytes) {
    if (end > Sh::kRing) {
      const uint32_t b = end - 1 - Sh::kRing;
      const uint32_t v = b / kTileBlocks * 2 + (b % kTileBlocks >= kKBlocks ? 1u : 0u);
      ok = wait_or_abort(&sm.abort, &sm.empty[v % kUnits], (v / kUnits) & 1u);
    }
    if (ok && rank == 0) {
      if (bytes) mbar_expect_tx(&sm.full[u % kUnits], CG * bytes);
      else mbar_arrive1(&sm.full[u % kUnits]);
    }
    return ok;
  };
  auto bar_of = [&](uint64_t* bar) { return CG == 1 ? smem_u32(bar) : leader_addr(bar); };
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok, it); ++n) {
    item_done(sm.work, n);
    if (lane == 0) {
      for (int t = it.t1 - 1; ok && t >= it.t0; --t) {
#pragma unroll 1
        for (int g = 0; ok && g < 2; ++g) {
          if (t != end_of(it, g) - 1) continue;  // the tile's first key tile: its queries
          if (loads[g] > 0) ok = wait_or_abort(&sm.abort, &sm.qempty[g], (loads[g] - 1) & 1u);
          if (!ok) break;
          if (rank == 0) mbar_expect_tx(&sm.qfull[g], CG * kQBlocks * kQBlock);
#pragma unroll 1
          for (int b = 0; b < kQBlocks; ++b)
            load_box<CG>(sm.q[g][b], tm_q, b * 64, it.head,
                         it.row0 + g * Sh::kGroup + (int)rank * kTileQ, bar_of(&sm.qfull[g]));
          ++loads[g];
        }
        const int key = it.key0 + t * kTileK;
        const uint32_t b0 = tile * kTileBlocks;
        auto block = [&](uint32_t b) { return sm.ring + (b0 + b) % Sh::kRing * Sh::kBlock; };
        if (!open_unit(2 * tile, b0 + kKBlocks, kKBlocks * Sh::kBlock)) break;
        const uint32_t kbar = bar_of(&sm.full[2 * tile % kUnits]);
        const int mine = key + (int)rank * Sh::kKeys;
        for (int b = 0; b < kDn / 64; ++b) load_box<CG>(block(b), tm_k, b * 64, it.head, mine, kbar);
        load_box<CG>(block(kKBlocks - 1), tm_pe, 0, mine, 0, kbar);
        const bool tail = has_tail(it.lk, t);
        uint64_t* vtail = &sm.vtail[tails & 1u];
        if (!open_unit(2 * tile + 1, b0 + kTileBlocks, tail ? 0 : kVBlocks * Sh::kBlock)) {
          ++tile;
          half_tile = true;
          break;
        }
        if (tail) {
          mbar_expect_tx(vtail, kVBlocks * Sh::kBlock);
          ++tails;
        }
        const uint32_t vbar = tail ? smem_u32(vtail) : bar_of(&sm.full[(2 * tile + 1) % kUnits]);
        for (int b = 0; b < kVBlocks; ++b)
          for (int c = 0; c < Sh::kAtoms; ++c)
            load_box<CG>(block(kKBlocks + b) + c * Sh::kAtom, tm_v, ((int)rank * Sh::kAtoms + c) * 64,
                         it.head, key + b * kVKeys, vbar);
        ++tile;
      }
    }
    ok = __shfl_sync(kFull, (int)ok, 0) != 0;
  }
  if (lane == 0 && !ok) {
    if (!cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
    // Every copy issued lands before the CTA ends (a pair's first CTA counts both's).
    if (rank == 0) {
      for (int g = 0; g < 2; ++g)
        if (loads[g] > 0) mbar_wait(&sm.qfull[g], (loads[g] - 1) & 1u);
      const uint32_t units = 2 * tile - (half_tile ? 1 : 0);
      for (uint32_t u = units > kUnits ? units - kUnits : 0; u < units; ++u)
        mbar_wait(&sm.full[u % kUnits], (u / kUnits) & 1u);
    }
    for (uint32_t k = tails > 2 ? tails - 2 : 0; k < tails; ++k)
      mbar_wait(&sm.vtail[k & 1u], (k >> 1) & 1u);
  }
  // The products' arrivals come to both CTAs of a pair: the second, which waits for few
  // of them, sees the last before it ends.
  if (CG == 2 && rank == 1) {
    wait_landed(&sm.drain[0], 0);
    wait_landed(&sm.drain[1], 0);
  }
  __syncwarp();
}

// ---- the issuing warps: the products of query tile 0 and 1 --------------------------
// A warp runs along converged and one elected lane issues (inside a branch of one
// lane the descriptors could not stay in uniform registers).  One for each query
// tile: a wait that is over already still costs about 100 cycles, an arrival as
// much, and in one warp either query tile's delay the other's products.
template <int CG, bool BF16>
__device__ __forceinline__ void issue_products(const PrefillArgs& a, PrefillSmem& sm, uint32_t tmem,
                                               int g) {
  using Sh = Shape<CG>;
  constexpr uint32_t kRing = Sh::kRing;
  const uint32_t id_s = idesc_f16(CG * kTileQ, kTileK, BF16, false) | a.negate;
  constexpr uint32_t id_o = idesc_f16(CG * kTileQ, kDv, BF16, true);
  constexpr int kStep = Sh::kBlock >> 4;     // a block in a descriptor's address field
  const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q[g][0]), 16, 1024);
  const uint64_t k0 = smem_desc_sw128(smem_u32(sm.ring), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(smem_u32(sm.ring), Sh::kAtom, 1024);
  const uint32_t d_s = tmem + s_col(g), d_o = tmem + o_col(g);
  Item it;
  uint32_t tk = 0, np = 0, nq = 0;           // tiles, weights and query tiles so far
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && warp_wait(&sm.abort, bar, parity);
    return ok;
  };
  auto landed = [&](uint32_t u) { return wait(&sm.full[u % kUnits], (u / kUnits) & 1u); };
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok, it); ++n) {
    item_done(sm.work, n);
    const int end = end_of(it, g);
    if (it.t1 == it.t0) continue;
    for (int t = it.t1 - 1; ok && t >= it.t0 - 1; --t, ++tk) {   // scores of tile t, values of t + 1
      const uint32_t kb = tk * kTileBlocks, vb = kb - kTileBlocks + kKBlocks;
      const bool values = t < it.t1 - 1, scores = t >= it.t0;
      // Copies are waited for ahead of the weights, and used or not: a unit freed
      // before it is there would count for the next one of its barriers.
      if (values && !landed(2 * tk - 1)) break;
      if (scores && !landed(2 * tk)) break;
      if (scores && t == end - 1) {
        if (!wait(&sm.qfull[g], nq & 1u)) break;
        ++nq;
      }
      const bool my_values = values && t + 1 < end, my_scores = scores && t < end;
      const int steps = my_values ? value_steps<CG>(a, it, g, t + 1) : 0;
      const uint32_t more = t + 1 < end - 1 ? 1u : 0u;   // not the item's first
      auto value_products = [&](int b) {
        const uint64_t vd = v0 + ((vb + b) % kRing) * kStep;
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (b * 4 + s < steps)
            mma_ts<CG>(d_o, d_s + b * 32 + s * 8, vd + s * (2048 >> 4), id_o, s > 0 || b > 0 ? 1u : more);
      };
      if (my_values) {                       // the first 64 keys' weights, then the others'
        if (!wait(&sm.phalf[g], np & 1u)) break;
        tc_fence_after();
        if (elect_one()) value_products(0);
        __syncwarp();
        if (!wait(&sm.pfull[g], np & 1u)) break;
        ++np;
      }
      tc_fence_after();
      if (elect_one()) {
        if (my_values) value_products(1);
        if (my_scores) {
#pragma unroll
          for (int b = 0; b < kKBlocks; ++b) {
            const uint64_t qd = q0 + b * (kQBlock >> 4), kd = k0 + ((kb + b) % kRing) * kStep;
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_ss<CG>(d_s, qd + s * 2, kd + s * 2, id_s, (b > 0 || s > 0) ? 1u : 0u);
          }
          tc_commit<CG>(&sm.sfull[g]);
          if (t == it.t0) tc_commit<CG>(&sm.qempty[g]);
        } else if (my_values && !scores) {
          tc_commit<CG>(&sm.ofull[g]);       // the output is complete
        }
        if (values) tc_commit<CG>(&sm.empty[(2 * tk - 1) % kUnits]);
        if (scores) tc_commit<CG>(&sm.empty[2 * tk % kUnits]);
      }
      __syncwarp();
      if (!scores) break;
    }
  }
  const int lane = threadIdx.x & 31;
  if (!ok && lane == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
  __syncwarp();
  // Every product issued completes before the tensor memory is freed (a commit
  // counts the thread's own: elect_one picks the same lane every time).
  if (elect_one()) {
    tc_commit<CG>(&sm.drain[g]);
    if (!mbar_wait(&sm.drain[g], 0)) cta_abort(&sm.abort, a.flags);
  }
  __syncwarp();
}

// ---- warps 0-15: softmax and outputs -------------------------------------------
// A warp has 16 rows of query tile g, four lanes a row and two rows a lane (tensor
// memory's fragments): twice the warps of a thread a row, so that the chain scores -
// weights - value product, which a tile waits for, is half as long, and a row's
// maximum still needs no more than shuffles.
// In binades: weights go up to kRescaleGap above the reference's (fp16: 2^15 of 65504).
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

template <int CG, bool BF16>
__device__ __forceinline__ void softmax_tiles(const PrefillArgs& a, PrefillSmem& sm, uint32_t tmem,
                                              int warp, uint32_t rank) {
  using Sh = Shape<CG>;
  const int lane = threadIdx.x & 31;
  const int g = warp >> 3, sub = (warp >> 2) & 1, quad = warp & 3;
  const int r0 = quad * 32 + sub * 16;       // the warp's first row of the CTA's tile
  const int br = g * Sh::kGroup + (int)rank * kTileQ + r0 + (lane >> 2);   // the lane's rows of the item's
  const int col = 2 * (lane & 3);            // block: br and br + 8; its first of 8 columns
  const uint32_t trow = tmem + ((uint32_t)r0 << 16);
  const uint32_t t_s = trow + s_col(g), t_o = trow + o_col(g);
  auto hand_over = [&](uint64_t* bar) {      // this warp's weights
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if constexpr (CG == 1) mbar_arrive1(bar);
      else mbar_arrive_leader(bar);
    }
  };
  // Over the four lanes of a row.
  auto row_max = [](float v) {
    v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
    return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
  };
  auto row_sum = [](float v) {
    v += __shfl_xor_sync(kFull, v, 1);
    return v + __shfl_xor_sync(kFull, v, 2);
  };
  uint32_t tile = 0, ns = 0, no = 0, tails = 0;   // tiles of earlier items; scores, outputs, tails so far
  bool ok = true;
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok); ++n) {
    // Read where it lies, so that a tile's registers are the scores'.
    const Item& it = sm.work.item[n & 1u];
    const int end = uni(end_of(it, g)), t0 = uni(it.t0), lk = uni(it.lk);
    const int seen = a.causal ? it.shift + br + 1 : lk;   // by the first row (causal: 8 more by the second)
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // references (less the lift), sums
    for (int t = end - 1; t >= t0; --t, ++ns) {
      ok = warp_wait(&sm.abort, &sm.sfull[g], ns & 1u);
      if (!ok) break;
      tc_fence_after();
      // Of this tile's keys from the lane's first column on, so many are seen.
      const int lim0 = min(seen, lk) - t * kTileK - col;
      const int lim1 = min(seen + (a.causal ? 8 : 0), lk) - t * kTileK - col;
      const bool masked = __any_sync(kFull, lim0 + col < kTileK);
      // Scores are read twice, 32 columns at a time, for the maximum and for the
      // weights: all of them at once leave too few registers.
      auto mask = [&](uint32_t (&x)[16], int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = c * 32 + i * 8;
          if (j >= lim0) x[4 * i] = 0xff800000u;
          if (j + 1 >= lim0) x[4 * i + 1] = 0xff800000u;
          if (j >= lim1) x[4 * i + 2] = 0xff800000u;
          if (j + 1 >= lim1) x[4 * i + 3] = 0xff800000u;
        }
      };
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        uint32_t x[2][16];
        tmem_load_frag(t_s + c * 32, x[0]);
        tmem_load_frag(t_s + c * 32 + 32, x[1]);
        tmem_wait_ld(x[0]);
        tmem_wait_ld(x[1]);
        if (masked) {
          keep_branch();
          mask(x[0], c);
          mask(x[1], c + 1);
          tmem_store_frag(t_s + c * 32, x[0]);   // as the weights will read them
          tmem_store_frag(t_s + c * 32 + 32, x[1]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {        // the lane's rows
          float v[2] = {top[k], -INFINITY};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              v[h] = fmax3(v[h], __uint_as_float(x[h][4 * i + 2 * k]), __uint_as_float(x[h][4 * i + 2 * k + 1]));
          top[k] = fmaxf(v[0], v[1]);
        }
      }
      float alpha[2];
      float2 nref[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mx = row_max(top[k]) * a.c2;
        // m = -inf takes any finite maximum.
        const float mn = mx > m[k] + (kRescaleGap + kLift<BF16>) ? mx - kLift<BF16> : m[k];
        alpha[k] = m[k] == -INFINITY ? 1.f : fast_exp2(m[k] - mn);
        const float ref = mn == -INFINITY ? 0.f : mn;
        nref[k] = make_float2(-ref, -ref);
        m[k] = mn;
        l[k] *= alpha[k];
      }
      // The scores of tile t were issued after the values of tile t + 1: O is at rest.
      if (__any_sync(kFull, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < kDv; c += 32) {
          uint32_t o[16];
          tmem_load_frag(t_o + (uint32_t)c, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[(j >> 1) & 1]);
          tmem_store_frag(t_o + (uint32_t)c, o);
        }
      }
      if (has_tail(lk, t)) {                 // values behind the sequence's end: zeros
        ok = warp_wait(&sm.abort, &sm.vtail[tails & 1u], (tails >> 1) & 1u);
        if (!ok) break;
        const uint32_t vb = (tile + (uint32_t)(it.t1 - 1 - t)) * kTileBlocks + kKBlocks;
        const int past = lk - t * kTileK, to = 16 * value_steps<CG>(a, it, g, t);
        for (int z = (warp & 7) * 32 + lane; z < (to - past) * Sh::kAtoms * 8; z += 256) {
          const int key = past + z / (Sh::kAtoms * 8), chunk = z % (Sh::kAtoms * 8);
          uint8_t* blk = sm.ring + ((vb + (uint32_t)(key / kVKeys)) % Sh::kRing) * Sh::kBlock;
          *reinterpret_cast<uint4*>(blk + (chunk >> 3) * Sh::kAtom + (key % kVKeys) * 128 + (chunk & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_for_products<CG>();            // before this warp hands its weights over
      }
      const float2 c2v = make_float2(a.c2, a.c2);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t y[2][16];
      if (masked) tmem_wait_st();
      tmem_load_frag(t_s, y[0]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t (&x)[16] = y[c & 1];
        tmem_wait_ld(x);
        if (c < 3) tmem_load_frag(t_s + (c + 1) * 32, y[(c + 1) & 1]);   // before weights overwrite it
        uint32_t p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 e = ffma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])),
                                 c2v, nref[j & 1]);
          const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
          p[j] = pack16<BF16>(e0, e1);
          sum[j & 1] = fadd2(sum[j & 1], make_float2(e0, e1));
        }
        tmem_store_pairs(t_s + c * 16, p);
        if (c == 1) hand_over(&sm.phalf[g]);
      }
      hand_over(&sm.pfull[g]);
#pragma unroll
      for (int k = 0; k < 2; ++k) l[k] += sum[k].x + sum[k].y;
    }
    if (it.t1 > t0) tails += has_tail(lk, it.t1 - 1);
    tile += (uint32_t)(it.t1 - t0);
    const bool some = end > t0;
    if (ok && some) {
      ok = warp_wait(&sm.abort, &sm.ofull[g], no & 1u);
      ++no;
    }
    if (!ok) break;
    if (some) tc_fence_after();
    const bool parts = a.splits > 1;
    const int64_t all = (int64_t)a.Tq * a.H;
    const int64_t to = (int64_t)(it.row0 + br) * a.H + it.head + (parts ? it.split * all : 0);
    const int64_t next = 8 * (int64_t)a.H;   // the second row
    bool active[2];
    float inv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      l[k] = row_sum(l[k]);
      active[k] = br + 8 * k < it.rows;
      inv[k] = l[k] == 0.f ? 0.f : 1.f / l[k];
      if (active[k] && (lane & 3) == 0)
        (parts ? a.part_l : a.lse2)[to + k * next] = l[k] == 0.f ? -INFINITY : m[k] + log2f(l[k]);
    }
    if (some || !parts) {                    // the merge does not read an empty part
      // Rows that saw nothing are zeros, whatever their columns hold.
      const bool seen_all = some && __all_sync(kFull, l[0] != 0.f && l[1] != 0.f);
      uint32_t y[2][16];
      if (some) tmem_load_frag(t_o, y[0]);
#pragma unroll
      for (int c = 0; c < kDv; c += 32) {
        uint32_t (&o)[16] = y[c / 32 & 1];
        if (some) {
          tmem_wait_ld(o);
          if (c + 32 < kDv) tmem_load_frag(t_o + (uint32_t)c + 32, y[(c / 32 + 1) & 1]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv[(j >> 1) & 1]);
        if (!seen_all) {
          keep_branch();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (!some || l[(j >> 1) & 1] == 0.f) o[j] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (parts) {
            if (active[k]) {
              float* dst = a.part_o + (to + k * next) * kDv + c + col;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint2*>(dst + 8 * i) = make_uint2(o[4 * i + 2 * k], o[4 * i + 2 * k + 1]);
            }
          } else {
            store_row<BF16>(o, k, lane, active[k], static_cast<uint16_t*>(a.out) + (to + k * next) * kDv + c);
          }
        }
        __syncwarp();                        // the next columns' load takes the whole warp
      }
    }
    item_done(sm.work, n);
  }
  if (!ok && lane == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
}

template <int CG, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_pe,
                       const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a) {
  using Sh = Shape<CG>;
  extern __shared__ unsigned char prefill_smem_raw[];
  PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(
      (reinterpret_cast<uintptr_t>(prefill_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = uni(tid >> 5);
  const uint32_t rank = CG == 2 ? pair_rank() : 0u;
  if (warp == kMmaWarp) {
    tmem_alloc<CG>(&sm.tmem, kTmemCols);
  } else if (warp == kClaimWarp) {
    bool bad;
    const int blocks = count_blocks(a.cu_q, a.Tq, a.cu_k, a.Tk, a.n, 1, Sh::kBlockQ, a.flags, bad);
    if ((tid & 31) == 0) sm.blocks = blocks, sm.bad = bad;
  } else if (tid == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sm.qfull[g], 1);
      mbar_init(&sm.qempty[g], 1);
      mbar_init(&sm.sfull[g], 1);
      mbar_init(&sm.phalf[g], 8 * CG);       // a warp each, of both CTAs in a pair's first
      mbar_init(&sm.pfull[g], 8 * CG);
      mbar_init(&sm.ofull[g], 1);
      mbar_init(&sm.vtail[g], 1);
      mbar_init(&sm.drain[g], 1);
    }
    for (int b = 0; b < kUnits; ++b) {
      mbar_init(&sm.full[b], 1 + (b == 0 ? kStalledArrivals : 0));
      mbar_init(&sm.empty[b], 2);            // both query tiles' products
    }
    init_slots(sm.work, CG, kSoftmaxWarps + 1 + (rank == 0 ? 2 : 0));
    sm.abort = 0;
    mbar_init_fence();
  }
  if (a.ordered)
    longest_first(sm.order, a.n, tid, [&](int i) { return __ldg(a.cu_k + i + 1) - __ldg(a.cu_k + i); });
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) pair_sync();        // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = uni(sm.tmem);
  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kLoadWarp) {
      load_tiles<CG>(a, sm, &tm_q, &tm_k, &tm_pe, &tm_v, rank);
    } else if (warp == kClaimWarp) {
      const int blocks = sm.blocks;
      const bool bad = sm.bad != 0;
      Cursor cur;
      share_out<CG>(sm.work, &sm.abort, a.flags, (int64_t)blocks * a.H * a.splits, rank,
                    [&](int64_t i) { return find_item<CG>(a, sm.order, blocks, bad, i, cur); });
    } else if (rank == 0) {
      issue_products<CG, BF16>(a, sm, tmem, warp - kMmaWarp);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    softmax_tiles<CG, BF16>(a, sm, tmem, warp, rank);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) pair_sync();        // neither CTA's memory goes while the other uses it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free<CG>(tmem, kTmemCols);
  }
}

constexpr int kSmem = (int)sizeof(PrefillSmem) + 1024;

// How a call is cut: CTAs that share a product, parts of the keys.
// Pairs against single CTAs, in us: one sequence of 8192 queries, 128 heads 1712 /
// 2214; 4096, 32 heads 281 / 358; 2048, 128 heads 167 / 204; eight of 1024, 32 heads
// 127 / 132; 16 of 512 (just a pair's item) 91 / 88.
// Bounds are the device's: means stand for them, in which empty sequences count.  A
// chunk of 500 queries of 16384 keys, 16 heads, is cut for 78 us alone; in a batch of
// eight or more whose others are empty, as single CTAs without parts, for 333.
struct Plan {
  int cg, splits, ordered;
};
Plan plan_for(int Tq, int Tk, int n, int H) {
  Plan p;
  p.cg = (int64_t)Tq > (int64_t)n * Shape<1>::kBlockQ ? 2 : 1;   // sequences longer than a CTA's block
  const int block = p.cg == 2 ? Shape<2>::kBlockQ : Shape<1>::kBlockQ;
  const int64_t items = std::max<int64_t>(((int64_t)Tq + block - 1) / block, n) * H;
  // A key tile takes an item about 1.9 us; a part has four at least.
  const int64_t tiles = (Tk / n + kTileK - 1) / kTileK;
  p.splits = choose_parts(items, kSms / p.cg, tiles * 1.9 + 5.0, (int64_t)Tq * H, kDv, tiles / 4);
  p.ordered = order_pays(n, items * p.splits, kSms / p.cg);
  return p;
}

template <int CG, bool BF16>
cudaError_t launch_prefill(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& pe,
                           const CUtensorMap& v, const PrefillArgs& a, cudaStream_t stream) {
  const auto kernel = mla_prefill_kernel<CG, BF16>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // An item a cluster; those that do not start at once are mostly taken over.
  const int64_t most = ((int64_t)a.Tq + (int64_t)a.n * (Shape<CG>::kBlockQ - 1)) / Shape<CG>::kBlockQ * a.H * a.splits;
  const unsigned grid = (unsigned)(most * CG);
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), (size_t)kSmem, stream, CG == 2 ? 2u : 0u,
                       q, k, pe, v, a);
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
  const int parts = plan_for(Tq, Tk, n, H).splits;
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
  if (((int64_t)Tq / Shape<1>::kBlockQ + n) * H > ((int64_t)1 << 26)) return DSA_ERR_UNSUPPORTED;
  const Plan p = plan_for(Tq, Tk, n, H);
  const int splits = work ? p.splits : 1;
  const int64_t all = (int64_t)Tq * H;
  if (!apart({bytes_of(out, all * kDv * 2), bytes_of(lse2, all * 4),
              bytes_of(splits > 1 ? work : nullptr, splits * all * (kDv + 1) * 4)},
             {rows_of(q, Tq, q_token, H, q_head, kDn + kDr, 2), rows_of(k_nope, Tk, k_token, H, k_head, kDn, 2),
              rows_of(k_pe, Tk, pe_token, 1, 0, kDr, 2), rows_of(v, Tk, v_token, H, v_head, kDv, 2),
              bytes_of(cu_q, ((int64_t)n + 1) * 4), bytes_of(cu_k, ((int64_t)n + 1) * 4)}))
    return DSA_ERR_INVALID_ARG;
  const bool bf16 = dtype == DSA_BF16;
  if (Tk == 0) k_nope = k_pe = v = q;        // never read
  // A dimension of one row has no stride of its own.
  auto map = [&](CUtensorMap* m, const void* p, int width, int heads, int T, int64_t token,
                 int64_t head, uint32_t rows) {
    const uint64_t hs = heads > 1 ? (uint64_t)head * 2 : (uint64_t)width * 2;
    const uint64_t ts = T > 1 ? (uint64_t)token * 2 : hs * heads;
    return encode_map16(m, p, bf16, width, heads, std::max(T, 1), hs, ts, 1, rows);
  };
  const uint32_t keys = (uint32_t)(kTileK / p.cg);
  CUtensorMap tm_q, tm_k, tm_pe, tm_v;
  if (!map(&tm_q, q, kDn + kDr, H, Tq, q_token, q_head, kTileQ) ||
      !map(&tm_k, k_nope, kDn, H, Tk, k_token, k_head, keys) ||
      !encode_map16(&tm_pe, k_pe, bf16, kDr, std::max(Tk, 1), 1, (uint64_t)(Tk > 1 ? pe_token : kDr) * 2,
                    (uint64_t)(Tk > 1 ? pe_token : kDr) * 2 * std::max(Tk, 1), keys, 1) ||
      !map(&tm_v, v, kDv, H, Tk, v_token, v_head, kVKeys))
    return DSA_ERR_CUDA;
  // Heads whose keys and values (512 bytes a token and head) fit half of L2.
  const int64_t fit = ((int64_t)48 << 20) / (512 * (int64_t)std::max(Tk, 1));
  PrefillArgs a{cu_q, cu_k, out, lse2, nullptr, nullptr, err_flags, n, Tq, Tk, H,
                (int)std::max<int64_t>(1, std::min<int64_t>(fit, H)), splits, causal != 0, p.ordered,
                scale == 0.f ? 0x1p-100f : fabsf(scale) * kLog2e, scale < 0.f ? kNegateA : 0u};
  if (splits > 1) {
    a.part_o = work;
    a.part_l = work + (int64_t)splits * Tq * H * kDv;
  }
  const auto launch = p.cg == 2 ? (bf16 ? launch_prefill<2, true> : launch_prefill<2, false>)
                                : (bf16 ? launch_prefill<1, true> : launch_prefill<1, false>);
  if (launch(tm_q, tm_k, tm_pe, tm_v, a, stream) != cudaSuccess) return DSA_ERR_CUDA;
  if (splits > 1) {
    const MergeArgs m{a.part_o, a.part_l, splits, (int64_t)Tq * H, cu_q, n, Tq, H, out, lse2};
    const cudaError_t e = bf16 ? launch_merge<kDv, true>(m, stream) : launch_merge<kDv, false>(m, stream);
    if (e != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}
