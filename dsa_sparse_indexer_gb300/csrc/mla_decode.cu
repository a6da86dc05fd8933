// Latent attention in its absorbed form over each shard's whole paged cache,
// for one token, a chain or a tree of drafted tokens a request (sm_103a).
//
// Request q's n rows (tokens) are the last n of the seq_lens[q] tokens in its
// cache.  Per shard s, row r, head h, over the tokens j of shard s that the row
// sees: x_j = scale * (q[r][h] . row_j), out = sum_j 2^(x_j log2 e) v_j / sum_j
// 2^(x_j log2 e), v_j the first 512 entries of row_j, lse2 = log2 sum_j exp(x_j).
// A row sees every token before the request's n, and of these the ones that its
// tree mask names, or (no mask) those up to itself.
//
// All heads and rows of a request share its keys, so that (row, head) pairs are
// the rows of one product.  Where they are many, an output of 512 values would fill
// tensor memory (512 columns), so an item takes half of it, and its scores are
// computed for both halves: 2304 + 1024 cycles of products for 128 keys where 2176
// are the least (65 %).  What the rows leave on chip decides how keys are held:
//  * Pair, more than 128 rows a request: two CTAs with 128 rows each issue one
//    product of M = 256, and either holds half of the keys' tile (of 128) and of the
//    values' columns.  All queries in shared memory (144 KB) and a ring of 80 KB
//    through which a tile's keys pass in three units, its values in one;
//  * Wide, 33 to 128: the queries' first 256 dimensions in tensor memory, which
//    leaves two stages of 72 KB for whole tiles of 64 keys: their value blocks stay
//    until the value product.  (Scores with N = 64 take 1800 cycles where N = 128
//    takes 1152 a tile, 4624 for 128 keys; one stage of 128 keys took 5.4 us a tile
//    against 4.7 for two of these: its values could not be copied ahead.)
//  * Narrow, up to 32: keys and values as the products' rows, see there.
// The first 256 of an item's output columns, and the last, are its half's value
// blocks; of a tile's nine 64-value blocks the scores take the other five first.
// One warp claims items while the kernel runs, one copies (tensor maps, a box per
// page or 64 keys), one issues products, eight run the softmax.  The keys may be
// split into parts that a second kernel joins.
// Measured, 64 requests of 8192 to 16384 tokens on 4 shards, 128 heads: one token
// 360 us (219 GFLOP, 949 MB; scores of both halves and the 64-key tiles' products
// take 2.2 us of the 4.7 a tile and half), a tree of eight 1465 us after a pause (1.05
// PFLOP/s of the work, 1.6 of what is issued: tensor pipes 68 % busy) and 1550 to 1590
// one after another, at the power limit; one sequence of 32768, one token, 32 us.
// The tail of a sequence's last page holds anything: its values are zeroed in
// shared memory up to the 16 keys that a product step reads, its scores masked.
// Every wait is bounded and raises DSA_FLAG_TIMEOUT when it runs out.
#include <algorithm>
#include <numeric>

#include "regions.h"
#include "split_merge.cuh"

namespace dsa {
namespace {

constexpr int kDqk = DSA_MLA_DQK, kDv = DSA_MLA_DV, kHalf = kDv / 2;
constexpr int kRows = 128;                   // rows of a CTA's product
constexpr int kBlocks = kDqk / 64;           // 9 blocks of 64 values
constexpr int kVBlocks = 4, kABlocks = kBlocks - kVBlocks;   // of a half's values; the others
constexpr int kQBox = 32;                    // rows of a copy of queries
constexpr int kInfo = 8;
constexpr int kCut = 8;                      // bit of a tile's first piece of 16 keys that is there in part
// Warps: 8 of the softmax (sub * 4 + quad: rows quad * 32 + sub * 16 to + 15), one
// issuing products, one copying, one claiming.
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kClaimWarp = 10, kThreads = 352;
constexpr int kTmemCols = 512, kOCol = 0, kQCol = 384;
#ifdef DSA_TEST_STALLED_COPY
// The test-only build (never libdsa.so): the ring's first barrier expects one
// arrival that nothing makes (its copy still lands).
constexpr uint32_t kStalledArrivals = 1;
#else
constexpr uint32_t kStalledArrivals = 0;
#endif

enum Mode { kNarrow16, kNarrow32, kWide, kPair };
template <int M>
struct Cut {
  static constexpr int CG = M == kPair ? 2 : 1;
  static constexpr int kItemRows = M == kNarrow16 ? 16 : M == kNarrow32 ? 32 : CG * kRows;
  static constexpr int kHalves = M == kWide || M == kPair ? 2 : 1;   // items of a row block
  static constexpr int kTile = M == kWide ? 64 : 128;          // keys of a tile
  static constexpr int kPieces = kTile / 16;
};
template <int M>              // Wide, Pair
struct Shape : Cut<M> {
  using Cut<M>::CG;
  static constexpr int kQTm = M == kWide ? 4 : 0;              // query blocks in tensor memory,
  static constexpr int kQBlock = kRows * 128;                  // the others in shared memory
  static constexpr int kQBytes = (kBlocks - kQTm) * kQBlock;
  static constexpr int kBlock = 8192;                          // bytes of 64 keys' 64 values
  // Wide: stages of a tile's nine blocks, the values' four first.
  static constexpr int kStages = 2;
  // Pair: the ring's blocks, 64-value columns of a CTA's values, keys of a value
  // block and bytes of a column in it.
  static constexpr int kRing = 10, kAtoms = kVBlocks / CG, kVKeys = 32, kAtom = kVKeys * 128;
  static constexpr int kKvBytes = (M == kPair ? kRing : kStages * kBlocks) * kBlock;
  __device__ static constexpr uint32_t s_col(uint32_t b) { return 256 + b * Cut<M>::kTile; }
};
// Barriers of key blocks: a pair's units, or a stage's values (at the stage) and
// its other blocks (at kStages + the stage).
constexpr int kUnits = 8;
// Pair: blocks of a unit of the ring.
constexpr uint32_t kKUnit = 3, kVUnit = 4;
__device__ __forceinline__ uint32_t wrap(uint32_t b) { return b >= 10 ? b - 10 : b; }   // into the ring

struct Item {
  int req, shard, half, split;
  int tok0, n;                // the request's rows
  int row0, rows;             // (row, head) pairs of the block: first of the request, how many
  int base;                   // tokens before the request's n (may be negative)
  int nall, nvis, nfree;      // local tokens: in the cache, seen by some row, by every row
  int t0, t1;                 // key tiles
  int bad;                    // a length below zero or past the table
};

template <int M>
struct alignas(1024) DecodeSmem {
  uint8_t q[Shape<M>::kQBytes];
  uint8_t kv[Shape<M>::kKvBytes];
  WorkSlots<Item> work;
  uint64_t full[kUnits], empty[kUnits], qfull, qtm, qempty, sfull[2], pfull[2], pvdone, vtail[2],
      info[kInfo], drain;
  uint32_t tail_seq[2];       // Pair: place in the ring of the values that vtail counts
  Order order;
  uint32_t pages[kInfo];      // pages of stream tile j, at j % kInfo: cache_row's bits, one per 16 keys
  uint32_t tmem;
  int blocks;                 // row blocks of all requests
  int bad;                    // query_starts is not ascending inside the rows
  int abort;
};
static_assert(sizeof(DecodeSmem<kWide>) + 1024 <= 232448 && sizeof(DecodeSmem<kPair>) + 1024 <= 232448,
              "shared memory of a CTA");

struct DecodeArgs {
  const __nv_bfloat16* q;     // [rows][H][kDqk]
  const int32_t* block_table; // [S][reqs][max_blocks]
  const int32_t *starts, *lens;
  const int32_t* mask;        // [rows][words] or null
  __nv_bfloat16* out;         // [S][rows][H][kDv]
  float* lse2;                // [S][rows][H]
  float *part_o, *part_l;     // [splits][S][rows][H][kDv], [splits][S][rows][H]
  uint32_t* flags;
  int64_t n_slots;
  int reqs, max_blocks, block, rows, H, words, splits;
  int ordered;                // items in the requests' order by length
  int cap;                    // local tokens that a table row names
  int kbox, vbox;             // keys of a copy
  // |scale| log2(e), and the score product's descriptor bit that negates A for a
  // negative scale.  A scale of 0 is taken as 2^-100: finite scores then count
  // alike, masked ones are -inf as ever.
  float c2;
  uint32_t negate;
  ShardMath sm;
  FastDiv fblock, fH;
};

struct Cursor {
  int req = 0, before = 0;    // the request's place in the order, row blocks before it
};

// Warp-wide: item `index` of blocks * halves * S * splits: halves and row blocks of a
// request, which read the same keys, beside one another.
template <int M>
__device__ __forceinline__ Item find_item(const DecodeArgs& a, const Order& order, int blocks, bool bad,
                                          int64_t index, Cursor& c) {
  constexpr int kItemRows = Cut<M>::kItemRows;
  const int lane = threadIdx.x & 31;
  Item it;
  it.half = (int)(index % Cut<M>::kHalves);
  const int64_t x = index / Cut<M>::kHalves;
  const int y = (int)(x / blocks), qb = (int)(x - (int64_t)y * blocks);
  it.shard = y / a.splits;
  it.split = y - it.shard * a.splits;
  if (qb < c.before) c = Cursor{};
  int local = 0;
  for (int at = c.req;; at += 32) {
    const int i = at + lane;
    int first = 0, end = 0;
    if (i < a.reqs) bounds_of(a.starts, in_order(order, a.ordered, i), a.rows, bad, first, end);
    const int mine = ((end - first) * a.H + kItemRows - 1) / kItemRows;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned past = __ballot_sync(kFull, c.before + incl > qb);
    if (past) {
      const int l = __ffs(past) - 1;
      c.before += __shfl_sync(kFull, incl - mine, l);
      c.req = at + l;
      local = qb - c.before;
      break;
    }
    c.before += __shfl_sync(kFull, incl, 31);
    if (at + 32 >= a.reqs) break;            // not reached: qb < blocks
  }
  it.req = in_order(order, a.ordered, c.req);
  int end;
  bounds_of(a.starts, it.req, a.rows, bad, it.tok0, end);
  it.n = end - it.tok0;
  it.row0 = local * kItemRows;
  it.rows = min(kItemRows, it.n * a.H - it.row0);
  const int len = max(__ldg(a.lens + it.req), 0);
  it.base = len - it.n;
  const int lo = (int)fdiv((uint32_t)it.row0, a.fH);
  const int hi = (int)fdiv((uint32_t)(it.row0 + it.rows - 1), a.fH);
  auto local_of = [&](int t) { return min((int)a.sm.local_len((uint32_t)max(t, 0), it.shard), a.cap); };
  it.bad = __ldg(a.lens + it.req) < 0 || (int)a.sm.local_len((uint32_t)len, it.shard) > a.cap;
  it.nall = local_of(len);
  it.nvis = a.mask ? it.nall : local_of(it.base + hi + 1);
  it.nfree = local_of(a.mask ? it.base : it.base + lo + 1);
  constexpr int kTile = Cut<M>::kTile;
  const int nt = (it.nvis + kTile - 1) / kTile, per = (nt + a.splits - 1) / a.splits;
  it.t0 = min(it.split * per, nt);
  it.t1 = min(it.t0 + per, nt);
  return it;
}

// Steps of 16 keys of tile t's value product, and whether it reads keys behind
// the sequence's end (zeroed in shared memory by the softmax warps).
template <int M>
__device__ __forceinline__ int value_steps(const Item& it, int t) {
  constexpr int kTile = Cut<M>::kTile;
  return (min(it.nvis - t * kTile, kTile) + 15) / 16;
}
template <int M>
__device__ __forceinline__ bool has_tail(const Item& it, int t) {
  return it.nall - t * Cut<M>::kTile < 16 * value_steps<M>(it, t);
}
// The i-th block that an item's scores take first, of the nine; its i-th value block.
__device__ __forceinline__ int block_a(int half, int i) {
  return half == 0 ? kVBlocks + i : (i < kVBlocks ? i : kBlocks - 1);
}
__device__ __forceinline__ int block_v(int half, int i) { return half * kVBlocks + i; }

// ---- the copies ---------------------------------------------------------------
// A tile's keys 16 l to 16 l + 15 lie in a page: lane l (of as many as the tile has
// such pieces, repeated) has the page's table entry, then the first one's cache row.
template <int M>
__device__ __forceinline__ int table_entry(const DecodeArgs& a, const Item& it, int t) {
  const int key = t * Cut<M>::kTile + (int)(threadIdx.x % Cut<M>::kPieces) * 16;
  if (t < it.t0 || key >= it.nall) return -1;
  return __ldg(a.block_table + ((int64_t)it.shard * a.reqs + it.req) * a.max_blocks +
               fdiv((uint32_t)key, a.fblock));
}
// That row, which may be `n_slots` (outside: reads as zero) where there is none;
// `valid` gets a bit a piece that there is, and at kCut one a piece that the cache's
// end cuts: pieces start at multiples of 16, so that n_slots % 16 slots are left of it.
template <int M>
__device__ __forceinline__ int cache_row(const DecodeArgs& a, const Item& it, int t, int entry, uint32_t& valid,
                                         bool& bad) {
  const int key = t * Cut<M>::kTile + (int)(threadIdx.x % Cut<M>::kPieces) * 16;
  int y = (int)a.n_slots;
  bool in = false, cut = false;
  if (key < it.nall) {
    uint32_t off;
    fdivmod((uint32_t)key, a.fblock, &off);
    const int64_t at = (int64_t)entry * a.block + off;
    in = at >= 0 && at + 16 <= a.n_slots;
    cut = at >= 0 && !in && at < a.n_slots;
    if (in || cut) y = (int)at;
    bad |= at < 0 || at + min(16, it.nall - key) > a.n_slots;
  }
  constexpr unsigned kAll = (1u << Cut<M>::kPieces) - 1u;
  valid = (__ballot_sync(kFull, in) & kAll) | (__ballot_sync(kFull, cut) & kAll) << kCut;
  return y;
}

// Ring of the pair: units are freed in the order in which they were copied.
struct Ring {
  uint32_t unit = 0, oldest = 0;             // the next unit; the oldest not known to be free
  uint32_t used = 0, at = 0;                 // blocks not known to be free; the next block's place
  uint32_t values = 0;                       // bit i: unit oldest + i is one of values
};

struct PendingV {              // values of a stream tile whose keys are copied
  int y, half, shard;          // lane l: row of the cache of its keys 16 l
  bool tail;
};

template <int M>
__device__ __forceinline__ void load_tiles(const DecodeArgs& a, DecodeSmem<M>& sm,
                                           const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                           const CUtensorMap* tm_v, uint32_t rank) {
  using Sh = Shape<M>;
  constexpr int CG = Sh::CG;
  const int lane = threadIdx.x & 31;
  const bool leader = rank == 0;
  Item it;
  constexpr int kPieces = Sh::kPieces;
  uint32_t j = 0, loads = 0, tails = 0;      // tiles, items' queries, tails so far
  bool ok = true, bad = false;
  bool half_tile = false;                    // the last tile's values were not copied
  Ring ring;
  PendingV p0{}, p1{};
  // Pair: waits for a unit's space; its barrier then expects the pair's bytes (or,
  // values with a tail, an arrival alone: they are counted elsewhere).
  auto open_unit = [&](uint32_t blocks, bool bytes) {
    while (ok && ring.used + blocks > Sh::kRing) {
      ok = warp_wait(&sm.abort, &sm.empty[ring.oldest % kUnits], (ring.oldest / kUnits) & 1u);
      ring.used -= ring.values & 1u ? kVUnit : kKUnit;
      ring.values >>= 1;
      ++ring.oldest;
    }
    if (ok && leader && lane == 0) {
      uint64_t* bar = &sm.full[ring.unit % kUnits];
      if (bytes) mbar_expect_tx(bar, (uint32_t)CG * blocks * Sh::kBlock);
      else mbar_arrive1(bar);
    }
    return ok;
  };
  auto close_unit = [&](uint32_t blocks, bool is_values) {
    ring.values |= (is_values ? 1u : 0u) << (ring.unit - ring.oldest);
    ++ring.unit;
    ring.used += blocks;
    ring.at = wrap(ring.at + blocks);
  };
  auto load_values = [&](const PendingV& p) {
    uint64_t* vtail = &sm.vtail[tails & 1u];
    if (p.tail && lane == 0) {
      sm.tail_seq[tails & 1u] = ring.at;     // published by the barrier
      mbar_expect_tx(vtail, (uint32_t)(kVBlocks * Sh::kBlock));
    }
    tails += p.tail;
    const int boxes = Sh::kVKeys / a.vbox, per = Sh::kAtoms * boxes;   // of a block
    for (uint32_t b = 0; b < kVBlocks; b += kVUnit) {
      if (!open_unit(kVUnit, !p.tail)) return;
      const uint32_t bar = p.tail ? smem_u32(vtail) : leader_addr(&sm.full[ring.unit % kUnits]);
      const int i = lane / per, atom = lane % per / boxes, key = lane % boxes * a.vbox;
      const int y = __shfl_sync(kFull, p.y, (((int)b + i) * Sh::kVKeys + key) >> 4 & 7);
      if (i < (int)kVUnit)
        load_box<CG>(sm.kv + wrap(ring.at + i) * Sh::kBlock + atom * Sh::kAtom + key * 128, tm_v,
                     p.half * kHalf + ((int)rank * Sh::kAtoms + atom) * 64, y, p.shard, bar);
      close_unit(kVUnit, true);
    }
  };
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok, it); ++n) {
    item_done(sm.work, n);
    bad |= it.bad != 0;
    int next = table_entry<M>(a, it, it.t1 - 1);
    for (int t = it.t1 - 1; ok && t >= it.t0; --t, ++j) {
      uint32_t valid;
      const int y = cache_row<M>(a, it, t, next, valid, bad);
      next = table_entry<M>(a, it, t - 1);   // on its way while this tile is copied
      if (M == kPair && t < it.t1 - 2) load_values(p0);
      if (!ok) break;
      if (t == it.t1 - 1) {                  // the item's queries
        if (loads > 0) ok = warp_wait(&sm.abort, &sm.qempty, (loads - 1) & 1u);
        if (!ok) break;
        ++loads;
        constexpr int kN = kBlocks - Sh::kQTm;
        auto boxes = [&](int r) { return (min(max(it.rows - r * kRows, 0), kRows) + kQBox - 1) / kQBox; };
        if (leader && lane == 0)
          mbar_expect_tx(&sm.qfull, (uint32_t)((boxes(0) + (CG == 2 ? boxes(1) : 0)) * kN * kQBox * 128));
        const uint32_t bar = CG == 1 ? smem_u32(&sm.qfull) : leader_addr(&sm.qfull);
        if (lane < kN)
          for (int b = 0; b < boxes((int)rank); ++b)
            load_box<CG>(sm.q + lane * Sh::kQBlock + b * kQBox * 128, tm_q, (Sh::kQTm + lane) * 64,
                         it.tok0 * a.H + it.row0 + (int)rank * kRows + b * kQBox, 0, bar);
      }
      if (lane == 0) {
        sm.pages[j % kInfo] = valid;
        mbar_arrive1(&sm.info[j % kInfo]);
      }
      const int boxes = 64 / a.kbox;         // of a block: 1 to 4
      const int i = lane / boxes, first = lane % boxes * a.kbox;
      const int yk = __shfl_sync(kFull, y, ((int)rank * 64 + first) / 16 % kPieces);
      if constexpr (M == kPair) {
        for (uint32_t b = 0; b < kBlocks; b += kKUnit) {
          if (!open_unit(kKUnit, true)) break;
          const uint32_t bar = leader_addr(&sm.full[ring.unit % kUnits]);
          if (i < (int)kKUnit)
            load_box<CG>(sm.kv + wrap(ring.at + i) * Sh::kBlock + first * 128, tm_k,
                         ((int)b + i) * 64, yk, it.shard, bar);
          close_unit(kKUnit, false);
        }
        p0 = p1;
        p1 = PendingV{y, it.half, it.shard, has_tail<M>(it, t)};
      } else {
        const uint32_t st = j % Sh::kStages, use = j / Sh::kStages;
        uint8_t* stage = sm.kv + st * kBlocks * Sh::kBlock;
        if (use > 0) ok = warp_wait(&sm.abort, &sm.empty[Sh::kStages + st], (use - 1) & 1u);
        if (!ok) break;
        uint64_t* bar = &sm.full[Sh::kStages + st];
        if (lane == 0) mbar_expect_tx(bar, kABlocks * Sh::kBlock);
        if (i < kABlocks)
          load_box<CG>(stage + (kVBlocks + i) * Sh::kBlock + first * 128, tm_k, block_a(it.half, i) * 64, yk,
                       it.shard, smem_u32(bar));
        if (use > 0) ok = warp_wait(&sm.abort, &sm.empty[st], (use - 1) & 1u);
        if (!ok) {
          half_tile = true;
          ++j;
          break;
        }
        bar = &sm.full[st];
        if (lane == 0) mbar_expect_tx(bar, kVBlocks * Sh::kBlock);
        if (i < kVBlocks)
          load_box<CG>(stage + i * Sh::kBlock + first * 128, tm_k, block_v(it.half, i) * 64, yk, it.shard,
                       smem_u32(bar));
      }
    }
    if (M == kPair && ok && it.t1 - it.t0 >= 2) load_values(p0);
    if (M == kPair && ok && it.t1 - it.t0 >= 1) load_values(p1);
  }
  if (__any_sync(kFull, bad) && lane == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  if (!ok && lane == 0) {
    if (!cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
    // The copies issued land before the CTA ends (a pair's first CTA counts both's).
    if (leader && loads > 0) mbar_wait(&sm.qfull, (loads - 1) & 1u);
    if constexpr (M == kPair) {
      for (uint32_t u = ring.oldest; leader && u < ring.unit; ++u)
        mbar_wait(&sm.full[u % kUnits], (u / kUnits) & 1u);
      for (uint32_t k = tails > 2 ? tails - 2 : 0; k < tails; ++k)
        mbar_wait(&sm.vtail[k & 1u], (k >> 1) & 1u);
    } else {
      for (uint32_t v = j > Sh::kStages ? j - Sh::kStages : 0; v < j; ++v) {
        mbar_wait(&sm.full[Sh::kStages + v % Sh::kStages], (v / Sh::kStages) & 1u);
        if (v + 1 < j || !half_tile) mbar_wait(&sm.full[v % Sh::kStages], (v / Sh::kStages) & 1u);
      }
    }
  }
  // The products' arrivals come to both CTAs of a pair: the second, which waits for few
  // of them, sees the last before it ends.
  if (CG == 2 && !leader) wait_landed(&sm.drain, 0);
  __syncwarp();
}

// ---- the products: a warp of the (first) CTA ------------------------------------
// It runs along converged and one elected lane issues: inside a branch of one lane
// the descriptors could not stay in uniform registers.
template <int M>
__device__ __forceinline__ void issue_products(const DecodeArgs& a, DecodeSmem<M>& sm, uint32_t tmem) {
  using Sh = Shape<M>;
  constexpr int CG = Sh::CG;
  const uint32_t id_s = idesc_f16(CG * kRows, Sh::kTile, true, false) | a.negate;
  constexpr uint32_t id_o = idesc_f16(CG * kRows, kHalf, true, true);
  constexpr int kStep = Sh::kBlock >> 4;     // a block in a descriptor's address field
  const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q), 16, 1024);
  const uint64_t k0 = smem_desc_sw128(smem_u32(sm.kv), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(smem_u32(sm.kv), M == kPair ? Sh::kAtom : Sh::kBlock, 1024);
  Item it;
  uint32_t j = 0, nq = 0;                    // tiles, items' queries so far
  uint32_t unit = 0, blk = 0;                // Pair: the ring's next unit and block
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && warp_wait(&sm.abort, bar, parity);
    tc_fence_after();
    return ok;
  };
  // Scores with block kb, whose keys' descriptor is kd.
  auto block_products = [&](uint32_t d, int kb, uint64_t kd, bool first) {
    if (kb < Sh::kQTm) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_ts<CG>(d, tmem + kQCol + kb * 32 + s * 8, kd + s * 2, id_s, (first && s == 0) ? 0u : 1u);
    } else {
      const uint64_t qd = q0 + (uint32_t)(kb - Sh::kQTm) * (Sh::kQBlock >> 4);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_ss<CG>(d, qd + s * 2, kd + s * 2, id_s, (first && s == 0) ? 0u : 1u);
    }
  };
  // Values of stream tile v: `steps` of 16 keys, the item's first or not.
  auto values = [&](uint32_t v, int steps, bool first) {
    const uint32_t b = v % 2, p = tmem + Sh::s_col(b);
    if (!wait(&sm.pfull[b], (v / 2) & 1u)) return;
    if constexpr (M == kPair) {
#pragma unroll 1
      for (uint32_t u = 0; u < kVBlocks / kVUnit; ++u, ++unit, blk = wrap(blk + kVUnit)) {
        if (!wait(&sm.full[unit % kUnits], (unit / kUnits) & 1u)) return;
        if (elect_one()) {
#pragma unroll
          for (uint32_t c = 0; c < kVUnit; ++c) {
            const uint64_t vd = v0 + wrap(blk + c) * kStep;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int step = (int)(u * kVUnit + c) * 2 + s;
              if (step < steps)
                mma_ts<CG>(tmem + kOCol, p + step * 8, vd + s * (2048 >> 4), id_o,
                           (first && step == 0) ? 0u : 1u);
            }
          }
          tc_commit<CG>(&sm.empty[unit % kUnits]);
          if (u == kVBlocks / kVUnit - 1) tc_commit<CG>(&sm.pvdone);
        }
        __syncwarp();
      }
    } else {
      const uint32_t st = v % Sh::kStages;
      const uint64_t vd = v0 + st * (kBlocks * kStep);
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < Sh::kTile / 16; ++s)
          if (s < steps)
            mma_ts<CG>(tmem + kOCol, p + s * 8, vd + s * (2048 >> 4), id_o, (first && s == 0) ? 0u : 1u);
        tc_commit<CG>(&sm.empty[st]);
        tc_commit<CG>(&sm.pvdone);
      }
      __syncwarp();
    }
  };
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok, it); ++n) {
    item_done(sm.work, n);
    for (int t = it.t1 - 1; ok && t >= it.t0; --t, ++j) {
      if (M == kPair && t < it.t1 - 2) values(j - 2, value_steps<M>(it, t + 2), t + 2 == it.t1 - 1);
      if (ok && t == it.t1 - 1) {
        if (!wait(&sm.qfull, nq & 1u)) break;
        if (Sh::kQTm > 0 && !wait(&sm.qtm, nq & 1u)) break;
        ++nq;
      }
      const uint32_t b = j % 2, d = tmem + Sh::s_col(b);
      auto scores_done = [&]() {
        tc_commit<CG>(&sm.sfull[b]);
        if (t == it.t0) tc_commit<CG>(&sm.qempty);
      };
      if constexpr (M == kPair) {
#pragma unroll 1
        for (uint32_t u = 0; ok && u < kBlocks / kKUnit; ++u, ++unit, blk = wrap(blk + kKUnit)) {
          if (!wait(&sm.full[unit % kUnits], (unit / kUnits) & 1u)) break;
          if (elect_one()) {
#pragma unroll
            for (uint32_t c = 0; c < kKUnit; ++c)
              block_products(d, (int)(u * kKUnit + c), k0 + wrap(blk + c) * kStep, u == 0 && c == 0);
            tc_commit<CG>(&sm.empty[unit % kUnits]);
            if (u == kBlocks / kKUnit - 1) scores_done();
          }
          __syncwarp();
        }
      } else {
        const uint32_t st = j % Sh::kStages, turn = (j / Sh::kStages) & 1u;
        const uint64_t kd = k0 + st * (kBlocks * kStep);
        if (!wait(&sm.full[Sh::kStages + st], turn)) break;
        if (elect_one()) {
#pragma unroll 1
          for (int i = 0; i < kABlocks; ++i)
            block_products(d, block_a(it.half, i), kd + (kVBlocks + i) * kStep, i == 0);
          tc_commit<CG>(&sm.empty[Sh::kStages + st]);
        }
        __syncwarp();
        if (!wait(&sm.full[st], turn)) break;
        if (elect_one()) {
#pragma unroll 1
          for (int i = 0; i < kVBlocks; ++i) block_products(d, block_v(it.half, i), kd + i * kStep, false);
          scores_done();
        }
        __syncwarp();
        // The last tile's values, under this tile's softmax.
        if (t < it.t1 - 1) values(j - 1, value_steps<M>(it, t + 1), t + 1 == it.t1 - 1);
      }
    }
    if (M != kPair && ok && it.t1 > it.t0) values(j - 1, value_steps<M>(it, it.t0), it.t0 == it.t1 - 1);
    if (M == kPair && ok && it.t1 - it.t0 >= 2)
      values(j - 2, value_steps<M>(it, it.t0 + 1), it.t0 + 1 == it.t1 - 1);
    if (M == kPair && ok && it.t1 > it.t0) values(j - 1, value_steps<M>(it, it.t0), it.t0 == it.t1 - 1);
  }
  const int lane = threadIdx.x & 31;
  if (!ok && lane == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
  __syncwarp();
  // Every product issued completes before the tensor memory is freed (a commit
  // counts the thread's own: elect_one picks the same lane every time).
  if (elect_one()) {
    tc_commit<CG>(&sm.drain);
    if (!mbar_wait(&sm.drain, 0)) cta_abort(&sm.abort, a.flags);
  }
  __syncwarp();
}

// Which of the 32 keys from local token `from` on row `tok` (of the request's) sees:
// those that all rows see, then the chain's up to itself, or a tree's one by one (as
// many as are drafted; every key asked for one by one took an item 4 us).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u;
}
// Of a tile's 16 keys `piece`, those that the cache holds.
__device__ __forceinline__ uint32_t piece_bits(const DecodeArgs& a, uint32_t pages, int piece) {
  return (pages >> piece) & 1u ? 0xffffu : (pages >> (kCut + piece)) & 1u ? first_bits((int)a.n_slots & 15) : 0u;
}
__device__ __forceinline__ uint32_t seen32(const DecodeArgs& a, const Item& it, int tok, int from) {
  if (!a.mask) {
    const int own = (int)a.sm.local_len((uint32_t)max(it.base + tok + 1, 0), it.shard);
    return first_bits(min(own, it.nvis) - from);
  }
  uint32_t seen = first_bits(it.nfree - from), word = 0;
  int at = -1;
#pragma unroll 1
  for (int l = max(from, it.nfree); l < min(from + 32, it.nvis); ++l) {
    const int i = (int)a.sm.global_id(it.shard, (uint32_t)l) - it.base;   // the request's row
    bool see = i < 0;
    if (!see && (i >> 5) < a.words) {
      if ((i >> 5) != at) {
        at = i >> 5;
        word = (uint32_t)__ldg(a.mask + (int64_t)(it.tok0 + tok) * a.words + at);
      }
      see = (word >> (i & 31)) & 1u;
    }
    seen |= (uint32_t)see << (l - from);
  }
  return seen;
}

// ---- softmax and outputs --------------------------------------------------------
// A warp has 16 rows, four lanes a row and two rows a lane (tensor memory's
// fragments).  Warps without a row of the item only keep step.
template <int M>
__device__ __forceinline__ void softmax_tiles(const DecodeArgs& a, DecodeSmem<M>& sm, uint32_t tmem,
                                              int warp, uint32_t rank) {
  using Sh = Shape<M>;
  constexpr int CG = Sh::CG;
  const int lane = threadIdx.x & 31;
  const int sub = warp >> 2, quad = warp & 3;
  const int r0 = quad * 32 + sub * 16;       // the warp's first row of the CTA's
  const int br = (int)rank * kRows + r0 + (lane >> 2);   // the lane's rows of the block: br, br + 8
  const int col = 2 * (lane & 3);            // its first of 8 columns
  const uint32_t trow = tmem + ((uint32_t)r0 << 16), t_o = trow + kOCol;
  // Over the four lanes of a row.
  auto row_max = [](float v) {
    v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
    return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
  };
  auto row_sum = [](float v) {
    v += __shfl_xor_sync(kFull, v, 1);
    return v + __shfl_xor_sync(kFull, v, 2);
  };
  uint32_t j = 0, tails = 0;                 // tiles and tails so far
  bool ok = true;
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok); ++n) {
    const Item& it = sm.work.item[n & 1u];   // read where it lies
    const int t0 = uni(it.t0), t1 = uni(it.t1), nall = uni(it.nall), nfree = uni(it.nfree);
    const bool mine = (int)rank * kRows + r0 < uni(it.rows);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    if (M == kWide && t1 > t0) {
      // The queries' first 256 dimensions into tensor memory, a row a lane (the last
      // item's scores are through: its outputs were waited for); rows past the
      // item's repeat its last.
      const int row = min(quad * 32 + lane, it.rows - 1);
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((int64_t)it.tok0 * a.H + it.row0 + row) * kDqk + sub * 128);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = __ldg(src + 4 * c + i);
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
        tmem_store(tmem + ((uint32_t)(quad * 32) << 16) + kQCol + sub * 64 + c * 16, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.qtm);
    }
    for (int t = t1 - 1; t >= t0; --t, ++j) {
      const uint32_t b = j % 2;
      ok = warp_wait(&sm.abort, &sm.sfull[b], (j / 2) & 1u) &&
           warp_wait(&sm.abort, &sm.info[j % kInfo], (j / kInfo) & 1u);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_s = trow + Sh::s_col(b);
      float alpha[2] = {1.f, 1.f};
      if (mine) {
        const uint32_t pages = *reinterpret_cast<volatile uint32_t*>(&sm.pages[j % kInfo]);
        const bool masked = pages != (1u << (Sh::kTile / 16)) - 1u || (t + 1) * Sh::kTile > nfree;
        uint32_t seen[2] = {kFull, kFull};   // of keys 32 (lane % 4) on, by either row
        if (masked) {
          keep_branch();
          const int c = lane & (Sh::kTile / 32 - 1);
          const uint32_t there = piece_bits(a, pages, 2 * c) | piece_bits(a, pages, 2 * c + 1) << 16;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int row = it.row0 + min(br + 8 * k, it.rows - 1);
            seen[k] = seen32(a, it, (int)fdiv((uint32_t)row, a.fH), t * Sh::kTile + c * 32) & there;
          }
        }
        auto mask = [&](uint32_t (&x)[16], int c) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w = __shfl_sync(kFull, seen[k], (lane & ~3) | c) >> col;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (!((w >> (8 * i)) & 1u)) x[4 * i + 2 * k] = 0xff800000u;
              if (!((w >> (8 * i + 1)) & 1u)) x[4 * i + 2 * k + 1] = 0xff800000u;
            }
          }
        };
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < Sh::kTile / 32; c += 2) {
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
          for (int k = 0; k < 2; ++k) {      // the lane's rows
            float v[2] = {top[k], -INFINITY};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                v[h] = fmax3(v[h], __uint_as_float(x[h][4 * i + 2 * k]),
                             __uint_as_float(x[h][4 * i + 2 * k + 1]));
            top[k] = fmaxf(v[0], v[1]);
          }
        }
        float2 nref[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float mx = row_max(top[k]) * a.c2;
          const float mn = mx > m[k] + kRescaleGap ? mx : m[k];   // m = -inf takes any finite maximum
          alpha[k] = m[k] == -INFINITY ? 1.f : fast_exp2(m[k] - mn);
          const float ref = mn == -INFINITY ? 0.f : mn;
          nref[k] = make_float2(-ref, -ref);
          m[k] = mn;
          l[k] *= alpha[k];
        }
        const float2 c2v = make_float2(a.c2, a.c2);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t y[2][16];
        if (masked) tmem_wait_st();
        tmem_load_frag(t_s, y[0]);
#pragma unroll
        for (int c = 0; c < Sh::kTile / 32; ++c) {
          uint32_t (&x)[16] = y[c & 1];
          tmem_wait_ld(x);
          if (c + 1 < Sh::kTile / 32) tmem_load_frag(t_s + (c + 1) * 32, y[(c + 1) & 1]);   // before weights overwrite it
          uint32_t p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 e = ffma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                   c2v, nref[i & 1]);
            const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
            p[i] = pack16<true>(e0, e1);
            sum[i & 1] = fadd2(sum[i & 1], make_float2(e0, e1));
          }
          tmem_store_pairs(t_s + c * 16, p);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) l[k] += sum[k].x + sum[k].y;
      }
      if (t < t1 - 1) {                      // the previous tile's values are in: O is at rest
        ok = warp_wait(&sm.abort, &sm.pvdone, (j - 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        if (__any_sync(kFull, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < kHalf; c += 32) {
            uint32_t o[16];
            tmem_load_frag(t_o + (uint32_t)c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha[(k >> 1) & 1]);
            tmem_store_frag(t_o + (uint32_t)c, o);
          }
        }
      }
      if (has_tail<M>(it, t)) {                 // values behind the sequence's end: zeros
        constexpr int kChunks = Sh::kAtoms * 8;   // 16-byte pieces of a key's values
        const int past = nall - t * Sh::kTile, to = 16 * value_steps<M>(it, t);
        if constexpr (M == kPair) {
          ok = warp_wait(&sm.abort, &sm.vtail[tails & 1u], (tails >> 1) & 1u);
          if (!ok) break;
        }
        const uint32_t seq = M == kPair ? *reinterpret_cast<volatile uint32_t*>(&sm.tail_seq[tails & 1u]) : 0u;
        ++tails;
        for (int z = warp * 32 + lane; z < (to - past) * kChunks; z += kSoftmaxWarps * 32) {
          const int key = past + z / kChunks, chunk = z % kChunks;
          uint8_t* at;
          if constexpr (M == kPair)
            at = sm.kv + wrap(seq + (uint32_t)(key / Sh::kVKeys)) * Sh::kBlock +
                 (chunk >> 3) * Sh::kAtom + (key % Sh::kVKeys) * 128;
          else
            at = sm.kv + ((j % Sh::kStages) * kBlocks + (chunk >> 3)) * Sh::kBlock + key * 128;
          *reinterpret_cast<uint4*>(at + (chunk & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_for_products<CG>();            // before this warp hands its weights over
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive1(&sm.pfull[b]);
        else mbar_arrive_leader(&sm.pfull[b]);
      }
    }
    const bool some = t1 > t0, parts = a.splits > 1;
    if (ok && some) ok = warp_wait(&sm.abort, &sm.pvdone, (j - 1) & 1u);
    if (!ok) break;
    if (some) tc_fence_after();
    if (mine) {
      const int64_t all = (int64_t)a.rows * a.H;
      const int64_t to = ((int64_t)(parts ? it.split : 0) * a.sm.S + it.shard) * all +
                         (int64_t)it.tok0 * a.H + it.row0 + br;   // [splits][S][rows][H]
      bool active[2];
      float inv[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] = row_sum(l[k]);
        active[k] = br + 8 * k < it.rows;
        inv[k] = l[k] == 0.f ? 0.f : 1.f / l[k];
        if (active[k] && it.half == 0 && (lane & 3) == 0)
          (parts ? a.part_l : a.lse2)[to + 8 * k] = l[k] == 0.f ? -INFINITY : m[k] + log2f(l[k]);
      }
      if (some || !parts) {                  // the merge does not read an empty part
        const int64_t at = to * kDv + it.half * kHalf;
        // Rows that saw nothing are zeros, whatever their columns hold.
        const bool seen_all = some && __all_sync(kFull, l[0] != 0.f && l[1] != 0.f);
        uint32_t y[2][16];
        if (some) tmem_load_frag(t_o, y[0]);
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t (&o)[16] = y[c / 32 & 1];
          if (some) {
            tmem_wait_ld(o);
            if (c + 32 < kHalf) tmem_load_frag(t_o + (uint32_t)c + 32, y[(c / 32 + 1) & 1]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv[(i >> 1) & 1]);
          if (!seen_all) {
            keep_branch();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!some || l[(i >> 1) & 1] == 0.f) o[i] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (parts) {
              if (active[k]) {
                float* dst = a.part_o + at + 8 * k * kDv + c + col;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  *reinterpret_cast<uint2*>(dst + 8 * i) = make_uint2(o[4 * i + 2 * k], o[4 * i + 2 * k + 1]);
              }
            } else {
              store_row<true>(o, k, lane, active[k],
                              reinterpret_cast<uint16_t*>(a.out) + at + 8 * k * kDv + c);
            }
          }
          __syncwarp();                      // the next columns' load takes the whole warp
        }
      }
    }
    item_done(sm.work, n);
  }
  if (!ok && lane == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
}

template <int M>
__global__ void __launch_bounds__(kThreads, 1)
    mla_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a) {
  using Sh = Shape<M>;
  constexpr int CG = Sh::CG;
  extern __shared__ unsigned char decode_smem_raw[];
  DecodeSmem<M>& sm = *reinterpret_cast<DecodeSmem<M>*>(
      (reinterpret_cast<uintptr_t>(decode_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = uni(tid >> 5);
  const uint32_t rank = CG == 2 ? pair_rank() : 0u;
  if (warp == kMmaWarp) {
    tmem_alloc<CG>(&sm.tmem, kTmemCols);
  } else if (warp == kClaimWarp) {
    bool bad;
    const int blocks = count_blocks(a.starts, a.rows, nullptr, 0, a.reqs, a.H, Cut<M>::kItemRows, a.flags, bad);
    if ((tid & 31) == 0) sm.blocks = blocks, sm.bad = bad;
  } else if (tid == 0) {
    for (int b = 0; b < kUnits; ++b) mbar_init(&sm.full[b], 1 + (b == 0 ? kStalledArrivals : 0));
    for (int b = 0; b < kUnits; ++b) mbar_init(&sm.empty[b], 1);
    mbar_init(&sm.qtm, kSoftmaxWarps);
    mbar_init(&sm.qfull, 1);
    mbar_init(&sm.qempty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.sfull[b], 1);
      mbar_init(&sm.pfull[b], kSoftmaxWarps * CG);   // a warp each, of both CTAs in a pair's first
      mbar_init(&sm.vtail[b], 1);
    }
    for (int b = 0; b < kInfo; ++b) mbar_init(&sm.info[b], 1);
    mbar_init(&sm.pvdone, 1);
    mbar_init(&sm.drain, 1);
    init_slots(sm.work, CG, kSoftmaxWarps + 1 + (rank == 0 ? 1 : 0));
    sm.abort = 0;
    mbar_init_fence();
  }
  if (a.ordered) longest_first(sm.order, a.reqs, tid, [&](int i) { return __ldg(a.lens + i); });
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) pair_sync();        // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = uni(sm.tmem);
  if (warp == kLoadWarp) {
    load_tiles<M>(a, sm, &tm_q, &tm_k, &tm_v, rank);
  } else if (warp < kSoftmaxWarps) {
    softmax_tiles<M>(a, sm, tmem, warp, rank);
  } else if (warp == kClaimWarp) {
    const int blocks = sm.blocks;
    const bool bad = sm.bad != 0;
    Cursor cur;
    share_out<CG>(sm.work, &sm.abort, a.flags, (int64_t)blocks * 2 * a.sm.S * a.splits, rank,
                  [&](int64_t i) { return find_item<M>(a, sm.order, blocks, bad, i, cur); });
  } else if (rank == 0) {
    issue_products<M>(a, sm, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) pair_sync();        // neither CTA's memory goes while the other uses it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free<CG>(tmem, kTmemCols);
  }
}

// ---- few rows: keys and values as the products' rows ----------------------------
// S^T = K Q^T (128 keys x N rows) and O^T = V^T P^T (512 values x N rows, four
// products of 128 values): all outputs fit 4 N columns, so that keys are read and
// scored once.  A step of 16 takes 60 cycles here and 82 with values (their rows lie
// across), whatever N up to 32, 4800 cycles for 128 keys where the rows as A would
// take 9250 for both halves.
//  * tensor memory: two tiles' scores (N columns each; a lane is a key), outputs
//    (4 N; a lane is one of 128 values);
//  * shared memory: a tile's 128 keys as four slots of 128 values (32 KB) and one
//    of the last 64 (16 KB), five and kTails of them; the queries; the weights (a
//    row's 64 keys to 128 bytes).  Keys stay for the value product, which frees
//    them slot by slot; what the slots have room for of the next tile is scored
//    under the softmax.
//  * four softmax warps, a thread a key, which exchange maxima and sums through
//    shared memory; one issuing products, one copying, one claiming.
// Measured, 128 requests of 2048 to 8192 tokens on 8 shards, 16 heads: 163 us, 4.7
// TB/s; a tile takes 6100 cycles (the products' 4800 and the softmax's part that
// they do not cover), 147 KB in 3.2 us of this SM's share.
constexpr int kNarrowWarps = 4, kNarrowMma = 4, kNarrowLoad = 5, kNarrowClaim = 6, kNarrowThreads = 224;
constexpr int kSlots = 5, kSlot = 32768, kSlotBlock = 16384;   // a slot's two blocks: 128 keys' 64 values

template <int M>
struct alignas(1024) NarrowSmem {
  static constexpr int N = Cut<M>::kItemRows;
  static constexpr int kTails = N == 16 ? 2 : 1;
  uint8_t kv[kSlots][kSlot];
  uint8_t tail[kTails][kSlotBlock];
  uint8_t q[kBlocks][N * 128];
  uint8_t p[2][N * 128];      // the weights of 64 keys each
  float exchange[2][kNarrowWarps][N];
  WorkSlots<Item> work;
  uint64_t full[kSlots], empty[kSlots], tail_full[kTails], tail_empty[kTails], qfull, qempty, sfull[2], pfull, pvdone,
      exchanged, info[kInfo], drain;
  uint32_t pages[kInfo];
  Order order;
  uint32_t tmem;
  int blocks, bad;
  int abort;
};
static_assert(sizeof(NarrowSmem<kNarrow16>) + 1024 <= 232448 && sizeof(NarrowSmem<kNarrow32>) + 1024 <= 232448,
              "shared memory of a CTA");

template <int M>
__device__ __forceinline__ void narrow_load(const DecodeArgs& a, NarrowSmem<M>& sm, const CUtensorMap* tm_q,
                                            const CUtensorMap* tm_k) {
  using Sm = NarrowSmem<M>;
  constexpr int kTails = Sm::kTails, kPieces = Cut<M>::kPieces;
  const int lane = threadIdx.x & 31;
  const int boxes = Cut<M>::kTile / a.kbox, i = lane / boxes, first = lane % boxes * a.kbox;   // 2 to 8 a block
  Item it;
  uint32_t j = 0, slot = 0, loads = 0;       // tiles, slots and items' queries so far
  uint32_t tails = 0;
  bool ok = true, bad = false;
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok, it); ++n) {
    item_done(sm.work, n);
    bad |= it.bad != 0;
    int next = table_entry<M>(a, it, it.t1 - 1);
    for (int t = it.t1 - 1; ok && t >= it.t0; --t, ++j) {
      uint32_t valid;
      const int y = cache_row<M>(a, it, t, next, valid, bad);
      next = table_entry<M>(a, it, t - 1);   // on its way while this tile is copied
      const int yk = __shfl_sync(kFull, y, first / 16 % kPieces);
      if (t == it.t1 - 1) {                  // the item's queries
        if (loads > 0) ok = warp_wait(&sm.abort, &sm.qempty, (loads - 1) & 1u);
        if (!ok) break;
        ++loads;
        if (lane == 0) mbar_expect_tx(&sm.qfull, kBlocks * Sm::N * 128);
        if (lane < kBlocks)
          load_box<1>(sm.q[lane], tm_q, lane * 64, it.tok0 * a.H + it.row0, 0, smem_u32(&sm.qfull));
      }
      if (lane == 0) {
        sm.pages[j % kInfo] = valid;
        mbar_arrive1(&sm.info[j % kInfo]);
      }
      const uint32_t at = tails % kTails, use = tails / kTails;
      if (use > 0) ok = warp_wait(&sm.abort, &sm.tail_empty[at], (use - 1) & 1u);
      if (!ok) break;
      ++tails;
      if (lane == 0) mbar_expect_tx(&sm.tail_full[at], kSlotBlock);
      if (i < 1)
        load_box<1>(sm.tail[at] + first * 128, tm_k, (kBlocks - 1) * 64, yk, it.shard, smem_u32(&sm.tail_full[at]));
      for (int m = 0; m < 4; ++m, ++slot) {
        const uint32_t k = slot % kSlots, turn = slot / kSlots;
        if (turn > 0) ok = warp_wait(&sm.abort, &sm.empty[k], (turn - 1) & 1u);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&sm.full[k], kSlot);
        if (i < 2)
          load_box<1>(sm.kv[k] + i * kSlotBlock + first * 128, tm_k, (2 * m + i) * 64, yk, it.shard,
                      smem_u32(&sm.full[k]));
      }
    }
  }
  if (__any_sync(kFull, bad) && lane == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  if (!ok && lane == 0) {
    if (!cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
    // The copies issued land before the CTA ends.
    if (loads > 0) mbar_wait(&sm.qfull, (loads - 1) & 1u);
    for (uint32_t v = tails > kTails ? tails - kTails : 0; v < tails; ++v)
      mbar_wait(&sm.tail_full[v % kTails], (v / kTails) & 1u);
    for (uint32_t v = slot > kSlots ? slot - kSlots : 0; v < slot; ++v)
      mbar_wait(&sm.full[v % kSlots], (v / kSlots) & 1u);
  }
  __syncwarp();
}

template <int M>
__device__ __forceinline__ void narrow_products(const DecodeArgs& a, NarrowSmem<M>& sm, uint32_t tmem) {
  using Sm = NarrowSmem<M>;
  constexpr int N = Sm::N, kTails = Sm::kTails;
  const uint32_t id_s = idesc_f16(128, N, true, false) | a.negate;
  constexpr uint32_t id_o = idesc_f16(128, N, true, false) | kAcrossA;
  const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q), 16, 1024), p0 = smem_desc_sw128(smem_u32(sm.p), 16, 1024);
  const uint64_t k0 = smem_desc_sw128(smem_u32(sm.kv), 16, 1024), t0 = smem_desc_sw128(smem_u32(sm.tail), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(smem_u32(sm.kv), kSlotBlock, 1024);
  constexpr int kRow = N * 128 >> 4;         // a block of queries or weights in an address field
  Item it;
  uint32_t j = 0, nq = 0;                    // tiles, items' queries so far
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && warp_wait(&sm.abort, bar, parity);
    tc_fence_after();
    return ok;
  };
  // Scores of stream tile v with its slot m, the tile's last 64 dimensions before the first.
  auto scores = [&](uint32_t v, int m) {
    const uint32_t d = tmem + (v & 1u) * N, at = v % kTails, u = 4 * v + m, k = u % kSlots;
    if (m == 0) {
      if (!wait(&sm.tail_full[at], (v / kTails) & 1u)) return;
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_ss<1>(d, t0 + at * (kSlotBlock >> 4) + s * 2, q0 + (kBlocks - 1) * kRow + s * 2, id_s, s == 0 ? 0u : 1u);
        tc_commit<1>(&sm.tail_empty[at]);
      }
      __syncwarp();
    }
    if (!wait(&sm.full[k], (u / kSlots) & 1u)) return;
    if (elect_one()) {
      const uint64_t kd = k0 + k * (kSlot >> 4), qd = q0 + 2 * m * kRow;
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_ss<1>(d, kd + (s / 4) * (kSlotBlock >> 4) + (s % 4) * 2, qd + (s / 4) * kRow + (s % 4) * 2, id_s, 1u);
    }
    __syncwarp();
  };
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok, it); ++n) {
    item_done(sm.work, n);
    for (int t = it.t1 - 1; ok && t >= it.t0; --t, ++j) {
      const bool first = t == it.t1 - 1, last = t == it.t0;
      if (first && wait(&sm.qfull, nq++ & 1u)) scores(j, 0);
      for (int m = 1; ok && m < 4; ++m) scores(j, m);
      if (!ok) break;
      if (elect_one()) {
        tc_commit<1>(&sm.sfull[j & 1u]);
        if (last) tc_commit<1>(&sm.qempty);
      }
      __syncwarp();
      if (!last) scores(j + 1, 0);           // what the slots have room for, under this tile's softmax
      const int steps = value_steps<M>(it, t);
      if (!ok || !wait(&sm.pfull, j & 1u)) break;
      if (elect_one()) {
#pragma unroll 1
        for (uint32_t m = 0; m < 4; ++m) {
          const uint32_t k = (4 * j + m) % kSlots, d = tmem + 2 * N + m * N;
          const uint64_t vd = v0 + k * (kSlot >> 4);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (s < steps)
              mma_ss<1>(d, vd + s * (2048 >> 4), p0 + (s / 4) * kRow + (s % 4) * 2, id_o, (first && s == 0) ? 0u : 1u);
          tc_commit<1>(&sm.empty[k]);
        }
        tc_commit<1>(&sm.pvdone);
      }
      __syncwarp();
    }
  }
  if (!ok && (threadIdx.x & 31) == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
  __syncwarp();
  // Every product issued completes before the tensor memory is freed.
  if (elect_one()) {
    tc_commit<1>(&sm.drain);
    if (!mbar_wait(&sm.drain, 0)) cta_abort(&sm.abort, a.flags);
  }
  __syncwarp();
}

template <int M>
__device__ __forceinline__ void narrow_softmax(const DecodeArgs& a, NarrowSmem<M>& sm, uint32_t tmem, int warp) {
  constexpr int N = NarrowSmem<M>::N, kTile = Cut<M>::kTile;
  const int lane = threadIdx.x & 31, key = warp * 32 + lane;   // the thread's key of a tile; value of an output block
  const uint32_t t_s = tmem + ((uint32_t)(warp * 32) << 16), t_o = t_s + 2 * N;
  uint32_t j = 0, rounds = 0;                // tiles, exchanges so far
  bool ok = true;
  // A value a row, one after another, which lane 0 of each warp has written.
  auto exchange = [&](auto&& write) {
    float(*buf)[N] = sm.exchange[rounds & 1u];
    write(buf[warp]);
    __syncwarp();
    if (lane == 0) mbar_arrive1(&sm.exchanged);
    ok = warp_wait(&sm.abort, &sm.exchanged, rounds & 1u);
    ++rounds;
    return buf;
  };
  auto load_rows = [&](uint32_t at, uint32_t (&x)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 16) tmem_load(at + c, reinterpret_cast<uint32_t(&)[16]>(x[c]));
#pragma unroll
    for (int c = 0; c < N; c += 16) tmem_wait_ld(reinterpret_cast<uint32_t(&)[16]>(x[c]));
  };
  for (uint32_t n = 0; next_item(sm.work, &sm.abort, n, ok); ++n) {
    const Item& it = sm.work.item[n & 1u];   // read where it lies
    const int i0 = uni(it.t0), i1 = uni(it.t1), nall = uni(it.nall), nfree = uni(it.nfree);
    const int row0 = uni(it.row0), rows = uni(it.rows), tok0 = uni(it.tok0);
    float m[N], l[N];                        // the same m in every thread; l of the thread's keys
#pragma unroll
    for (int r = 0; r < N; ++r) m[r] = -INFINITY, l[r] = 0.f;
    for (int t = i1 - 1; t >= i0; --t, ++j) {
      ok = warp_wait(&sm.abort, &sm.sfull[j & 1u], (j >> 1) & 1u) &&
           warp_wait(&sm.abort, &sm.info[j % kInfo], (j / kInfo) & 1u);
      if (!ok) break;
      tc_fence_after();
      uint32_t x[N];
      load_rows(t_s + (j & 1u) * N, x);
      const uint32_t pages = *reinterpret_cast<volatile uint32_t*>(&sm.pages[j % kInfo]);
      if (pages != 0xffu || (t + 1) * kTile > nfree) {
        keep_branch();
        const int local = t * kTile + key;
        const bool there = ((piece_bits(a, pages, key >> 4) >> (key & 15)) & 1u) && local < nall;
        const int own = !there || local < nfree ? -1 : (int)a.sm.global_id(it.shard, (uint32_t)local) - it.base;
        if (__any_sync(kFull, own >= 0)) {
          keep_branch();
#pragma unroll
          for (int r = 0; r < N; ++r) {
            const int tok = (int)fdiv((uint32_t)(row0 + min(r, rows - 1)), a.fH);
            bool see = own <= tok;
            if (own >= 0 && a.mask)
              see = (own >> 5) < a.words &&
                    ((uint32_t)__ldg(a.mask + (int64_t)(tok0 + tok) * a.words + (own >> 5)) >> (own & 31)) & 1u;
            if (!see) x[r] = 0xff800000u;
          }
        }
#pragma unroll
        for (int r = 0; r < N; ++r) x[r] = there ? x[r] : 0xff800000u;
      }
      const auto top = exchange([&](float* mine) {
        float v[N];
#pragma unroll
        for (int r = 0; r < N; ++r) v[r] = warp_max(__uint_as_float(x[r]));
        if (lane == 0)
#pragma unroll
          for (int r = 0; r < N; r += 4)
            *reinterpret_cast<float4*>(mine + r) = make_float4(v[r], v[r + 1], v[r + 2], v[r + 3]);
      });
      if (!ok) break;
      // Rows r to r + 3: the tile's maxima, scaled.
      auto maxima = [&](int r, float (&mx)[4]) {
        float4 w[kNarrowWarps];
#pragma unroll
        for (int k = 0; k < kNarrowWarps; ++k) w[k] = *reinterpret_cast<const float4*>(&top[k][r]);
        mx[0] = fmaxf(fmax3(w[0].x, w[1].x, w[2].x), w[3].x) * a.c2;
        mx[1] = fmaxf(fmax3(w[0].y, w[1].y, w[2].y), w[3].y) * a.c2;
        mx[2] = fmaxf(fmax3(w[0].z, w[1].z, w[2].z), w[3].z) * a.c2;
        mx[3] = fmaxf(fmax3(w[0].w, w[1].w, w[2].w), w[3].w) * a.c2;
      };
      bool up = false;                       // some row's maximum is above its reference: alike in all threads
#pragma unroll
      for (int r = 0; r < N; r += 4) {
        float mx[4];
        maxima(r, mx);
#pragma unroll
        for (int e = 0; e < 4; ++e) up |= mx[e] > m[r + e] + kRescaleGap;   // m = -inf takes any finite maximum
      }
      if (t < i1 - 1) {                      // the last tile's values are in: weights and outputs are at rest
        ok = warp_wait(&sm.abort, &sm.pvdone, (j - 1) & 1u);
        if (!ok) break;
        tc_fence_after();
      }
      if (up) {
        keep_branch();
        float alpha[N];
#pragma unroll
        for (int r = 0; r < N; r += 4) {
          float mx[4];
          maxima(r, mx);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float old = m[r + e];
            if (mx[e] > old + kRescaleGap) m[r + e] = mx[e];
            alpha[r + e] = old == -INFINITY ? 1.f : fast_exp2(old - m[r + e]);
            l[r + e] *= alpha[r + e];
          }
        }
        if (t < i1 - 1) {
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t o[N];
            load_rows(t_o + b * N, o);
#pragma unroll
            for (int r = 0; r < N; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
#pragma unroll
            for (int c = 0; c < N; c += 16) tmem_store(t_o + b * N + c, reinterpret_cast<uint32_t(&)[16]>(o[c]));
          }
          tmem_wait_st();
        }
      }
      // The weights, rounded to bf16: row r's 64 keys of half key / 64 in 128 bytes,
      // its 16-byte pieces swizzled by r % 8.
      uint8_t* p = sm.p[key >> 6] + (key & 7) * 2;
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const float ref = m[r] == -INFINITY ? 0.f : m[r];
        const float e = fast_exp2(fmaf(__uint_as_float(x[r]), a.c2, -ref));
        l[r] += e;
        *reinterpret_cast<__nv_bfloat16*>(p + r * 128 + ((((key & 63) >> 3) ^ (r & 7)) << 4)) = __float2bfloat16_rn(e);
      }
      if (has_tail<M>(it, t)) {              // values behind the sequence's end: zeros
        const int past = nall - t * kTile, to = 16 * value_steps<M>(it, t);
        for (int z = key; z < (to - past) * 64; z += kNarrowWarps * 32) {
          const int k = past + z / 64, piece = z % 64;   // of 16 bytes
          uint8_t* block = sm.kv[(4 * j + (piece >> 4)) % kSlots] + ((piece >> 3) & 1) * kSlotBlock;
          *reinterpret_cast<uint4*>(block + k * 128 + (piece & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_async_smem();                    // read next by products
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.pfull);
    }
    if (!ok) break;
    const bool some = i1 > i0, parts = a.splits > 1;
    const int64_t to = ((int64_t)(parts ? it.split : 0) * a.sm.S + it.shard) * a.rows * a.H +
                       (int64_t)tok0 * a.H + row0;   // [splits][S][rows][H]
    float scale = 0.f, lse = -INFINITY;      // row lane's: 1 / its sum
    if (some) {
      const auto sums = exchange([&](float* mine) {
#pragma unroll
        for (int r = 0; r < N; ++r) {
          float v = l[r];
#pragma unroll
          for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
          if (lane == 0) mine[r] = v;
        }
      });
      if (ok) ok = warp_wait(&sm.abort, &sm.pvdone, (j - 1) & 1u);
      if (!ok) break;
      tc_fence_after();
      if (lane < N) {
        const float sum = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
        if (sum != 0.f) {                    // a NaN too
          scale = 1.f / sum;
          lse = log2f(sum);
        }
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < N; ++r)
        if (lane == r) lse += m[r] == -INFINITY ? 0.f : m[r];   // (-inf: no sum either)
    }
    if (warp == 0 && lane < rows) (parts ? a.part_l : a.lse2)[to + lane] = lse;
    if (some || !parts) {                    // the merge does not read an empty part
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t o[N];
        if (some) load_rows(t_o + b * N, o);
#pragma unroll
        for (int r = 0; r < N; ++r) {        // a row that saw nothing is zeros, whatever its column holds
          const float inv = __shfl_sync(kFull, scale, r);
          o[r] = inv == 0.f || !some ? 0u : __float_as_uint(__uint_as_float(o[r]) * inv);
        }
        if (parts) {
          float* at = a.part_o + to * kDv + b * 128 + key;
#pragma unroll
          for (int r = 0; r < N; ++r)
            if (r < rows) at[r * kDv] = __uint_as_float(o[r]);
        } else {
          // Lanes swap until each has four neighbouring values of every fourth row.
          const bool odd = (lane & 1) != 0, high = (lane & 2) != 0;
          uint16_t* at = reinterpret_cast<uint16_t*>(a.out) + to * kDv + b * 128 + (key & ~3);
#pragma unroll
          for (int r = 0; r < N; r += 4) {
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x0 = __uint_as_float(o[r + 2 * h]), x1 = __uint_as_float(o[r + 2 * h + 1]);
              const float x = __shfl_xor_sync(kFull, odd ? x0 : x1, 1);
              w[h] = odd ? pack16<true>(x, x1) : pack16<true>(x0, x);
            }
            const uint32_t x = __shfl_xor_sync(kFull, high ? w[0] : w[1], 2);
            const int row = r + (lane & 3);
            if (row < rows) *reinterpret_cast<uint2*>(at + row * kDv) = high ? make_uint2(x, w[1]) : make_uint2(w[0], x);
          }
        }
        __syncwarp();
      }
    }
    tc_fence_before();
    item_done(sm.work, n);
  }
  if (!ok && lane == 0 && !cta_aborted(&sm.abort)) cta_abort(&sm.abort, a.flags);
}

template <int M>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    mla_decode_narrow_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                             const DecodeArgs a) {
  using Sm = NarrowSmem<M>;
  constexpr uint32_t kCols = Sm::N == 16 ? 128 : 256;   // 6 N, as a power of two
  extern __shared__ unsigned char narrow_smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(narrow_smem_raw) + 1023) &
                                  ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = uni(tid >> 5);
  if (warp == kNarrowMma) {
    tmem_alloc<1>(&sm.tmem, kCols);
  } else if (warp == kNarrowClaim) {
    bool bad;
    const int blocks = count_blocks(a.starts, a.rows, nullptr, 0, a.reqs, a.H, Cut<M>::kItemRows, a.flags, bad);
    if ((tid & 31) == 0) sm.blocks = blocks, sm.bad = bad;
  } else if (tid == 0) {
    for (int b = 0; b < kSlots; ++b) {
      mbar_init(&sm.full[b], 1 + (b == 0 ? kStalledArrivals : 0));
      mbar_init(&sm.empty[b], 1);
    }
    for (int b = 0; b < Sm::kTails; ++b) {
      mbar_init(&sm.tail_full[b], 1);
      mbar_init(&sm.tail_empty[b], 1);
    }
    mbar_init(&sm.qfull, 1);
    mbar_init(&sm.qempty, 1);
    for (int b = 0; b < 2; ++b) mbar_init(&sm.sfull[b], 1);
    mbar_init(&sm.pfull, kNarrowWarps);
    mbar_init(&sm.pvdone, 1);
    mbar_init(&sm.exchanged, kNarrowWarps);
    for (int b = 0; b < kInfo; ++b) mbar_init(&sm.info[b], 1);
    mbar_init(&sm.drain, 1);
    init_slots(sm.work, 1, kNarrowWarps + 2);
    sm.abort = 0;
    mbar_init_fence();
  }
  if (a.ordered) longest_first(sm.order, a.reqs, tid, [&](int i) { return __ldg(a.lens + i); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uni(sm.tmem);
  if (warp < kNarrowWarps) {
    narrow_softmax<M>(a, sm, tmem, warp);
  } else if (warp == kNarrowLoad) {
    narrow_load<M>(a, sm, &tm_q, &tm_k);
  } else if (warp == kNarrowClaim) {
    const int blocks = sm.blocks;
    const bool bad = sm.bad != 0;
    Cursor cur;
    share_out<1>(sm.work, &sm.abort, a.flags, (int64_t)blocks * a.sm.S * a.splits, 0u,
                 [&](int64_t i) { return find_item<M>(a, sm.order, blocks, bad, i, cur); });
  } else {
    narrow_products<M>(a, sm, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kNarrowMma) {
    tc_fence_after();
    tmem_free<1>(tmem, kCols);
  }
}


constexpr int kNarrowMost = 32;
// How a call is cut: by the rows of a request (on average), and its keys into parts
// where items are few.  Lengths are the device's: the table's width stands for them, and
// one wider than the sequences makes parts that are not needed: the 64 requests below
// with 128 heads 354 us, 472 with a table of 65536 tokens or more (two parts); 64 of
// 2000 tokens on one shard 63, 138 with one of 32768 or more (seven).
// Rows of 64 requests, 8192 to 16384 tokens on 4 shards, in us: Narrow of 16 against
// 32 rows an item 201 / 227 (16 rows); Narrow against Wide 201 / 354 (16), 238 / 376
// (32), two items of it 397 / 392 (48), 413 / 410 (64), three 519 / 385 (96); Wide
// against Pair 584 / 492 (256), 1020 / 784 (512).
struct Plan {
  int mode, halves, item_rows, splits, ordered;
};
Plan plan_for(int rows, int S, int H, int reqs, int64_t cap) {
  const int64_t pairs = ((int64_t)rows * H + reqs - 1) / reqs;
  Plan p;
  p.mode = pairs > Cut<kWide>::kItemRows ? kPair : pairs > kNarrowMost ? kWide : pairs > 16 ? kNarrow32 : kNarrow16;
  p.halves = p.mode == kPair || p.mode == kWide ? 2 : 1;
  p.item_rows = p.mode == kPair ? Cut<kPair>::kItemRows : p.mode == kWide ? Cut<kWide>::kItemRows
                : p.mode == kNarrow32 ? Cut<kNarrow32>::kItemRows : Cut<kNarrow16>::kItemRows;
  const int64_t items = (pairs + p.item_rows - 1) / p.item_rows * reqs * p.halves * S;
  // 128 keys take a pair about 2.9 us (a half), a CTA alone 3.2 to 4.7; a part has as
  // many at least.
  const int64_t tiles = (cap + 127) / 128, ctas = kSms / (p.mode == kPair ? 2 : 1);
  p.splits = choose_parts(items, ctas, tiles * (p.mode == kPair ? 2.9 : 3.4) + 4.0, (int64_t)rows * S * H, kDv,
                          tiles);
  p.ordered = order_pays(reqs, items * p.splits, ctas);
  return p;
}

// Local tokens that a table row names, as far as the kernels count.
int64_t table_tokens(int max_blocks, int block_size) {
  return std::min<int64_t>((int64_t)max_blocks * block_size, (int64_t)1 << 30);
}

template <int M>
cudaError_t launch_decode(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const DecodeArgs& a, int64_t items, cudaStream_t stream) {
  const auto kernel = mla_decode_kernel<M>;
  constexpr int kSmem = (int)sizeof(DecodeSmem<M>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // An item a cluster; those that do not start at once are mostly taken over.
  const unsigned grid = (unsigned)(items * Shape<M>::CG);
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), (size_t)kSmem, stream,
                       Shape<M>::CG == 2 ? 2u : 0u, q, k, v, a);
}

template <int M>
cudaError_t launch_narrow(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap&, const DecodeArgs& a,
                          int64_t items, cudaStream_t stream) {
  const auto kernel = mla_decode_narrow_kernel<M>;
  constexpr int kSmem = (int)sizeof(NarrowSmem<M>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3((unsigned)items), dim3(kNarrowThreads), (size_t)kSmem, stream, 0u, q, k, a);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int64_t dsa_mla_decode_work(int rows, int S, int H, int reqs, int max_blocks,
                                       int block_size) {
  if (rows < 1 || S < 1 || H < 1 || reqs < 1 || max_blocks < 1 || block_size < 1) return 0;
  const int parts = plan_for(rows, S, H, reqs, table_tokens(max_blocks, block_size)).splits;
  return parts == 1 ? 0 : (int64_t)parts * S * rows * H * (kDv + 1) * 4;
}

extern "C" dsa_status dsa_mla_decode(const uint16_t* q, const uint16_t* kv_cache, int64_t n_slots,
                                     const int32_t* block_table, int reqs, int max_blocks,
                                     int block_size, const int32_t* query_starts,
                                     const int32_t* seq_lens, const int32_t* tree_mask,
                                     int mask_words, int rows, int S, int I, int H, float scale,
                                     uint16_t* out, float* lse2, float* work, uint32_t* err_flags,
                                     cudaStream_t stream) {
  if (rows < 0 || reqs < 0 || H < 1 || max_blocks < 1 || block_size < 1 || n_slots < 1 ||
      (tree_mask && mask_words < 1) || !(scale == scale) || isinf(scale))
    return DSA_ERR_INVALID_ARG;
  if (S < 1 || S > DSA_MAX_SHARDS || I < 1 || (int64_t)I * S > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size % 64) return DSA_ERR_UNSUPPORTED;
  if (rows == 0 || reqs == 0) return DSA_OK;
  if (!q || !kv_cache || !block_table || !query_starts || !seq_lens || !out || !lse2)
    return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out) || !aligned16(work))
    return DSA_ERR_INVALID_ARG;
  const int64_t pairs = (int64_t)rows * H;
  if (n_slots > INT32_MAX || pairs > ((int64_t)1 << 30) || (int64_t)S * reqs > ((int64_t)1 << 30))
    return DSA_ERR_UNSUPPORTED;
  const int64_t cap = table_tokens(max_blocks, block_size);
  Plan p = plan_for(rows, S, H, reqs, cap);
  if (!work) p.splits = 1;
  const int64_t outs = S * pairs;
  if (!apart({bytes_of(out, outs * kDv * 2), bytes_of(lse2, outs * 4),
              bytes_of(p.splits > 1 ? work : nullptr, p.splits * outs * (kDv + 1) * 4)},
             {bytes_of(q, pairs * kDqk * 2), bytes_of(kv_cache, S * n_slots * kDqk * 2),
              bytes_of(block_table, (int64_t)S * reqs * max_blocks * 4), bytes_of(query_starts, ((int64_t)reqs + 1) * 4),
              bytes_of(seq_lens, (int64_t)reqs * 4), bytes_of(tree_mask, (int64_t)rows * mask_words * 4)}))
    return DSA_ERR_INVALID_ARG;
  DecodeArgs a{reinterpret_cast<const __nv_bfloat16*>(q), block_table, query_starts, seq_lens, tree_mask, reinterpret_cast<__nv_bfloat16*>(out),
               lse2, nullptr, nullptr, err_flags, n_slots, reqs, max_blocks, block_size, rows, H,
               mask_words, p.splits, p.ordered, (int)cap, std::min(block_size, 64), std::min(block_size, (int)Shape<kPair>::kVKeys),
               scale == 0.f ? 0x1p-100f : fabsf(scale) * kLog2e, scale < 0.f ? kNegateA : 0u,
               ShardMath(S, I), FastDiv(block_size), FastDiv(H)};
  if (p.splits > 1) {
    a.part_o = work;
    a.part_l = work + (int64_t)p.splits * S * pairs * kDv;
  }
  CUtensorMap tq, tk, tv;
  const uint64_t row = kDqk * 2;
  if (!encode_map16(&tq, q, true, kDqk, pairs, 1, row, row * pairs, std::min(p.item_rows, kQBox), 1) ||
      !encode_map16(&tk, kv_cache, true, kDqk, n_slots, S, row, row * n_slots, a.kbox, 1) ||
      !encode_map16(&tv, kv_cache, true, kDqk, n_slots, S, row, row * n_slots, a.vbox, 1))
    return DSA_ERR_CUDA;
  // At most: a request's pairs are a multiple of H, so that its last block has a
  // common divisor at least.  (Clusters without an item have to be cancelled too.)
  const int64_t blocks = (pairs + (int64_t)reqs * (p.item_rows - std::gcd(H, p.item_rows))) / p.item_rows;
  const int64_t items = blocks * p.halves * S * p.splits;
  if (items * 2 > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  const auto launch = p.mode == kPair ? launch_decode<kPair> : p.mode == kWide ? launch_decode<kWide>
                      : p.mode == kNarrow32 ? launch_narrow<kNarrow32> : launch_narrow<kNarrow16>;
  const cudaError_t e = launch(tq, tk, tv, a, items, stream);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  if (p.splits > 1) {
    const MergeArgs m{a.part_o, a.part_l, p.splits, S * pairs, query_starts, reqs, rows, H, out, lse2};
    if (launch_merge<kDv, true>(m, stream) != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}
