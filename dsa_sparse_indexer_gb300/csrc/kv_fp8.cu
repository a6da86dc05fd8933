// New rows into an 8-bit MLA cache with a scale for each block of slots
// (sm_103a).
//
// A row is 576 bf16 values in and 576 e4m3 codes out; its scale belongs to a
// block of block_tokens slots.  Scales are powers of two: a division by one is
// exact, so a code is the value rounded once, and when a later, larger row
// raises a block's scale, the codes already there move by whole binades
// (exact but for values that drop below the format's smallest step).  The
// work is by block, so that a block's scale is decided once: a thread block
// ("CTA" below) takes one cache block with all rows that the call writes to
// it, reads them once, and writes their codes.  No result depends on the order
// of atomics: of several tokens with one slot the last is written, as if the
// rows had been inserted one after another.
//
// Bound by memory: 1152 + 576 bytes a token, and twice 576 for every row that
// has to be requantised; small calls by a launch's latency (64 tokens 3.0 us).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kDc = DSA_MLA_DV;                // 512 latent values
constexpr int kRow = DSA_MLA_DQK;              // 576 codes of a row
constexpr int kDr = kRow - kDc;                // 64 rope values
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kHeld = 4;                       // rows that a warp keeps in registers
constexpr int kMaxBlock = 1024;                // slots of a block
constexpr int kTokensPerCta = 64;              // tokens whose blocks a CTA looks after, at most
constexpr int kSms = 152;                      // of a GB300
constexpr int kAlone = 32;                     // new rows of a block that a warp takes alone

struct InsertArgs {
  const uint16_t* kv;
  const uint16_t* kpe;
  const int32_t* slots;
  uint8_t* cache;
  float* scales;
  int32_t* owner;           // [n_slots] 1 + the token written to a slot (large calls)
  int32_t* leader;          // [blocks] 1 + a token of the block
  uint32_t* flags;
  int T, n_slots, block;
  int each;                 // tokens whose blocks a CTA looks after
  FastDiv fblock;
};

// A token's row: 16 latent values and 2 rope values a lane.
struct RowRegs {
  uint4 a, b;
  uint32_t p;
};

__device__ __forceinline__ RowRegs load_row(const InsertArgs& a, int t, int lane) {
  RowRegs r;
  const uint4* src = reinterpret_cast<const uint4*>(a.kv + (int64_t)t * kDc) + 2 * lane;
  r.a = __ldg(src);
  r.b = __ldg(src + 1);
  r.p = __ldg(reinterpret_cast<const uint32_t*>(a.kpe + (int64_t)t * kDr) + lane);
  return r;
}

// The row's largest magnitude in this lane, as bf16 bits (which order
// magnitudes), two values at a time; infinities and NaN count as 0.
__device__ __forceinline__ uint32_t finite(uint32_t w) {
  const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  return max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u);
}
// Read again: the common path keeps its rows in registers.
__device__ __noinline__ uint32_t row_amax_finite(const InsertArgs& a, int t, int lane) {
  const RowRegs r = load_row(a, t, lane);
  const uint32_t w[9] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w, r.p};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 9; ++i) m = max(m, finite(w[i]));
  return m;
}
__device__ __forceinline__ uint32_t row_amax(const InsertArgs& a, const RowRegs& r, int t, int lane) {
  const uint32_t w[9] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w, r.p};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 9; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  return m < 0x7F80u ? m : row_amax_finite(a, t, lane);
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 2^8)
// for amax = 1.f 2^e given as bf16 bits; 0 for 0.
__device__ __forceinline__ float scale_for(uint32_t amax) {
  if (amax == 0) return 0.f;
  const int e = (int)(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 0x60u);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t encode2(uint32_t w, float inv) {
  return codes2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xFFFF0000u) * inv);
}

// The row's codes, for a scale that is a power of two (the product with its
// inverse is the quotient).
__device__ __forceinline__ void store_row(const InsertArgs& a, int64_t slot, const RowRegs& r,
                                          float inv, int lane) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = encode2(w[2 * i], inv) | (encode2(w[2 * i + 1], inv) << 16);
  uint8_t* dst = a.cache + slot * kRow;
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
  reinterpret_cast<uint16_t*>(dst + kDc)[lane] = (uint16_t)encode2(r.p, inv);
}

// Any other scale (another quantiser's): token t's row divided by it.
__device__ __noinline__ void store_row_divided(const InsertArgs& a, int64_t slot, int t, float scale) {
  uint8_t* dst = a.cache + slot * kRow;
  for (int i = threadIdx.x & 31; i < kRow / 2; i += 32) {
    const uint32_t w = i < kDc / 2
                           ? __ldg(reinterpret_cast<const uint32_t*>(a.kv + (int64_t)t * kDc) + i)
                           : __ldg(reinterpret_cast<const uint32_t*>(a.kpe + (int64_t)t * kDr) + i - kDc / 2);
    reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)codes2(
        __fdiv_rn(__uint_as_float(w << 16), scale), __fdiv_rn(__uint_as_float(w & 0xFFFF0000u), scale));
  }
}

// Four codes times `ratio`, rounded once more.
__device__ __forceinline__ uint32_t requantise4(uint32_t c, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    out |= codes2(f.x * ratio, f.y * ratio) << (16 * i);
  }
  return out;
}

__device__ __noinline__ void requantise_row(const InsertArgs& a, int64_t slot, float ratio,
                                               int lane) {
  uint4* row = reinterpret_cast<uint4*>(a.cache + slot * kRow);
  for (int i = lane; i < kRow / 16; i += 32) {
    uint4 v = row[i];
    v.x = requantise4(v.x, ratio);
    v.y = requantise4(v.y, ratio);
    v.z = requantise4(v.z, ratio);
    v.w = requantise4(v.w, ratio);
    row[i] = v;
  }
}

// What a block's new rows make of its scale.
struct BlockScale {
  float div, inv, ratio;    // the divisor; 1 / div where exact (a power of two), else 0; old / div
  bool grown;               // rows that stay are requantised
};
__device__ __forceinline__ BlockScale block_scale(const InsertArgs& a, int b, float held,
                                                  uint32_t amax, bool writer) {
  const float old = held > 0.f ? held : 0.f, scale = fmaxf(old, scale_for(amax));
  if (writer && !(held == scale)) a.scales[b] = scale;
  BlockScale s;
  s.div = scale > 0.f ? scale : 1.f;
  s.inv = (__float_as_uint(s.div) & 0x7FFFFFu) == 0 ? 1.f / s.div : 0.f;
  s.ratio = __fdiv_rn(old, s.div);
  s.grown = old > 0.f && scale > old;
  return s;
}

// One cache block b: row_tok[r] = 1 + the token of its row r, 0 for a row that
// stays.  Every thread of the CTA calls it.  Rows up to kHeld a warp are kept
// in registers between the maximum and the store; a larger block's are read
// again (from L2).
__device__ __forceinline__ void write_block(const InsertArgs& a, int b, const int* row_tok,
                                            uint32_t* warp_max) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t slot0 = (int64_t)b * a.block;
  const float held = a.scales[b];
  RowRegs regs[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int r = warp + k * kWarps;
    if (r < a.block && row_tok[r] != 0) regs[k] = load_row(a, row_tok[r] - 1, lane);
    else regs[k] = RowRegs{};
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int r = warp + k * kWarps;
    if (r < a.block && row_tok[r] != 0) m = max(m, row_amax(a, regs[k], row_tok[r] - 1, lane));
  }
  for (int r = warp + kHeld * kWarps; r < a.block; r += kWarps)
    if (row_tok[r] != 0)
      m = max(m, row_amax(a, load_row(a, row_tok[r] - 1, lane), row_tok[r] - 1, lane));
  m = __reduce_max_sync(kFull, m);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = max(m, warp_max[w]);
  const BlockScale sc = block_scale(a, b, held, m, threadIdx.x == 0);
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int r = warp + k * kWarps;
    if (r >= a.block) continue;
    if (row_tok[r] != 0 && sc.inv != 0.f) store_row(a, slot0 + r, regs[k], sc.inv, lane);
  }
  for (int r = warp + kHeld * kWarps; r < a.block; r += kWarps)
    if (row_tok[r] != 0 && sc.inv != 0.f)
      store_row(a, slot0 + r, load_row(a, row_tok[r] - 1, lane), sc.inv, lane);
  if (sc.inv != 0.f && !sc.grown) return;
  for (int r = warp; r < a.block; r += kWarps) {
    if (row_tok[r] == 0 && sc.grown) requantise_row(a, slot0 + r, sc.ratio, lane);
    if (row_tok[r] != 0 && sc.inv == 0.f) store_row_divided(a, slot0 + r, row_tok[r] - 1, sc.div);
  }
}

// The token that row `slot` gets from this call, plus 1; 0 for none (large calls).
__device__ __forceinline__ int owner_of(const InsertArgs& a, int slot) {
  const int o = a.owner[slot];
  return o >= 1 && o <= a.T && __ldg(a.slots + o - 1) == slot ? o : 0;
}

// A block with up to kAlone new rows, by one warp: several at a time in a CTA
// when the call's tokens are spread over many blocks.  `list` is the warp's
// space for the rows and their tokens.  Four rows are kept in registers, more
// are read again for the store (from L2): 16384 scattered tokens into 131072
// slots of blocks of 64 take 27 us, and 70 if all CTAs take blocks of more than
// four rows together.  False: more rows.
__device__ __forceinline__ bool write_block_alone(const InsertArgs& a, int b, int2* list) {
  const int lane = threadIdx.x & 31;
  const int64_t slot0 = (int64_t)b * a.block;
  const float held = a.scales[b];
  int n = 0;
  for (int r0 = 0; r0 < a.block; r0 += 32) {
    const int tok = r0 + lane < a.block ? owner_of(a, (int)slot0 + r0 + lane) : 0;
    const unsigned there = __ballot_sync(kFull, tok != 0);
    if (n + __popc(there) > kAlone) return false;
    if (tok != 0) list[n + __popc(there & lanemask_lt())] = make_int2(r0 + lane, tok - 1);
    n += __popc(there);
  }
  __syncwarp();
  RowRegs regs[kHeld];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) regs[i] = i0 + i < n ? load_row(a, list[i0 + i].y, lane) : RowRegs{};
  };
  uint32_t m = 0;
  for (int i0 = 0; i0 < n; i0 += kHeld) {
    load(i0);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i0 + i < n) m = max(m, row_amax(a, regs[i], list[i0 + i].y, lane));
  }
  const BlockScale sc = block_scale(a, b, held, __reduce_max_sync(kFull, m), lane == 0);
  for (int i0 = 0; i0 < n; i0 += kHeld) {
    if (n > kHeld) load(i0);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i0 + i < n) {
        const int2 e = list[i0 + i];
        if (sc.inv != 0.f) store_row(a, slot0 + e.x, regs[i], sc.inv, lane);
        else store_row_divided(a, slot0 + e.x, e.y, sc.div);
      }
  }
  if (sc.grown) {
    const int mine = lane < n ? list[lane].x : -1;
    for (int r = 0; r < a.block; ++r)
      if (!__any_sync(kFull, mine == r)) requantise_row(a, slot0 + r, sc.ratio, lane);
  }
  __syncwarp();                              // the list is free
  return true;
}

// Few tokens: one kernel, no workspace.  CTA t looks through the call's slots
// for the rows of its token's block; the block's first token does the work.
__global__ void __launch_bounds__(kThreads) insert_few_kernel(const __grid_constant__ InsertArgs a) {
  __shared__ int row_tok[kMaxBlock];
  __shared__ uint32_t warp_max[kWarps];
  const int t = blockIdx.x;
  // The row is on its way to L2 while its block is looked up.
  if (threadIdx.x < 10) {
    const char* row = threadIdx.x < 8 ? reinterpret_cast<const char*>(a.kv + (int64_t)t * kDc) + threadIdx.x * 128
                                      : reinterpret_cast<const char*>(a.kpe + (int64_t)t * kDr) + (threadIdx.x - 8) * 64;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
  }
  const int slot = __ldg(a.slots + t);
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (threadIdx.x == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
    return;
  }
  const int b = (int)fdiv((uint32_t)slot, a.fblock);
  const int base = b * a.block;
  for (int r = threadIdx.x; r < a.block; r += kThreads) row_tok[r] = 0;
  __syncthreads();
  bool earlier = false;
  for (int u = threadIdx.x; u < a.T; u += kThreads) {
    const int other = __ldg(a.slots + u);
    if (other >= base && other - base < a.block) {
      atomicMax(&row_tok[other - base], u + 1);
      earlier |= u < t;
    }
  }
  if (__syncthreads_or(earlier)) return;
  write_block(a, b, row_tok, warp_max);
}

// Many tokens: the first kernel writes, for every slot, the last token that
// names it, and for every block one token that looks after it.  The words may
// hold anything before: one counts only if the token it names has that slot.
__global__ void __launch_bounds__(kThreads) insert_claim_kernel(const __grid_constant__ InsertArgs a) {
  int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.T) return;
  const int slot = __ldg(a.slots + t);
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    raise_flag(a.flags, DSA_FLAG_BOUNDS);
    return;
  }
  a.leader[fdiv((uint32_t)slot, a.fblock)] = t + 1;   // whichever is left names the block
  // The token's own number takes the slot's place; a later token's that it finds
  // there, it puts back, unless a still later one has come.
  int* owner = a.owner + slot;
  auto later = [&](int word) {
    return word > t + 1 && word <= a.T && __ldg(a.slots + word - 1) == slot;
  };
  int seen = atomicExch(owner, t + 1);
  while (later(seen)) {
    t = seen - 1;
    seen = atomicExch(owner, t + 1);
  }
}

// The second writes the blocks: a CTA looks at some tokens and takes the blocks
// that they lead, first those of few rows, a warp each, then the others
// together.  Their number gives every SM a CTA, from 16 on (2048 scattered
// tokens: 17.5 us with 64 each, 9.3 with 16) up to 64 (16384 tokens of a
// prompt: 13.7 us with 16 each, 9.4 with 64).
__global__ void __launch_bounds__(kThreads, 2) insert_many_kernel(const __grid_constant__ InsertArgs a) {
  __shared__ int row_tok[kMaxBlock];
  __shared__ uint32_t warp_max[kWarps];
  __shared__ int lead[kTokensPerCta], large[kTokensPerCta], n_lead, n_large;
  __shared__ int2 list[kWarps][kAlone];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) n_large = 0;
  // Neighbouring tokens mostly share blocks: their rows are on their way to L2
  // while the blocks are looked up.
  const int t0 = blockIdx.x * a.each, mine = min(a.each, a.T - t0);
  for (int i = threadIdx.x; i < mine * 9; i += kThreads) {
    const char* row = i < mine * 8 ? reinterpret_cast<const char*>(a.kv + (int64_t)t0 * kDc) + i * 128
                                   : reinterpret_cast<const char*>(a.kpe + (int64_t)t0 * kDr) + (i - mine * 8) * 128;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
  }
  if (warp == 0) {
    int n = 0;
    for (int i = lane; i < kTokensPerCta; i += 32) {
      const int t = t0 + i;
      const int slot = i < mine ? __ldg(a.slots + t) : -1;
      const int b = slot >= 0 && slot < a.n_slots ? (int)fdiv((uint32_t)slot, a.fblock) : -1;
      const bool leads = b >= 0 && a.leader[b] == t + 1;
      const unsigned all = __ballot_sync(kFull, leads);
      if (leads) lead[n + __popc(all & lanemask_lt())] = b;
      n += __popc(all);
    }
    if (lane == 0) n_lead = n;
  }
  __syncthreads();
  // (One or two blocks hold many rows each, as in a prompt, or nothing is lost.)
  if (n_lead > 2) {
    for (int i = warp; i < n_lead; i += kWarps)
      if (!write_block_alone(a, lead[i], list[warp]) && lane == 0) large[atomicAdd(&n_large, 1)] = lead[i];
  } else if (threadIdx.x == 0) {
    for (n_large = 0; n_large < n_lead; ++n_large) large[n_large] = lead[n_large];
  }
  __syncthreads();
  for (int i = 0; i < n_large; ++i) {
    const int b = large[i], base = b * a.block;
    for (int r = threadIdx.x; r < a.block; r += kThreads) row_tok[r] = owner_of(a, base + r);
    __syncthreads();
    write_block(a, b, row_tok, warp_max);
    __syncthreads();
  }
}

// Or a CTA takes each block of the cache and looks whether it has a token: no
// CTA has a block more than another, and of a CTA's few loads none waits for a
// list.  For calls of at least a quarter of the cache's slots, whose untouched
// blocks are few, and eight tokens a block (or about as many blocks as CTAs fit
// at a time).  32768 tokens, a tenth left out, into 65536 slots of blocks of
// 64 (56 MB; replays, in L2): in a prompt's order 11.7 us, by the tokens' CTAs
// above 14.5; in any order 16.3 and 55.  At the
// lower bound a prompt's order loses a little (16384 into 65536 of blocks of 64
// 10.2 us, above 9.4) for what any order gains.  Past the bounds it loses: 8192
// into 65536 of blocks of 128 11.1 us, above 9.8; 16384 into 65536 of blocks
// of 16 17.7, above 12.4.
__global__ void __launch_bounds__(kThreads, 2) insert_blocks_kernel(const __grid_constant__ InsertArgs a) {
  __shared__ int row_tok[kMaxBlock];
  __shared__ uint32_t warp_max[kWarps];
  const int b = blockIdx.x, base = b * a.block;
  const int o = a.leader[b];
  for (int r = threadIdx.x; r < a.block; r += kThreads) row_tok[r] = owner_of(a, base + r);
  if (o < 1 || o > a.T) return;
  const int slot = __ldg(a.slots + o - 1);
  if (slot < base || slot - base >= a.block) return;   // the CTA alike
  __syncthreads();
  write_block(a, b, row_tok, warp_max);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_kv_cache_insert_fp8(const uint16_t* kv_rows, const uint16_t* kpe_rows,
                                              const int32_t* slot_mapping, int T,
                                              uint8_t* kv_cache, float* block_scales,
                                              int64_t n_slots, int block_tokens, int32_t* work,
                                              uint32_t* err_flags, cudaStream_t stream) {
  if (T < 0 || n_slots < 1 || block_tokens < 1 || n_slots % block_tokens) return DSA_ERR_INVALID_ARG;
  if (block_tokens > kMaxBlock || n_slots > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!kv_rows || !kpe_rows || !slot_mapping || !kv_cache || !block_scales ||
      (T > DSA_INSERT_FP8_SMALL && !work))
    return DSA_ERR_INVALID_ARG;
  if (!aligned16(kv_rows) || !aligned16(kpe_rows) || !aligned16(kv_cache)) return DSA_ERR_INVALID_ARG;
  const int64_t n_blocks = n_slots / block_tokens;
  int each = 16;
  while (each < kTokensPerCta && (int64_t)each * kSms < T) each *= 2;
  const InsertArgs a{kv_rows,
                     kpe_rows,
                     slot_mapping,
                     kv_cache,
                     block_scales,
                     work,
                     work ? work + n_slots : nullptr,
                     err_flags,
                     T,
                     (int)n_slots,
                     block_tokens,
                     each,
                     FastDiv((uint32_t)block_tokens)};
  cudaError_t e;
  if (T <= DSA_INSERT_FP8_SMALL) {
    e = launch_kernel(insert_few_kernel, dim3((unsigned)T), dim3(kThreads), 0, stream, 0u, a);
  } else {
    e = launch_kernel(insert_claim_kernel, dim3((unsigned)((T + kThreads - 1) / kThreads)),
                      dim3(kThreads), 0, stream, 0u, a);
    if (e == cudaSuccess && n_slots / 4 <= T && n_blocks <= std::max(T / 8, 4 * kSms))
      e = launch_kernel(insert_blocks_kernel, dim3((unsigned)n_blocks), dim3(kThreads), 0, stream,
                        0u, a);
    else if (e == cudaSuccess)
      e = launch_kernel(insert_many_kernel, dim3((unsigned)((T + each - 1) / each)),
                        dim3(kThreads), 0, stream, 0u, a);
  }
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
