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
// has to be requantised.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kDc = DSA_MLA_DV;                // 512 latent values
constexpr int kRow = DSA_MLA_DQK;              // 576 codes of a row
constexpr int kDr = kRow - kDc;                // 64 rope values
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeld = 8;                       // rows that a warp keeps in registers
constexpr int kMaxBlock = 1024;                // slots of a block
constexpr int kTokensPerCta = 8;               // tokens whose blocks a CTA looks after

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

// The larger magnitude of two packed bf16, as bits (the order of magnitudes);
// infinities and NaN count as 0.
__device__ __forceinline__ uint32_t pair_amax(uint32_t w) {
  const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  return max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u);
}

__device__ __forceinline__ uint32_t row_amax(const RowRegs& r) {
  uint32_t m = pair_amax(r.p);
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, pair_amax(w[i]));
  return m;
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

__device__ __forceinline__ uint32_t encode2(uint32_t w, float scale, float inv) {
  const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
  return inv != 0.f ? codes2(lo * inv, hi * inv) : codes2(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale));
}

__device__ __forceinline__ void store_row(const InsertArgs& a, int64_t slot, const RowRegs& r,
                                          float scale, float inv, int lane) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = encode2(w[2 * i], scale, inv) | (encode2(w[2 * i + 1], scale, inv) << 16);
  uint8_t* dst = a.cache + slot * kRow;
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
  reinterpret_cast<uint16_t*>(dst + kDc)[lane] = (uint16_t)encode2(r.p, scale, inv);
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

__device__ __forceinline__ void requantise_row(const InsertArgs& a, int64_t slot, float ratio,
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

// One cache block b: row_tok[r] = 1 + the token of its row r, 0 for a row that
// stays.  Every thread of the CTA calls it.  Rows up to kHeld a warp are kept
// in registers between the maximum and the store; a larger block's are read
// again (from L2).
__device__ __forceinline__ void write_block(const InsertArgs& a, int b, const int* row_tok,
                                            uint32_t* warp_max) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t slot0 = (int64_t)b * a.block;
  const float held = a.scales[b];
  const float old = held > 0.f ? held : 0.f;
  RowRegs regs[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int r = warp + k * kWarps;
    if (r < a.block && row_tok[r] != 0) regs[k] = load_row(a, row_tok[r] - 1, lane);
    else regs[k] = RowRegs{};
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) m = max(m, row_amax(regs[k]));
  for (int r = warp + kHeld * kWarps; r < a.block; r += kWarps)
    if (row_tok[r] != 0) m = max(m, row_amax(load_row(a, row_tok[r] - 1, lane)));
  m = __reduce_max_sync(kFull, m);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = max(m, warp_max[w]);
  const float scale = fmaxf(old, scale_for(m));
  if (threadIdx.x == 0 && !(held == scale)) a.scales[b] = scale;
  // 1 / scale where that is exact (a power of two), else 0: divide.
  const float div = scale > 0.f ? scale : 1.f;
  const float inv = (__float_as_uint(div) & 0x7FFFFFu) == 0 ? 1.f / div : 0.f;
  const bool grown = old > 0.f && scale > old;
  const float ratio = __fdiv_rn(old, div);
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int r = warp + k * kWarps;
    if (r >= a.block) continue;
    if (row_tok[r] != 0) store_row(a, slot0 + r, regs[k], div, inv, lane);
    else if (grown) requantise_row(a, slot0 + r, ratio, lane);
  }
  for (int r = warp + kHeld * kWarps; r < a.block; r += kWarps) {
    if (row_tok[r] != 0) store_row(a, slot0 + r, load_row(a, row_tok[r] - 1, lane), div, inv, lane);
    else if (grown) requantise_row(a, slot0 + r, ratio, lane);
  }
}

// Few tokens: one kernel, no workspace.  CTA t looks through the call's slots
// for the rows of its token's block; the block's first token does the work.
__global__ void __launch_bounds__(kThreads) insert_few_kernel(const InsertArgs a) {
  __shared__ int row_tok[kMaxBlock];
  __shared__ uint32_t warp_max[kWarps];
  const int t = blockIdx.x;
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
// hold anything before: one counts only if the token it names has that slot
// (that block).
__global__ void __launch_bounds__(kThreads) insert_claim_kernel(const InsertArgs a) {
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.T) return;
  const int slot = __ldg(a.slots + t);
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    raise_flag(a.flags, DSA_FLAG_BOUNDS);
    return;
  }
  auto names = [&](int word) { return word >= 1 && word <= a.T; };
  int cur = *const_cast<volatile int32_t*>(a.owner + slot);
  while (!(names(cur) && __ldg(a.slots + cur - 1) == slot && cur > t)) {
    const int seen = atomicCAS(a.owner + slot, cur, t + 1);
    if (seen == cur) break;
    cur = seen;
  }
  const int b = (int)fdiv((uint32_t)slot, a.fblock);
  const int base = b * a.block;
  cur = *const_cast<volatile int32_t*>(a.leader + b);
  for (;;) {
    if (names(cur)) {
      const int other = __ldg(a.slots + cur - 1);
      if (other >= base && other - base < a.block) break;
    }
    const int seen = atomicCAS(a.leader + b, cur, t + 1);
    if (seen == cur) break;
    cur = seen;
  }
}

// The second writes the blocks: a CTA looks at kTokensPerCta tokens and takes
// the blocks that they lead.
__global__ void __launch_bounds__(kThreads) insert_many_kernel(const InsertArgs a) {
  __shared__ int row_tok[kMaxBlock];
  __shared__ uint32_t warp_max[kWarps];
  const int t0 = blockIdx.x * kTokensPerCta;
  int lead[kTokensPerCta];
#pragma unroll
  for (int i = 0; i < kTokensPerCta; ++i) {
    const int slot = t0 + i < a.T ? __ldg(a.slots + t0 + i) : -1;
    lead[i] = slot >= 0 && slot < a.n_slots ? (int)fdiv((uint32_t)slot, a.fblock) : -1;
  }
#pragma unroll
  for (int i = 0; i < kTokensPerCta; ++i)
    if (lead[i] >= 0 && a.leader[lead[i]] != t0 + i + 1) lead[i] = -1;
#pragma unroll 1
  for (int i = 0; i < kTokensPerCta; ++i) {
    const int b = lead[i];
    if (b < 0) continue;
    const int base = b * a.block;
    for (int r = threadIdx.x; r < a.block; r += kThreads) {
      const int o = a.owner[base + r];
      row_tok[r] = o >= 1 && o <= a.T && __ldg(a.slots + o - 1) == base + r ? o : 0;
    }
    __syncthreads();
    write_block(a, b, row_tok, warp_max);
    __syncthreads();
  }
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
  const InsertArgs a{kv_rows,  kpe_rows, slot_mapping, kv_cache, block_scales, work,
                     work ? work + n_slots : nullptr, err_flags, T, (int)n_slots, block_tokens,
                     FastDiv((uint32_t)block_tokens)};
  cudaError_t e;
  if (T <= DSA_INSERT_FP8_SMALL) {
    e = launch_kernel(insert_few_kernel, dim3((unsigned)T), dim3(kThreads), 0, stream, 0u, a);
  } else {
    e = launch_kernel(insert_claim_kernel, dim3((unsigned)((T + kThreads - 1) / kThreads)),
                      dim3(kThreads), 0, stream, 0u, a);
    if (e == cudaSuccess)
      e = launch_kernel(insert_many_kernel,
                        dim3((unsigned)((T + kTokensPerCta - 1) / kTokensPerCta)), dim3(kThreads),
                        0, stream, 0u, a);
  }
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
