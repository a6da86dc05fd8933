// The 8-bit operands of the indexer's logits: keys into the paged key cache,
// queries with their scales folded into the head weights (sm_103a).
//
// Key: y = (k - mean) / sqrt(var + eps) * weight + bias over its 128 values, the
// values [first, first + rot) turned by the position's row of the table, e4m3
// codes (round to nearest even, saturating) to the token's slot.  Query: each
// head's 128 values turned alike, code = e4m3(y / s) with s the smallest power
// of two with max |y| <= 448 s, and the head's weight times factor * s.
//
// Memory-bound: 256 bytes in and 128 out a row, and the arithmetic close behind
// (an issue slot of 16 a value is what the bandwidth leaves).  Sixteen lanes take a
// row, eight values (16 bytes) each, so that sums and maxima are four shuffles.
// Where a value's partner lies decides how it is fetched: in the same lane
// (interleaved pairs at an even offset), in a lane a fixed way off (the half layout
// at multiples of 8), or anywhere, through shared memory.  A thread finds its cosines
// and sines once and uses them for all heads it takes.
// Queries round as the exact values do: a scaled value within the arithmetic's error
// of a middle between two codes, a largest one near a border between two scales, or a
// head below 2^-60, sends its head once more through the arithmetic, with its errors.
// Infinities saturate; a value that turns past fp32's range is finite all the same.
// Measured: 64 keys into 4 shards 4.3 us, 32768 keys 12.4 us and 131072 35.7 (86 MB,
// 2.4 TB/s: the issue slots of norm, rotation and stores); the queries of 64 tokens,
// 64 heads 6.3 us, of 4096 tokens 40 us (104 MB, 2.6 TB/s: the issue slots of
// rotation, scale and rounding).  Two or four keys a thread, its weights read once:
// 32768 keys 10.7 and 13.3 us where one takes 10.0, back to back.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "regions.h"

namespace dsa {
namespace {

constexpr int kDim = DSA_IDX_DIM;            // 128
constexpr int kLanes = 16, kVals = kDim / kLanes;
constexpr int kThreads = 128, kRows = kThreads / kLanes;   // rows in a block at a time

struct TurnArgs {
  const int32_t* positions;
  const float* table;                        // [max_pos][rot]
  int max_pos, rot, first, layout;
  uint32_t* flags;
};

enum Partner { kInLane, kLaneOff, kAnywhere };

// How this lane's eight values turn: y_e = x_e cos_e + x_partner sin_e, partner
// the other value of the pair (the sine negative for a pair's first, 0 where the
// value is carried).
template <int P>
struct Turn {
  float c[kVals], s[kVals];
  int off;                                   // kLaneOff: the partner's lane
  bool any;                                  // one of the eight turns (kLaneOff: all or none do)
  uint32_t turning;                          // the others: bit e, value e turns
  int partner[P == kAnywhere ? kVals : 1];   // kAnywhere: its place in the row
};

template <int P>
__device__ __forceinline__ bool turns_at(const Turn<P>& t, int e) {
  return P == kLaneOff ? t.any : (t.turning >> e) & 1u;
}

template <int P>
__device__ __forceinline__ Turn<P> find_turn(const TurnArgs& a, int token, int lane16) {
  Turn<P> t;
  const int pos = __ldg(a.positions + token);
  const bool in = pos >= 0 && pos < a.max_pos;
  if (!in && lane16 == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  const float* row = a.table + (int64_t)(in ? pos : 0) * a.rot;
  const int half = a.rot / 2, i0 = lane16 * kVals - a.first;   // the first value's place among the turning
  t.off = lane16;
  t.any = in && i0 + kVals > 0 && i0 < a.rot;
  t.turning = 0u;
  if (P == kLaneOff && i0 >= 0 && i0 < a.rot) t.off = lane16 + (i0 < half ? half : -half) / kVals;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    const int i = i0 + e;
    t.c[e] = 1.f;
    t.s[e] = 0.f;
    if (P == kAnywhere) t.partner[e] = lane16 * kVals + e;
    if (!in || i < 0 || i >= a.rot) continue;
    t.turning |= 1u << e;
    const bool inter = P == kInLane || (P == kAnywhere && a.layout == DSA_ROPE_INTERLEAVED);
    const bool second = inter ? (i & 1) != 0 : i >= half;
    const int pair = inter ? i >> 1 : (second ? i - half : i);
    t.c[e] = __ldg(row + pair);
    const float sn = __ldg(row + half + pair);
    t.s[e] = second ? sn : -sn;
    if (P == kAnywhere) t.partner[e] = a.first + (inter ? i ^ 1 : (second ? i - half : i + half));
  }
  return t;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[kVals]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 codes8(const float (&y)[kVals]) {
  return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                    e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

// Sum over the 16 lanes of a row.
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Every value's partner.  Rows are of one warp: no barrier of the block.
template <int P>
__device__ __forceinline__ void partners(const Turn<P>& t, float* row, int lane16, const float (&x)[kVals],
                                         float (&p)[kVals]) {
  if constexpr (P == kInLane) {
#pragma unroll
    for (int e = 0; e < kVals; ++e) p[e] = x[e ^ 1];
  } else if constexpr (P == kLaneOff) {
#pragma unroll
    for (int e = 0; e < kVals; ++e) p[e] = __shfl_sync(kFull, x[e], t.off, kLanes);
  } else {
    __syncwarp();
    *reinterpret_cast<float4*>(row + lane16 * kVals) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(row + lane16 * kVals + 4) = make_float4(x[4], x[5], x[6], x[7]);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kVals; ++e) p[e] = row[t.partner[e]];
  }
}
// Value e of the row, turned; a carried one as it is (its partner may be infinite).
template <int P>
__device__ __forceinline__ float turned(const Turn<P>& t, int e, float x, float p) {
  const bool turns = turns_at(t, e);
  const float y = fmaf(x, t.c[e], p * t.s[e]);
  return turns ? y : x;
}

// The same without the first product's rounding: within 2^-23 of itself and 2^-48 of
// the product of the exact value, however much of the products cancels (2^-24 of the
// product alone may be any part of what they leave).  `y` is the value before, which
// shows an infinity where this is NaN.
template <int P>
__device__ __forceinline__ float turned_close(const Turn<P>& t, int e, float x, float p, float& y) {
  const bool turns = turns_at(t, e);
  const float b = __fmul_rn(p, t.s[e]);
  const float v = __fmaf_rn(x, t.c[e], b);
  y = turns ? v : x;
  return turns ? __fsub_rn(v, __fmaf_rn(-p, t.s[e], b)) : x;
}

struct KeyArgs {
  const __nv_bfloat16* k;
  int64_t stride;
  const float *weight, *bias;
  float eps;
  TurnArgs turn;
  const int32_t* slots;                      // [S][T]
  int T, S;
  int64_t n_slots;
  uint8_t* cache;                            // [S][n_slots][kDim]
};

template <int P>
__global__ void __launch_bounds__(kThreads) indexer_key_kernel(const KeyArgs a) {
  __shared__ __align__(16) float rows[P == kAnywhere ? kRows : 1][kDim];
  const int lane16 = threadIdx.x & (kLanes - 1), r = threadIdx.x / kLanes;
  const int token = blockIdx.x * kRows + r;
  const bool there = token < a.T;
  const int tok = there ? token : a.T - 1;   // the last block's idle lanes: a row not stored
  float x[kVals], w[kVals], b[kVals];
  unpack8(__ldg(reinterpret_cast<const uint4*>(a.k + tok * a.stride) + lane16), x);
  // The first 16 shards' slots, a lane each, on their way with the rest.
  const int mine = lane16 < a.S ? __ldg(a.slots + (int64_t)lane16 * a.T + tok) : -1;
  const Turn<P> t = find_turn<P>(a.turn, tok, lane16);
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float4 wv = __ldg(reinterpret_cast<const float4*>(a.weight) + lane16 * 2 + v);
    const float4 bv = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias) + lane16 * 2 + v)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    w[4 * v] = wv.x, w[4 * v + 1] = wv.y, w[4 * v + 2] = wv.z, w[4 * v + 3] = wv.w;
    b[4 * v] = bv.x, b[4 * v + 1] = bv.y, b[4 * v + 2] = bv.z, b[4 * v + 3] = bv.w;
  }
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < kVals; ++e) s += x[e];
  const float mean = sum16(s) * (1.f / kDim);
  float q = 0.f;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    x[e] -= mean;
    q = fmaf(x[e], x[e], q);
  }
  const float inv = 1.f / sqrtf(sum16(q) * (1.f / kDim) + a.eps);
#pragma unroll
  for (int e = 0; e < kVals; ++e) x[e] = fmaf(x[e] * inv, w[e], b[e]);
  float p[kVals];
  partners<P>(t, rows[P == kAnywhere ? r : 0], lane16, x, p);
#pragma unroll
  for (int e = 0; e < kVals; ++e) p[e] = turned<P>(t, e, x[e], p[e]);
  const uint2 code = codes8(p);
  for (int sh = 0; sh < a.S; ++sh) {
    const int slot = sh < kLanes ? __shfl_sync(kFull, mine, sh, kLanes) : __ldg(a.slots + (int64_t)sh * a.T + tok);
    if (!there || slot < 0) continue;
    if (slot >= a.n_slots) {
      if (lane16 == 0) raise_flag(a.turn.flags, DSA_FLAG_BOUNDS);
      continue;
    }
    *reinterpret_cast<uint2*>(a.cache + ((int64_t)sh * a.n_slots + slot) * kDim + lane16 * kVals) = code;
  }
}

struct QueryArgs {
  const __nv_bfloat16* q;
  int64_t token, head;                       // strides in elements
  const float* weights;                      // [T][H]
  float factor;
  TurnArgs turn;
  int T, H, per_token;                       // blocks of kRows * kHeads heads
  uint8_t* q_out;                            // [T][H][kDim]
  float* w_out;                              // [T][H]
};

constexpr float kLargest = 3.4028235e38f;    // fp32's largest finite value

// The exponent field of the smallest power of two s with amax <= 448 s (448 = 1.75 *
// 2^8), from 2^-126 on, from amax's bits; s = 1 where amax is 0.
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 127 : max(e, 1);
}
__device__ __forceinline__ float power(int exponent_field) { return __uint_as_float((uint32_t)exponent_field << 23); }

// Value e turned and rounded to odd: cut to fp32, with the last bit set where
// anything was cut, so that a further rounding sees on which side of a middle the
// exact value lay.  The products' and the sum's errors are held in a second fp32
// (Dekker's and Knuth's error-free transformations), 48 bits in all.  (In fp64 a
// head took 5 us.)  An infinite sum, of infinite values or past fp32's range, is itself
// (its errors would be NaN).
template <int P>
__device__ __forceinline__ float turned_to_odd(const Turn<P>& t, int e, float x, float p) {
  const bool turns = turns_at(t, e);
  if (!turns) return x;
  const float a = __fmul_rn(x, t.c[e]), b = __fmul_rn(p, t.s[e]);
  const float ea = __fmaf_rn(x, t.c[e], -a), eb = __fmaf_rn(p, t.s[e], -b);
  const float sum = __fadd_rn(a, b), part = __fsub_rn(sum, a);
  if (!(fabsf(sum) <= kLargest)) return sum;
  const float es = __fadd_rn(__fsub_rn(a, __fsub_rn(sum, part)), __fsub_rn(b, part));
  const float low = __fadd_rn(es, __fadd_rn(ea, eb));
  float z = low == 0.f ? sum : __fadd_rn(sum, low);   // (-0 stays)
  const float rest = __fsub_rn(low, __fsub_rn(z, sum));
  const uint32_t bits = __float_as_uint(z);
  if (rest != 0.f && z != 0.f && fabsf(z) <= kLargest && !(bits & 1u))
    z = __uint_as_float((rest > 0.f) == (z > 0.f) ? bits + 1u : bits - 1u);
  return z;
}

// Nine blocks an SM (56 registers) hide more of a row's latency than the seven that
// 72 registers leave: 4096 tokens of 64 heads 39.1 us against 43.7; ten 42.9.
template <int P, int kHeads>
__global__ void __launch_bounds__(kThreads, kHeads == 4 && P != kAnywhere ? 9 : 1) indexer_query_kernel(const QueryArgs a) {
  __shared__ __align__(16) float rows[P == kAnywhere ? kRows : 1][kDim];
  const int lane16 = threadIdx.x & (kLanes - 1), r = threadIdx.x / kLanes;
  const int token = blockIdx.x / a.per_token;
  const int h0 = (blockIdx.x - token * a.per_token) * (kRows * kHeads) + r;
  uint4 raw[kHeads];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int h = h0 + k * kRows;
    raw[k] = h < a.H ? __ldg(reinterpret_cast<const uint4*>(a.q + token * a.token + h * a.head) + lane16)
                     : make_uint4(0, 0, 0, 0);
  }
  const Turn<P> t = find_turn<P>(a.turn, token, lane16);
  auto store = [&](int h, uint2 code, int field) {
    const int64_t row = (int64_t)token * a.H + h;
    *reinterpret_cast<uint2*>(a.q_out + row * kDim + lane16 * kVals) = code;
    if (lane16 == 0) a.w_out[row] = a.weights[row] * a.factor * power(field);
  };
  uint32_t again = 0;                        // bit k: the warp's k-th two heads go once more
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int h = h0 + k * kRows;
    float x[kVals], p[kVals], y[kVals];
    unpack8(raw[k], x);
    partners<P>(t, rows[P == kAnywhere ? r : 0], lane16, x, p);
    float own = 0.f;                         // the lane's largest (of what is no NaN)
#pragma unroll
    for (int e = 0; e < kVals; ++e) {
      float v;
      y[e] = turned_close<P>(t, e, x[e], p[e], v);
      own = fmaxf(own, fabsf(v));
    }
    float amax = own;
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const int field = scale_exponent(__float_as_uint(amax));
    const float inv = power(254 - field);    // 1 / s
    // The error may have moved a turned value across the middle between two codes if its
    // codes 2^-21 of it further in and out differ (carried values are exact); and the
    // lane's largest across the border between two scales if it is near: its error is 2.1
    // units of its last place at most, as a product is no larger than the pair, and that
    // no more than sqrt(2) times the head's largest.  Those heads, infinite ones, and
    // those whose errors may be subnormal go once more, exactly.
    const float in = t.any ? inv * (1.f - 0x1p-21f) : inv, out = t.any ? inv * (1.f + 0x1p-21f) : inv;
    float z[kVals];
#pragma unroll
    for (int e = 0; e < kVals; ++e) z[e] = y[e] * in;
    const uint2 code = codes8(z);
#pragma unroll
    for (int e = 0; e < kVals; ++e) z[e] = y[e] * out;
    const uint2 outer = codes8(z);
    const uint32_t border = (__float_as_uint(amax) & 0x7F800000u) | 0x600000u;
    const bool near = code.x != outer.x || code.y != outer.y || !(amax <= kLargest) ||
                      (t.any && (__float_as_uint(own) - (border - 8u) <= 16u || (amax < 0x1p-60f && amax > 0.f)));
    if (__any_sync(kFull, near)) again |= 1u << k;
    else if (h < a.H) store(h, code, field);
  }
  // Behind the others, read again: inlined above, the second pass's registers cost every
  // head (4096 tokens of 64 heads 43.7 us against 40.0).
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int h = h0 + (__ffs(again) - 1) * kRows;
    float x[kVals], p[kVals], z[kVals];
    unpack8(h < a.H ? __ldg(reinterpret_cast<const uint4*>(a.q + token * a.token + h * a.head) + lane16)
                    : make_uint4(0, 0, 0, 0), x);
    partners<P>(t, rows[P == kAnywhere ? r : 0], lane16, x, p);
    // Finite values may turn past fp32's range (by a factor of |cos| + |sin|; where these
    // are below 64, to values that a scale reaches), and errors below it: such heads go
    // once more 2^16 smaller, where their largest values lose nothing, or 2^64 larger.
    float top;
    int down = 0;                            // by 2^down smaller
#pragma unroll 1
    for (int trip = 0;; ++trip) {
      const float pre = power(127 - down);
      const float most = down > 0 ? 448.f * 0x1p111f : kLargest;   // what the largest s reaches, 448 * 2^127
      bool past = false;
      top = 0.f;
#pragma unroll
      for (int e = 0; e < kVals; ++e) {
        // (An infinite value stays: larger, the finite one beside it may be so too.)
        if (trip == 0 || down >= 0 || fabsf(z[e]) <= kLargest)
          z[e] = turned_to_odd<P>(t, e, x[e] * pre, p[e] * pre);
        past |= !(fabsf(z[e]) <= kLargest) && fabsf(x[e]) <= kLargest && fabsf(p[e]) <= kLargest &&
                fabsf(t.c[e]) <= 64.f && fabsf(t.s[e]) <= 64.f;
        if (fabsf(z[e]) <= most) top = fmaxf(top, fabsf(z[e]));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      if (trip > 0) break;
      const unsigned past_rows = __ballot_sync(kFull, past);
      down = past_rows & (0xffffu << (threadIdx.x & kLanes)) ? 16 : top < 0x1p-60f ? -64 : 0;
      if (!__any_sync(kFull, down != 0)) break;
    }
    const int field = top == 0.f ? 127 : max(scale_exponent(__float_as_uint(top)) + down, 1);
#pragma unroll
    for (int e = 0; e < kVals; ++e) z[e] *= power(254 - field + down);
    if (h < a.H) store(h, codes8(z), field);
  }
}

// Where a value's partner lies.
int partner_of(int rot, int first, int layout) {
  if (layout == DSA_ROPE_INTERLEAVED && first % 2 == 0) return kInLane;
  if (layout == DSA_ROPE_HALF && first % kVals == 0 && rot % (2 * kVals) == 0) return kLaneOff;
  return kAnywhere;
}

template <int P>
cudaError_t launch_query(QueryArgs& a, bool few, cudaStream_t stream) {
  // Four heads a thread share its cosines and sines; with few tokens, two, which
  // are more blocks.  (4096 tokens, 64 heads: 64, 58, 58 us with two, four, eight
  // before scales came from exponent fields.)
  const int heads = kRows * (few ? 2 : 4);
  a.per_token = (a.H + heads - 1) / heads;
  const dim3 grid((unsigned)((int64_t)a.T * a.per_token));
  return few ? launch_kernel(indexer_query_kernel<P, 2>, grid, dim3(kThreads), 0, stream, 0, a)
             : launch_kernel(indexer_query_kernel<P, 4>, grid, dim3(kThreads), 0, stream, 0, a);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

dsa_status check_turn(int max_pos, int rot, int first, int layout) {
  if (max_pos < 1 || rot < 2 || rot % 2 || first < 0 || first > kDim || rot > kDim - first)
    return DSA_ERR_INVALID_ARG;
  return layout == DSA_ROPE_INTERLEAVED || layout == DSA_ROPE_HALF ? DSA_OK : DSA_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_indexer_key_insert(const uint16_t* k, int64_t k_token,
                                             const float* norm_weight, const float* norm_bias,
                                             float eps, const int32_t* positions,
                                             const float* cos_sin_cache, int max_pos, int rot_dim,
                                             int first, int layout, const int32_t* slot_mapping,
                                             int T, int S, uint8_t* k_cache, int64_t n_slots,
                                             uint32_t* err_flags, cudaStream_t stream) {
  if (T < 0 || n_slots < 1 || !(eps >= 0.f) || isinf(eps)) return DSA_ERR_INVALID_ARG;
  if (const dsa_status st = check_turn(max_pos, rot_dim, first, layout)) return st;
  if (S < 1 || S > DSA_MAX_SHARDS) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!k || !norm_weight || !positions || !cos_sin_cache || !slot_mapping || !k_cache)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(norm_weight, 16) || !aligned(norm_bias, 16) ||
      !aligned(k_cache, 16) || !aligned(positions, 4) || !aligned(cos_sin_cache, 4) ||
      !aligned(slot_mapping, 4) || (T > 1 && (k_token < 0 || k_token % 8)))
    return DSA_ERR_INVALID_ARG;
  if (!apart({bytes_of(k_cache, S * n_slots * kDim)},
             {rows_of(k, T, k_token, 1, 0, kDim, 2), bytes_of(norm_weight, kDim * 4), bytes_of(norm_bias, kDim * 4),
              bytes_of(positions, (int64_t)T * 4), bytes_of(cos_sin_cache, (int64_t)max_pos * rot_dim * 4),
              bytes_of(slot_mapping, (int64_t)S * T * 4)}))
    return DSA_ERR_INVALID_ARG;
  const KeyArgs a{reinterpret_cast<const __nv_bfloat16*>(k), T > 1 ? k_token : 0, norm_weight, norm_bias, eps,
                  {positions, cos_sin_cache, max_pos, rot_dim, first, layout, err_flags},
                  slot_mapping, T, S, n_slots, k_cache};
  const unsigned blocks = (unsigned)(((int64_t)T + kRows - 1) / kRows);
  const int part = partner_of(rot_dim, first, layout);
  const auto kernel = part == kInLane ? indexer_key_kernel<kInLane>
                      : part == kLaneOff ? indexer_key_kernel<kLaneOff> : indexer_key_kernel<kAnywhere>;
  return launch_kernel(kernel, dim3(blocks), dim3(kThreads), 0, stream, 0, a) == cudaSuccess ? DSA_OK
                                                                                            : DSA_ERR_CUDA;
}

extern "C" dsa_status dsa_indexer_query_fp8(const uint16_t* q, int64_t q_token, int64_t q_head,
                                            const float* weights, float factor,
                                            const int32_t* positions, const float* cos_sin_cache,
                                            int max_pos, int rot_dim, int first, int layout, int T,
                                            int H, uint8_t* q_out, float* weights_out,
                                            uint32_t* err_flags, cudaStream_t stream) {
  if (T < 0 || H < 1 || !(factor == factor) || isinf(factor)) return DSA_ERR_INVALID_ARG;
  if (const dsa_status st = check_turn(max_pos, rot_dim, first, layout)) return st;
  if (T == 0) return DSA_OK;
  if (!q || !weights || !positions || !cos_sin_cache || !q_out || !weights_out)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(weights, 4) || !aligned(weights_out, 4) ||
      !aligned(positions, 4) || !aligned(cos_sin_cache, 4) ||
      (T > 1 && (q_token < 0 || q_token % 8)) || (H > 1 && (q_head < 0 || q_head % 8)))
    return DSA_ERR_INVALID_ARG;
  QueryArgs a{reinterpret_cast<const __nv_bfloat16*>(q), T > 1 ? q_token : 0, H > 1 ? q_head : 0, weights, factor,
              {positions, cos_sin_cache, max_pos, rot_dim, first, layout, err_flags},
              T, H, 0, q_out, weights_out};
  const int64_t heads = (int64_t)T * H;
  if (heads > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  const Region w = weights_out == weights ? Region{} : bytes_of(weights, heads * 4);   // in place, or apart
  if (!apart({bytes_of(q_out, heads * kDim), bytes_of(weights_out, heads * 4)},
             {rows_of(q, T, q_token, H, q_head, kDim, 2), w, bytes_of(positions, (int64_t)T * 4),
              bytes_of(cos_sin_cache, (int64_t)max_pos * rot_dim * 4)}))
    return DSA_ERR_INVALID_ARG;
  const int part = partner_of(rot_dim, first, layout);
  const bool few = heads < 65536;
  const cudaError_t e = part == kInLane    ? launch_query<kInLane>(a, few, stream)
                        : part == kLaneOff ? launch_query<kLaneOff>(a, few, stream)
                                           : launch_query<kAnywhere>(a, few, stream);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
