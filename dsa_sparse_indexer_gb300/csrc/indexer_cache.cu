// The 8-bit operands of the indexer's logits: keys into the paged key cache,
// queries with their scales folded into the head weights (sm_103a).
//
// Key: y = (k - mean) / sqrt(var + eps) * weight + bias over its 128 values, the
// values [first, first + rot) turned by the position's row of the table, e4m3
// codes (round to nearest even, saturating) to the token's slot.  Query: each
// head's 128 values turned alike, code = e4m3(y / s) with s the smallest power
// of two with max |y| <= 448 s, and the head's weight times factor * s.
//
// Memory-bound: 256 bytes in and 128 out a row.  Sixteen lanes take a row, eight
// values (16 bytes) each, so that sums and maxima are four shuffles.  A pair's
// other half may lie in any lane (half layout, odd widths): the rows pass
// through shared memory as fp32, and every lane turns its own eight values with
// cosines, sines and partners found once and used for all heads it takes.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

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

// How this lane's eight values turn: y_e = x_e cos_e + x_partner sin_e, partner
// the other value of the pair (the sine negative for a pair's first).
struct Turn {
  float c[kVals], s[kVals];
  int8_t partner[kVals];
  bool any;
};

__device__ __forceinline__ Turn find_turn(const TurnArgs& a, int token, int lane16) {
  Turn t;
  const int pos = __ldg(a.positions + token);
  const bool in = pos >= 0 && pos < a.max_pos;
  if (!in && lane16 == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  const float* row = a.table + (int64_t)(in ? pos : 0) * a.rot;
  const int half = a.rot / 2;
  t.any = false;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    const int at = lane16 * kVals + e, i = at - a.first;
    t.c[e] = 1.f;
    t.s[e] = 0.f;
    t.partner[e] = (int8_t)at;
    if (!in || i < 0 || i >= a.rot) continue;
    const bool inter = a.layout == DSA_ROPE_INTERLEAVED;
    const int pair = inter ? i >> 1 : (i < half ? i : i - half);
    const bool second = inter ? (i & 1) != 0 : i >= half;
    const int other = inter ? i ^ 1 : (second ? i - half : i + half);
    t.c[e] = __ldg(row + pair);
    const float sn = __ldg(row + half + pair);
    t.s[e] = second ? sn : -sn;
    t.partner[e] = (int8_t)(a.first + other);
    t.any = true;
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

// The row's values in shared memory for the others' partners, then this lane's
// turned.  Rows are of one warp: no barrier of the block.
__device__ __forceinline__ void turn8(const Turn& t, float* row, int lane16, float (&x)[kVals]) {
  __syncwarp();
  *reinterpret_cast<float4*>(row + lane16 * kVals) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(row + lane16 * kVals + 4) = make_float4(x[4], x[5], x[6], x[7]);
  __syncwarp();
  if (!t.any) return;
#pragma unroll
  for (int e = 0; e < kVals; ++e)
    if (t.partner[e] != lane16 * kVals + e) x[e] = fmaf(x[e], t.c[e], row[t.partner[e]] * t.s[e]);
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

__global__ void __launch_bounds__(kThreads) indexer_key_kernel(const KeyArgs a) {
  __shared__ __align__(16) float rows[kRows][kDim];
  const int lane16 = threadIdx.x & (kLanes - 1), r = threadIdx.x / kLanes;
  const int token = blockIdx.x * kRows + r;
  const bool there = token < a.T;
  const int tok = there ? token : a.T - 1;   // the last block's idle lanes: a row not stored
  float x[kVals], w[kVals], b[kVals];
  unpack8(__ldg(reinterpret_cast<const uint4*>(a.k + tok * a.stride) + lane16), x);
  const Turn t = find_turn(a.turn, tok, lane16);
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
  turn8(t, rows[r], lane16, x);
  const uint2 code = codes8(x);
  if (!there) return;
  for (int sh = 0; sh < a.S; ++sh) {
    const int slot = __ldg(a.slots + (int64_t)sh * a.T + token);
    if (slot < 0) continue;
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

// The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), from 2^-126
// on; 1 where amax is 0.
template <typename F>
__device__ __forceinline__ float scale_for(F amax) {
  if (!(amax > 0)) return 1.f;
  int e;
  const F m = frexp(amax, &e);
  return ldexpf(1.f, max(m > (F)0.875 ? e - 8 : e - 9, -126));
}

template <int kHeads>
__global__ void __launch_bounds__(kThreads) indexer_query_kernel(const QueryArgs a) {
  __shared__ __align__(16) float rows[kRows][kDim];
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
  const Turn t = find_turn(a.turn, token, lane16);
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int h = h0 + k * kRows;
    float x[kVals];
    unpack8(raw[k], x);
    turn8(t, rows[r], lane16, x);
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < kVals; ++e) amax = fmaxf(amax, isfinite(x[e]) ? fabsf(x[e]) : 0.f);
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    float scale = scale_for(amax);
    // A largest value within fp32's error of the border between two scales: found
    // again in 64 bits, so that the scale is that of the exact values (one head
    // in a hundred: bf16 values lie on the border itself).
    const bool near = fabsf(amax / scale - 448.f) < 448.f * 1e-6f || fabsf(amax / scale - 224.f) < 224.f * 1e-6f;
    if (__any_sync(kFull, near)) {
      float x0[kVals];
      unpack8(raw[k], x0);
      double top = 0.0;
#pragma unroll
      for (int e = 0; e < kVals; ++e) {
        double y = x0[e];
        if (t.any && t.partner[e] != lane16 * kVals + e)
          y = y * (double)t.c[e] + (double)rows[r][t.partner[e]] * (double)t.s[e];
        if (isfinite(x[e])) top = fmax(top, fabs(y));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, o));
      scale = scale_for(top);
    }
    if (h >= a.H) continue;
    const float inv = 1.f / scale;           // exact: a power of two (of 2^-126, 2^126)
#pragma unroll
    for (int e = 0; e < kVals; ++e) x[e] *= inv;
    const int64_t row = (int64_t)token * a.H + h;
    *reinterpret_cast<uint2*>(a.q_out + row * kDim + lane16 * kVals) = codes8(x);
    if (lane16 == 0) a.w_out[row] = a.weights[row] * a.factor * scale;
  }
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
  const KeyArgs a{reinterpret_cast<const __nv_bfloat16*>(k), T > 1 ? k_token : 0, norm_weight, norm_bias, eps,
                  {positions, cos_sin_cache, max_pos, rot_dim, first, layout, err_flags},
                  slot_mapping, T, S, n_slots, k_cache};
  const unsigned blocks = (unsigned)(((int64_t)T + kRows - 1) / kRows);
  return launch_kernel(indexer_key_kernel, dim3(blocks), dim3(kThreads), 0, stream, 0, a) == cudaSuccess
             ? DSA_OK : DSA_ERR_CUDA;
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
  constexpr int kHeads = 4;
  a.per_token = (H + kRows * kHeads - 1) / (kRows * kHeads);
  const int64_t blocks = (int64_t)T * a.per_token;
  if (blocks > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  return launch_kernel(indexer_query_kernel<kHeads>, dim3((unsigned)blocks), dim3(kThreads), 0,
                       stream, 0, a) == cudaSuccess
             ? DSA_OK : DSA_ERR_CUDA;
}
