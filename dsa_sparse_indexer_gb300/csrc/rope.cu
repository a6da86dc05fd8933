// Rotary positions (sm_103a): tables of cosines and sines, scaled for contexts
// longer than the trained one, and the rotation of queries, keys or their
// gradients by such a table.  The table's layout is the one fused_norm_rope
// reads: per position, rot_dim / 2 cosines, then as many sines.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "rope_steps.h"

namespace dsa {
namespace {

template <typename E, int V>
struct alignas(sizeof(E) * V) Vec {
  E e[V];
};

// ---- the table ---------------------------------------------------------------
//
// Entry (p, i) is the angle p w_i.  A far position's angle loses its fraction
// of a turn in fp32, and fp64 arithmetic is slow here, so the angle is an
// integer: w_i / 2 pi as a 64-bit fraction of a turn (rounded once, on the
// host: rope_steps.h), p times that modulo 2^64, the whole turns falling off the
// top.  Its upper 32 bits are the angle cut to 2^-32 turns, whatever p (an
// absolute error: the first sines of a slow pair, below 2^-28, have few bits):
// the nearest quarter turn in whole, and within an eighth of a turn of it a
// fraction whose sine and cosine are their power series (to x^9 and x^10: the next
// terms are below 2e-9 there).  A thread keeps its pair i and steps its phase by
// whole positions (one 64-bit addition each); four pairs where 16-byte stores
// fit.  Bound by its stores, with the arithmetic close behind: 131072 positions
// of 64 values (33.5 MB, in replays into L2) take 6.4 us (a pair a thread 7.7, and
// 8.4 with sincospif, whose own reduction is not needed here); 62 values, 8.0.
// 4096 positions of 128 take 2.0 us, a launch's latency.
constexpr int kMaxPairs = 128;
static_assert((int)DSA_ROPE_NONE == RopeScaling::kNone && (int)DSA_ROPE_LINEAR == RopeScaling::kLinear &&
                  (int)DSA_ROPE_NTK == RopeScaling::kNtk && (int)DSA_ROPE_YARN == RopeScaling::kYarn,
              "the scalings' numbers");
constexpr int kTableThreads = 256;

struct TableArgs {
  uint64_t step[kMaxPairs];                    // 2^64 w_i / (2 pi)
  float* table;
  float amplitude;
  int max_pos, half, group, steps;             // group: positions side by side in a block
};

// Sine and cosine of u 2^-32 turns.
__device__ __forceinline__ void sincos_turn(uint32_t u, float* s, float* c) {
  const uint32_t q = (u + 0x20000000u) >> 30;  // quarter turns
  const float x = (float)(int32_t)(u - (q << 30)) * (6.283185307179586f * 0x1p-32f), y = x * x;
  float t = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  t = fmaf(y, t, 1.f / 120.f);
  t = fmaf(y, t, -1.f / 6.f);
  const float sine = fmaf(x * y, t, x);
  t = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  t = fmaf(y, t, -1.f / 720.f);
  t = fmaf(y, t, 1.f / 24.f);
  t = fmaf(y, t, -0.5f);
  const float cosine = fmaf(y, t, 1.f);
  const bool odd = q & 1u;
  *s = __uint_as_float(__float_as_uint(odd ? cosine : sine) ^ ((q & 2u) << 30));
  *c = __uint_as_float(__float_as_uint(odd ? sine : cosine) ^ (((q + 1u) & 2u) << 30));
}

// V pairs a thread, side by side.
template <int V>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ TableArgs a) {
  __shared__ uint64_t step[kMaxPairs];
  if (threadIdx.x < a.half) step[threadIdx.x] = a.step[threadIdx.x];
  __syncthreads();
  const int each = a.half / V, q = threadIdx.x / each, i = (threadIdx.x - q * each) * V;
  if (q >= a.group) return;
  const int64_t p0 = (int64_t)blockIdx.x * (a.group * a.steps);
  const int end = (int)min((int64_t)a.max_pos - p0, (int64_t)a.group * a.steps);
  uint64_t phase[V];
#pragma unroll
  for (int k = 0; k < V; ++k) phase[k] = step[i + k] * (uint64_t)(p0 + q);
  float* row = a.table + (p0 + q) * (2 * a.half) + i;
  for (int p = q; p < end; p += a.group) {
    Vec<float, V> s, c;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      sincos_turn((uint32_t)(phase[k] >> 32), &s.e[k], &c.e[k]);
      s.e[k] *= a.amplitude;
      c.e[k] *= a.amplitude;
      phase[k] += step[i + k] * (uint64_t)a.group;
    }
    *reinterpret_cast<Vec<float, V>*>(row) = c;
    *reinterpret_cast<Vec<float, V>*>(row + a.half) = s;
    row += (int64_t)a.group * (2 * a.half);
  }
}

// ---- the rotation --------------------------------------------------------------
//
// A row is one head of one token: D values, of which [first, first + rot) turn
// in pairs and the rest is carried.  Memory-bound, and the arithmetic (unpacking,
// four multiply-adds a pair, packing) close behind, so addresses and the
// table's values are shared: a unit is what one thread takes of a row, a 16-byte
// vector (interleaved pairs lie within it) or the two vectors at i and
// i + rot / 2 of the half layout, and a thread takes the same unit of kRows
// consecutive heads of a token, all loads in flight at once.  Rows that no
// 16-byte vectors fit (odd widths, offsets) take vectors of two elements or one.
// Measured: 4096 tokens of 128 heads of 64 (67 MB in, 67 MB out, strided) in
// 37 us with every row's token, address and table read found anew, 27.3 so (24.5
// in replays, 5.5 TB/s); a plain copy of as much takes 23.  64 tokens take 2.0
// us, a launch's latency.  8192 tokens of 32 heads of 130 (136 MB) take 28 us, at
// odd offsets 36 to 41 for 125 values; a head and an element a thread, 134 and 81.

enum { kInterleaved = DSA_ROPE_INTERLEAVED, kHalf = DSA_ROPE_HALF };
constexpr int kMaxWidth = 1024;               // values of a row

struct RotArgs {
  const void* x;
  void* out;
  int64_t x_token, x_head, out_token, out_head;   // strides in elements
  const int32_t* positions;
  const float* table;
  uint32_t* flags;
  int max_pos, rot, first, D, T, H;
  int units, turning;       // units of a row (the rotating ones first)
  int per_block;            // groups of rows side by side in a block
  float sign;               // -1 for the inverse rotation
  int64_t groups;           // of kRows heads
  FastDiv fgroups;          // groups of a token
};

template <typename E> __device__ __forceinline__ float to_float(E v);
template <> __device__ __forceinline__ float to_float(float v) { return v; }
template <> __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E from_float(float v);
template <> __device__ __forceinline__ float from_float(float v) { return v; }
template <> __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = fmaf(x, c, -y * s);
  b = fmaf(y, c, x * s);
}

// V elements per vector: 16 bytes, or less where a row's layout is not so
// aligned (of one element, an interleaved unit is the two of a pair).
// kTail: a token's last thread may have fewer than kRows heads.
template <typename E, int LAYOUT, int V, int kRows, bool kTail>
__global__ void __launch_bounds__(V * sizeof(E) == 16 ? 256 : kMaxWidth / 2) rotary_kernel(const RotArgs a) {
  constexpr int kVecs = LAYOUT == kHalf || V == 1 ? 2 : 1;   // vectors of a rotating unit
  constexpr int kPairs = kVecs * V / 2;
  using VecT = Vec<E, V>;
  const int side = threadIdx.x / a.units, u = threadIdx.x - side * a.units;
  const int64_t g = (int64_t)blockIdx.x * a.per_block + side;
  if (side >= a.per_block || g >= a.groups) return;
  uint32_t part;
  const uint32_t tok = fdivmod((uint32_t)g, a.fgroups, &part);
  const uint32_t head = part * kRows;
  const int rows = kTail ? min(kRows, a.H - (int)head) : kRows;
  const bool turning = u < a.turning;
  // Element offsets of the unit's vectors, and its first pair.  A carried unit
  // has as many vectors as a turning one, the last unit perhaps one less.
  int at0, apart, pair = 0;
  bool both = true;
  if (turning) {
    pair = u * kPairs;
    at0 = a.first + (LAYOUT == kHalf ? pair : 2 * pair);
    apart = LAYOUT == kHalf ? a.rot / 2 : 1;
  } else {
    at0 = (u - a.turning) * (kVecs * V);
    both = at0 + V < a.D - a.rot;
    apart = at0 < a.first && at0 + V >= a.first ? V + a.rot : V;
    if (at0 >= a.first) at0 += a.rot;
  }
  const E* src = static_cast<const E*>(a.x) + tok * a.x_token + head * a.x_head + at0;
  VecT v[kRows][kVecs];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (k < rows) v[k][0] = *reinterpret_cast<const VecT*>(src + k * a.x_head);
    if (kVecs == 2 && both && k < rows)
      v[k][kVecs - 1] = *reinterpret_cast<const VecT*>(src + k * a.x_head + apart);
  }
  if (turning) {
    constexpr int kP = kPairs > 4 ? 4 : kPairs;
    using VecP = Vec<float, kP>;
    float c[kPairs], s[kPairs];
    const int pos = __ldg(a.positions + tok);
    if (pos >= 0 && pos < a.max_pos) {
      const float* row = a.table + (int64_t)pos * a.rot + pair;
#pragma unroll
      for (int j = 0; j < kPairs; j += kP) {
        const VecP cv = *reinterpret_cast<const VecP*>(row + j);
        const VecP sv = *reinterpret_cast<const VecP*>(row + a.rot / 2 + j);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          c[j + i] = cv.e[i];
          s[j + i] = sv.e[i] * a.sign;
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          E& ea = kVecs == 2 ? v[k][0].e[j] : v[k][0].e[2 * j];
          E& eb = kVecs == 2 ? v[k][kVecs - 1].e[j] : v[k][0].e[(2 * j + 1) % V];
          float fa = to_float(ea), fb = to_float(eb);
          turn(fa, fb, c[j], s[j]);
          ea = from_float<E>(fa);
          eb = from_float<E>(fb);
        }
    } else if (u == 0) {                     // carried: its bits as they are
      raise_flag(a.flags, DSA_FLAG_BOUNDS);
    }
  }
  E* dst = static_cast<E*>(a.out) + tok * a.out_token + head * a.out_head + at0;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (k < rows) *reinterpret_cast<VecT*>(dst + k * a.out_head) = v[k][0];
    if (kVecs == 2 && both && k < rows)
      *reinterpret_cast<VecT*>(dst + k * a.out_head + apart) = v[k][kVecs - 1];
  }
}

// No two of the T x H output rows of D elements lie on one another.
bool rows_apart(int T, int64_t token, int H, int64_t head, int D) {
  if ((T > 1 && token < D) || (H > 1 && head < D)) return false;
  if (T == 1 || H == 1) return true;
  const int64_t near = std::min(token, head), far = std::max(token, head);
  const int64_t n = token < head ? T : H, m = token < head ? H : T;   // rows `near` and `far` apart
  if ((far - D) / near >= n - 1) return true;   // one dimension's rows within a step of the other
  // Row i of the far ones lies `rest` behind row j of the near ones.  j >= i, so
  // that this takes fewer steps than either dimension has rows.
  int64_t j = 0, rest = 0;
  for (int64_t i = 1; i < m; ++i) {
    j += far / near;
    rest += far % near;
    if (rest >= near) rest -= near, ++j;
    if (j >= n) break;
    if (rest < D || (near - rest < D && j + 1 < n)) return false;
  }
  return true;
}

template <typename E, int LAYOUT, int V>
cudaError_t launch_rotary(RotArgs& a, bool in_place, cudaStream_t stream) {
  constexpr int kVecs = LAYOUT == kHalf || V == 1 ? 2 : 1;
  a.turning = a.rot / (kVecs * V);
  const int carried = in_place ? 0 : (a.D - a.rot) / V;
  a.units = a.turning + (carried + kVecs - 1) / kVecs;
  // A block holds whole rows, at most kMaxWidth / 2 units; so many side by side
  // as leave the fewest threads over, in about 128 threads: small blocks leave
  // an SM sooner and take the next row's loads up earlier (128 threads measured
  // 28 us where 256 took 31).
  int threads = 0;
  for (int n = (127 + a.units) / a.units; n * a.units <= 256 || threads == 0; ++n) {
    const int all = (n * a.units + 31) / 32 * 32;
    if (threads == 0 || n * a.units * threads > a.per_block * a.units * all) {
      threads = all;
      a.per_block = n;
    }
  }
  auto go = [&](auto kernel, int rows_each) {
    const int parts = (a.H + rows_each - 1) / rows_each;
    a.groups = (int64_t)a.T * parts;
    a.fgroups = FastDiv((uint32_t)parts);
    const int64_t blocks = (a.groups + a.per_block - 1) / a.per_block;
    return launch_kernel(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), 0, stream, 0u,
                         a);
  };
  // Several heads a thread, 32 or 64 bytes in flight, once that still fills the
  // GPU's 152 SMs twice over; below that the call is latency, and a head a
  // thread spreads it widest.  Narrow vectors take eight when they fill all
  // threads and the heads divide (8192 tokens of 32 heads of 130, bf16: 27.6
  // us, with four 35).
  constexpr int kBytes = kVecs * V * (int)sizeof(E), kMany = kBytes > 16 ? 2 : 4;
  const int64_t all = (int64_t)a.T * a.H * a.units;
  const bool many = all >= (int64_t)152 * 2 * 256 * 4;
  if constexpr (kBytes <= 8)
    if (all >= (int64_t)152 * 2048 * 8 && a.H % 8 == 0)
      return go(rotary_kernel<E, LAYOUT, V, 8, false>, 8);
  if (many && a.H % kMany == 0) return go(rotary_kernel<E, LAYOUT, V, kMany, false>, kMany);
  if (many && a.H > kMany) return go(rotary_kernel<E, LAYOUT, V, kMany, true>, kMany);
  return go(rotary_kernel<E, LAYOUT, V, 1, false>, 1);
}

template <typename E, int LAYOUT>
cudaError_t launch_rotary(RotArgs& a, bool in_place, cudaStream_t stream) {
  // Vectors of V: both tensors' rows, the turning part's ends (and middle, in
  // the half layout) and the table's pairs on their boundaries.
  auto fits = [&](int V) {
    auto lined = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    return lined(a.x, V * sizeof(E)) && lined(a.out, V * sizeof(E)) && lined(a.table, 16) &&
           a.x_token % V == 0 && a.x_head % V == 0 && a.out_token % V == 0 &&
           a.out_head % V == 0 && a.D % V == 0 && a.first % V == 0 &&
           a.rot % (LAYOUT == kHalf ? 2 * V : V) == 0;
  };
  constexpr int kWide = 16 / (int)sizeof(E);
  if (fits(kWide)) return launch_rotary<E, LAYOUT, kWide>(a, in_place, stream);
  if (fits(2)) return launch_rotary<E, LAYOUT, 2>(a, in_place, stream);
  return launch_rotary<E, LAYOUT, 1>(a, in_place, stream);
}

template <typename E>
cudaError_t launch_rotary_of(RotArgs& a, int layout, bool in_place, cudaStream_t stream) {
  return layout == kHalf ? launch_rotary<E, kHalf>(a, in_place, stream)
                         : launch_rotary<E, kInterleaved>(a, in_place, stream);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_rope_table(int max_pos, int rot_dim, double base, int scaling,
                                     double factor, int orig_max_pos, double beta_fast,
                                     double beta_slow, float amplitude, float* table,
                                     cudaStream_t stream) {
  if (max_pos < 0 || rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base) ||
      !(factor >= 1.0) || !std::isfinite(factor) || !std::isfinite(amplitude))
    return DSA_ERR_INVALID_ARG;
  if (scaling < DSA_ROPE_NONE || scaling > DSA_ROPE_YARN) return DSA_ERR_INVALID_ARG;
  if (scaling == DSA_ROPE_YARN &&
      (orig_max_pos < 1 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
       !std::isfinite(beta_fast)))
    return DSA_ERR_INVALID_ARG;
  if (rot_dim > 2 * kMaxPairs) return DSA_ERR_UNSUPPORTED;
  if (max_pos == 0) return DSA_OK;
  if (!table || (reinterpret_cast<uintptr_t>(table) & 3u)) return DSA_ERR_INVALID_ARG;
  TableArgs a{};
  rope_steps(rot_dim, base,
             {static_cast<RopeScaling::Kind>(scaling), factor, orig_max_pos, beta_fast, beta_slow}, a.step);
  a.table = table;
  a.amplitude = amplitude;
  a.max_pos = max_pos;
  a.half = rot_dim / 2;
  // 16-byte stores where the rows allow it.
  const bool wide = a.half % 4 == 0 && (reinterpret_cast<uintptr_t>(table) & 15u) == 0;
  a.group = kTableThreads / (wide ? a.half / 4 : a.half);
  // As many positions a thread as leave every SM two blocks: up to 32 entries.
  a.steps = wide ? 4 : 8;
  while (a.steps > 1 && (int64_t)a.group * a.steps * 2 * 152 > max_pos) a.steps /= 2;
  const int64_t positions = (int64_t)a.group * a.steps;
  const unsigned grid = (unsigned)((max_pos + positions - 1) / positions);
  const cudaError_t e =
      launch_kernel(wide ? rope_table_kernel<4> : rope_table_kernel<1>, dim3(grid), dim3(kTableThreads), 0, stream, 0u, a);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

extern "C" dsa_status dsa_rotary_embed(const void* x, int64_t x_token, int64_t x_head,
                                       const int32_t* positions, const float* cos_sin_cache,
                                       int max_pos, int rot_dim, int first, int T, int H, int D,
                                       int dtype, int layout, int inverse, void* out,
                                       int64_t out_token, int64_t out_head, uint32_t* err_flags,
                                       cudaStream_t stream) {
  if (T < 0 || H < 0 || D < 1 || max_pos < 1 || rot_dim < 2 || rot_dim % 2 || first < 0 ||
      first > D - rot_dim || x_token < 0 || x_head < 0 || out_token < 0 || out_head < 0)
    return DSA_ERR_INVALID_ARG;
  if (dtype < DSA_BF16 || dtype > DSA_FP32 || layout < DSA_ROPE_INTERLEAVED ||
      layout > DSA_ROPE_HALF)
    return DSA_ERR_INVALID_ARG;
  if (D > kMaxWidth || (int64_t)T * H > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return DSA_OK;
  if (!x || !out || !positions || !cos_sin_cache) return DSA_ERR_INVALID_ARG;
  if (!rows_apart(T, out_token, H, out_head, D)) return DSA_ERR_INVALID_ARG;
  const uintptr_t es = dtype == DSA_FP32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(x) & es) || (reinterpret_cast<uintptr_t>(out) & es) ||
      (reinterpret_cast<uintptr_t>(cos_sin_cache) & 3u))
    return DSA_ERR_INVALID_ARG;
  RotArgs a{};
  a.x = x;
  a.out = out;
  a.x_token = x_token;
  a.x_head = x_head;
  a.out_token = out_token;
  a.out_head = out_head;
  a.positions = positions;
  a.table = cos_sin_cache;
  a.flags = err_flags;
  a.max_pos = max_pos;
  a.rot = rot_dim;
  a.first = first;
  a.D = D;
  a.T = T;
  a.H = H;
  a.sign = inverse ? -1.f : 1.f;
  const bool in_place = x == out && (T == 1 || x_token == out_token) && (H == 1 || x_head == out_head);
  if (x == out && !in_place) return DSA_ERR_INVALID_ARG;
  cudaError_t e;
  if (dtype == DSA_BF16) e = launch_rotary_of<__nv_bfloat16>(a, layout, in_place, stream);
  else if (dtype == DSA_FP16) e = launch_rotary_of<__half>(a, layout, in_place, stream);
  else e = launch_rotary_of<float>(a, layout, in_place, stream);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
