// Joining the parts of an attention whose keys were split over several CTAs.
//
// Part p of row i holds O_p (fp32, normalised by its own sum) and l_p, the
// base-2 log of that sum (-inf: nothing visible, O_p then unwritten and not
// read): out = sum_p w_p O_p / sum_p w_p and lse2 = M + log2 sum_p w_p with
// M = max_p l_p, w_p = 2^(l_p - M).  A warp takes a row, its lanes four
// neighbouring values each of every 128; the parts' loads are independent.
#pragma once

#include "tcgen05.cuh"

namespace dsa {

struct MergeArgs {
  const float* o;            // [parts][rows][D]
  const float* l;            // [parts][rows]
  int parts;
  int64_t rows;              // outer * per_outer * H
  // Rows of entries outside [bounds[0], bounds[n]) are left as they are; entry
  // = row / H mod per_outer.
  const int32_t* bounds;
  int n, per_outer, H;
  void* out;                 // [rows][D], 16-bit floats
  float* lse2;               // [rows]
};

template <int D, bool BF16>
__global__ void __launch_bounds__(256) merge_parts_kernel(const MergeArgs a) {
  constexpr int kV = D / 128;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int entry = (int)((row / a.H) % a.per_outer);
  if (entry < __ldg(a.bounds) || entry >= __ldg(a.bounds + a.n)) return;
  float m = -INFINITY;
  for (int p = lane; p < a.parts; p += 32) m = fmaxf(m, a.l[p * a.rows + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float total = 0.f;
  float4 acc[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p) {
    const float w = fast_exp2(a.l[p * a.rows + row] - ref);
    if (w != 0.f) {
      const float4* src = reinterpret_cast<const float4*>(a.o + (p * a.rows + row) * D) + lane;
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const float4 x = src[v * 32];
        acc[v].x = fmaf(w, x.x, acc[v].x);
        acc[v].y = fmaf(w, x.y, acc[v].y);
        acc[v].z = fmaf(w, x.z, acc[v].z);
        acc[v].w = fmaf(w, x.w, acc[v].w);
      }
    }
    total += w;
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D) + lane;
#pragma unroll
  for (int v = 0; v < kV; ++v)
    dst[v * 32] = make_uint2(pack16<BF16>(acc[v].x * inv, acc[v].y * inv),
                             pack16<BF16>(acc[v].z * inv, acc[v].w * inv));
  if (lane == 0) a.lse2[row] = total == 0.f ? -INFINITY : ref + log2f(total);
}

template <int D, bool BF16>
inline cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream) {
  return launch_kernel(merge_parts_kernel<D, BF16>, dim3((unsigned)((a.rows + 7) / 8)), dim3(256), 0,
                       stream, 0, a);
}

}  // namespace dsa
