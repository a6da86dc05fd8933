// Joining the parts of an attention whose keys were split over several CTAs.
//
// Part p of row i holds O_p (fp32, normalised by its own sum) and l_p, the
// base-2 log of that sum (-inf: nothing visible, O_p then unwritten and not
// read): out = sum_p w_p O_p / sum_p w_p and lse2 = M + log2 sum_p w_p with
// M = max_p l_p, w_p = 2^(l_p - M).  A block takes a row or, with many parts, a
// quarter of it: groups of threads take every kGroups-th part, a thread four
// neighbouring values, and add up in shared memory; the parts' loads are
// independent.  (128 rows of 76 parts, 20 MB: a warp a row with all parts in turn
// left most SMs idle, 45 us.)
#pragma once

#include "tcgen05.cuh"

namespace dsa {

struct MergeArgs {
  const float* o;            // [parts][rows][D]
  const float* l;            // [parts][rows]
  int parts;
  int64_t rows;              // outer * per_outer * H
  // Rows of entries below bounds[0], or not below any, are left as they are; entry = row
  // / H mod per_outer.
  const int32_t* bounds;
  int n, per_outer, H;
  void* out;                 // [rows][D], 16-bit floats
  float* lse2;               // [rows]
};

constexpr int kMaxParts = 128;

template <int D, int kGroups>
struct MergeCut {
  static constexpr int kLanes = D / 4 < 512 / kGroups ? D / 4 : 512 / kGroups;   // threads of a group
  static constexpr int kBlocks = D / 4 / kLanes;                                 // blocks of a row
};

template <int D, bool BF16, int kGroups>
__global__ void __launch_bounds__(kGroups * MergeCut<D, kGroups>::kLanes) merge_parts_kernel(const MergeArgs a) {
  constexpr int kLanes = MergeCut<D, kGroups>::kLanes, kBlocks = MergeCut<D, kGroups>::kBlocks;
  __shared__ float weight[kMaxParts];
  __shared__ float4 sums[kGroups - 1][kLanes];
  const int64_t row = blockIdx.x / kBlocks;
  const int entry = (int)((row / a.H) % a.per_outer);
  const int tid = threadIdx.x, group = tid / kLanes;
  if (entry < __ldg(a.bounds)) return;
  if (entry >= __ldg(a.bounds + a.n)) {      // of no sequence, unless bounds descend
    bool below = false;
    for (int i = tid; i < a.n; i += blockDim.x) below |= __ldg(a.bounds + i) > entry;
    if (!__syncthreads_or(below)) return;
  }
  const int at = (int)(blockIdx.x % kBlocks) * kLanes + tid % kLanes;
  float lse = 0.f;
  if (tid < 32) {                            // the first warp: weights and their sum
    float l[kMaxParts / 32], m = -INFINITY, total = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxParts / 32; ++k) {
      const int p = tid + 32 * k;
      l[k] = p < a.parts ? a.l[p * a.rows + row] : -INFINITY;
      m = fmaxf(m, l[k]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < kMaxParts / 32; ++k) total += l[k] = fast_exp2(l[k] - ref);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int k = 0; k < kMaxParts / 32; ++k) weight[tid + 32 * k] = l[k] * inv;
    lse = total == 0.f ? -INFINITY : ref + log2f(total);
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = group; p < a.parts; p += kGroups) {
    const float w = weight[p];
    if (w != 0.f) {                          // else it may be unwritten
      const float4 x = __ldg(reinterpret_cast<const float4*>(a.o + (p * a.rows + row) * D) + at);
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
  }
  if (group > 0) sums[group - 1][tid % kLanes] = acc;
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int g = 0; g < kGroups - 1; ++g) {
    const float4 x = sums[g][tid];
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
  }
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D)[at] =
      make_uint2(pack16<BF16>(acc.x, acc.y), pack16<BF16>(acc.z, acc.w));
  if (at == 0) a.lse2[row] = lse;
}

template <int D, bool BF16, int kGroups>
inline cudaError_t launch_merge_by(const MergeArgs& a, cudaStream_t stream) {
  using Cut = MergeCut<D, kGroups>;
  return launch_kernel(merge_parts_kernel<D, BF16, kGroups>, dim3((unsigned)(a.rows * Cut::kBlocks)),
                       dim3(kGroups * Cut::kLanes), 0, stream, 0, a);
}
template <int D, bool BF16>
inline cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream) {
  // Many parts of few rows, 16 groups against four, whole calls in us: 16 rows of 128
  // parts 24.6 / 27.1, 128 of 76 31.2 / 33.0; but 256 rows of 38 parts 31.2 / 29.5 and
  // 5856 of three 231 / 181.
  return a.parts > 16 && a.rows <= kSms ? launch_merge_by<D, BF16, 16>(a, stream)
                                       : launch_merge_by<D, BF16, 4>(a, stream);
}

// Parts to split each of `items` (of about `item_us` microseconds) into, for `ctas`
// at a time: the rounds that the parts take, and what writing and reading a
// part's outputs again costs (rows of 4 D bytes, at 5 TB/s, and a launch).
inline int choose_parts(int64_t items, int64_t ctas, double item_us, int64_t rows, int D, int64_t most) {
  if (rows > (1 << 24)) return 1;
  int best = 1;
  double least = (double)((items + ctas - 1) / ctas) * item_us;
  for (int p = 2; p <= (int)(most < kMaxParts ? most : kMaxParts); ++p) {
    const double us = (double)((items * p + ctas - 1) / ctas) * item_us / p + 4.0 + 1.6e-6 * D * rows * p;
    if (us < least * 0.97) least = us, best = p;
  }
  return best;
}

}  // namespace dsa
