// Sparse MLA decode attention over an 8-bit cache with a scale for each block
// of slots (sm_103a).
//
// Per (shard s, row r, head h), over the valid slots j of the row's list:
// x_j = scale t_j (q . c_j), t_j the scale of the slot's block and c_j its 576
// e4m3 codes; O = sum_j 2^(x_j log2 e) t_j c_j[0..512) / sum_j 2^(x_j log2 e).
//
// A CTA per (row, shard, group of 16 heads), two heads a warp, one pass over
// the slots in tiles of 32 with the running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kDqk = DSA_MLA_DQK, kDv = DSA_MLA_DV;
constexpr int kTile = 32, kHeadsPerCta = 16, kWarps = 8, kThreads = kWarps * 32;
constexpr int kHeadsPerWarp = kHeadsPerCta / kWarps;
constexpr int kPitch = kDqk + 1;               // lanes of a column in different banks
constexpr float kLog2e = 1.4426950408889634f;

struct MlaFp8Args {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const float* scales;
  const int32_t* slots;
  const int32_t* counts;
  int64_t n_slots, n_blocks;
  int rows, H, K, hgroups;
  float c2;
  __nv_bfloat16* out;
  float* lse2;
  uint32_t* flags;
  FastDiv fblock;
};

struct Smem {
  float k[kTile * kPitch];
  float q[kHeadsPerCta][kDqk];
  int ok[kTile];
};

__global__ void __launch_bounds__(kThreads) sparse_mla_decode_fp8_kernel(const MlaFp8Args a) {
  extern __shared__ unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hg = blockIdx.x % a.hgroups, pair = blockIdx.x / a.hgroups;
  const int s = pair / a.rows, r = pair - s * a.rows;
  int count = __ldg(a.counts + pair);
  if ((count < 0 || count > a.K) && tid == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
  count = min(max(count, 0), a.K);
  for (int i = tid; i < kHeadsPerCta * kDqk; i += kThreads) {
    const int h = hg * kHeadsPerCta + i / kDqk;
    sm.q[i / kDqk][i % kDqk] =
        h < a.H ? __bfloat162float(a.q[((int64_t)r * a.H + h) * kDqk + i % kDqk]) : 0.f;
  }
  float m[kHeadsPerWarp], l[kHeadsPerWarp], o[kHeadsPerWarp][kDv / 32];
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < kDv / 32; ++d) o[i][d] = 0.f;
  }
  const int32_t* list = a.slots + (int64_t)pair * a.K;
  for (int t = 0; t < count; t += kTile) {
    __syncthreads();
    for (int j = warp; j < kTile; j += kWarps) {
      const int slot = t + j < count ? __ldg(list + t + j) : -1;
      const bool in = slot >= 0 && slot < a.n_slots;
      if (t + j < count && !in && lane == 0) raise_flag(a.flags, DSA_FLAG_BOUNDS);
      if (lane == 0) sm.ok[j] = in;
      const float ts = in ? __ldg(a.scales + s * a.n_blocks + fdiv((uint32_t)slot, a.fblock)) : 0.f;
      const uint8_t* row = a.cache + ((int64_t)s * a.n_slots + (in ? slot : 0)) * kDqk;
      for (int d = lane; d < kDqk; d += 32) {
        __nv_fp8_e4m3 c;
        c.__x = row[d];
        sm.k[j * kPitch + d] = in ? (float)c * ts : 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp; ++i) {
      const float* q = sm.q[warp * kHeadsPerWarp + i];
      float x = 0.f;
      for (int d = 0; d < kDqk; ++d) x = fmaf(q[d], sm.k[lane * kPitch + d], x);
      x = sm.ok[lane] ? x * a.c2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, k));
      const float mn = fmaxf(m[i], mx);
      if (mn == -INFINITY) continue;
      const float alpha = exp2f(m[i] - mn), p = exp2f(x - mn);
      m[i] = mn;
      float sum = p;
#pragma unroll
      for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(kFull, sum, k);
      l[i] = l[i] * alpha + sum;
#pragma unroll
      for (int d = 0; d < kDv / 32; ++d) o[i][d] *= alpha;
      for (int j = 0; j < kTile; ++j) {
        const float pj = __shfl_sync(kFull, p, j);
#pragma unroll
        for (int d = 0; d < kDv / 32; ++d) o[i][d] = fmaf(pj, sm.k[j * kPitch + d * 32 + lane], o[i][d]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp; ++i) {
    const int h = hg * kHeadsPerCta + warp * kHeadsPerWarp + i;
    if (h >= a.H) continue;
    const int64_t at = (int64_t)pair * a.H + h;
    const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
    for (int d = 0; d < kDv / 32; ++d)
      a.out[at * kDv + d * 32 + lane] = __float2bfloat16_rn(o[i][d] * inv);
    if (lane == 0) a.lse2[at] = l[i] > 0.f ? m[i] + log2f(l[i]) : -INFINITY;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_sparse_mla_decode_fp8(const uint16_t* q, const uint8_t* kv_cache,
                                                const float* block_scales, int64_t n_slots,
                                                int block_tokens, const int32_t* slots,
                                                const int32_t* counts, int rows, int S, int H,
                                                int K, float scale, uint16_t* out, float* lse2,
                                                uint32_t* err_flags, cudaStream_t stream) {
  if (rows < 0 || K < 1 || H < 1 || n_slots < 1 || block_tokens < 1 || n_slots % block_tokens ||
      !std::isfinite(scale))
    return DSA_ERR_INVALID_ARG;
  if (S < 1 || S > DSA_MAX_SHARDS || n_slots > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (rows == 0) return DSA_OK;
  if (!q || !kv_cache || !block_scales || !slots || !counts || !out || !lse2)
    return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  const int hgroups = (H + kHeadsPerCta - 1) / kHeadsPerCta;
  const int64_t blocks = (int64_t)rows * S * hgroups;
  if (blocks > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  const int smem = (int)sizeof(Smem);
  if (cudaFuncSetAttribute(sparse_mla_decode_fp8_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const MlaFp8Args a{reinterpret_cast<const __nv_bfloat16*>(q),
                     kv_cache,
                     block_scales,
                     slots,
                     counts,
                     n_slots,
                     n_slots / block_tokens,
                     rows,
                     H,
                     K,
                     hgroups,
                     scale * kLog2e,
                     reinterpret_cast<__nv_bfloat16*>(out),
                     lse2,
                     err_flags,
                     FastDiv((uint32_t)block_tokens)};
  const cudaError_t e = launch_kernel(sparse_mla_decode_fp8_kernel, dim3((unsigned)blocks),
                                      dim3(kThreads), (size_t)smem, stream, 0u, a);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
