// k_attn_merge.hip -- joins the partial results of the splits of an attention call.
//
// A row's splits hold (M_s, l_s) and sums o_s relative to their own reference exponent M_s; with
// M = max_s M_s:  o = sum_s 2^(M_s - M) o_s / sum_s 2^(M_s - M) l_s, in a fixed order.  Bound by latency: a call's
// partial sums are a small part of its cache.
#include <hip/hip_runtime.h>

#include "bq_attn.h"
#include "bq_internal.h"
#include "bq_launch.h"

namespace bq {
namespace {

// One workgroup per row: wave w takes splits w, w + 4, ..., lane by lane over head_dim.
constexpr int kWaves = 4;

template <int D>
__global__ __launch_bounds__(64 * kWaves) void merge_kernel(KvAttendArgs aa, int nsplit, int bf16) {
  __shared__ float s_sum[kWaves][D];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Sequence sq = sequence(aa, blockIdx.y);
  const int64_t row = blockIdx.x;
  if (row >= (int64_t)min(sq.nq, aa.max_q_len) * aa.heads) return;
  const int64_t at = (int64_t)sq.q0 * aa.heads + row;  // token * heads + head
  const float* sums = static_cast<const float*>(aa.workspace) + at * nsplit * D;
  const Partial* parts =
      reinterpret_cast<const Partial*>(static_cast<const float*>(aa.workspace) + aa.tokens * aa.heads * nsplit * D) +
      at * nsplit;
  const Partial mine = lane < nsplit ? parts[lane] : Partial{-INFINITY, 0.0f};
  constexpr int kPer = D / 64;
  float v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] = 0.0f;
  // splits past the last repeat it with weight zero, so that four loads are in flight without a condition
  float top = mine.m;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float f = mine.m == -INFINITY ? 0.0f : exp2_hw(mine.m - top);
  float l = f * mine.l;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
  for (int s0 = wave; s0 < nsplit; s0 += 4 * kWaves) {
    float x[4][kPer];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* src = sums + (int64_t)min(s0 + i * kWaves, nsplit - 1) * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[i][k] = src[k];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + i * kWaves;
      const float fs = s < nsplit ? bits_f32(__builtin_amdgcn_readlane(f32_bits(f), min(s, 63))) : 0.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = fmaf(fs, x[i][k], v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) s_sum[wave][lane * kPer + k] = v[k];
  __syncthreads();
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  const int64_t token = at / aa.heads, head = at - token * aa.heads;
  if (tid < D / 2) {
    const int d = 2 * tid;
    float o[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      o[k] = ((s_sum[0][d + k] + s_sum[1][d + k]) + (s_sum[2][d + k] + s_sum[3][d + k])) * inv;
    uint16_t* out = static_cast<uint16_t*>(aa.out) + token * aa.out_stride + head * D;
    *reinterpret_cast<uint32_t*>(out + d) = pack16(o[0], o[1], bf16);
  }
  if (aa.lse != nullptr && tid == 0) aa.lse[at] = log_sum(top, l);
}

}  // namespace

int launch_kv_merge(const KvAttendArgs& a, int dtype, int nsplit, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)((int64_t)a.max_q_len * a.heads), (unsigned)a.num_seqs);
  const dim3 block(64 * kWaves);
  const int bf16 = dtype == BF16;
  if (a.cache.head_dim == 64) return (int)launch_kernel(merge_kernel<64>, grid, block, s, a, nsplit, bf16);
  if (a.cache.head_dim == 128) return (int)launch_kernel(merge_kernel<128>, grid, block, s, a, nsplit, bf16);
  return (int)launch_kernel(merge_kernel<256>, grid, block, s, a, nsplit, bf16);
}

}  // namespace bq
