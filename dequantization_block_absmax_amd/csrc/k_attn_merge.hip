// k_attn_merge.hip -- joins the partial results of the splits of an attention call.
//
// A row's splits hold (M_s, l_s) and sums o_s relative to their own reference exponent M_s; with
// M = max_s M_s:  o = sum_s 2^(M_s - M) o_s / sum_s 2^(M_s - M) l_s, in split order.  One wave per row:
// lane s works out split s's factor, then the lanes take head_dim.  Bound by latency: a call's
// partial sums are a small part of its cache.
#include <hip/hip_runtime.h>

#include "bq_attn.h"
#include "bq_internal.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kWaves = 4;

template <int D>
__global__ __launch_bounds__(64 * kWaves) void merge_kernel(KvAttendArgs aa, int nsplit, int bf16) {
  const int lane = threadIdx.x & 63;
  const Sequence sq = sequence(aa, blockIdx.y);
  const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (row >= (int64_t)min(sq.nq, aa.max_q_len) * aa.heads) return;
  const int64_t at = (int64_t)sq.q0 * aa.heads + row;  // token * heads + head
  const float* sums = static_cast<const float*>(aa.workspace) + at * nsplit * D;
  const Partial* parts =
      reinterpret_cast<const Partial*>(static_cast<const float*>(aa.workspace) + aa.tokens * aa.heads * nsplit * D) +
      at * nsplit;
  const Partial mine = lane < nsplit ? parts[lane] : Partial{-INFINITY, 0.0f};
  float top = mine.m;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float f = mine.m == -INFINITY ? 0.0f : exp2_hw(mine.m - top);
  float l = f * mine.l;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);

  constexpr int kPer = D / 64;
  float v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < nsplit; ++s) {
    const float fs = bits_f32(__builtin_amdgcn_readlane(f32_bits(f), s));
    const float* src = sums + (int64_t)s * D + lane * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = fmaf(fs, src[k], v[k]);
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  const int64_t token = at / aa.heads, head = at - token * aa.heads;
  uint16_t* out = static_cast<uint16_t*>(aa.out) + token * aa.out_stride + head * D + lane * kPer;
  if constexpr (kPer == 1) {
    *out = (uint16_t)pack16(v[0] * inv, 0.0f, bf16);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; k += 2) reinterpret_cast<uint32_t*>(out)[k / 2] = pack16(v[k] * inv, v[k + 1] * inv, bf16);
  }
  if (aa.lse != nullptr && lane == 0) aa.lse[at] = log_sum(top, l);
}

}  // namespace

int launch_kv_merge(const KvAttendArgs& a, int dtype, int nsplit, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(((int64_t)a.max_q_len * a.heads + kWaves - 1) / kWaves), (unsigned)a.num_seqs);
  const dim3 block(64 * kWaves);
  const int bf16 = dtype == BF16;
  if (a.cache.head_dim == 64) return (int)launch_kernel(merge_kernel<64>, grid, block, s, a, nsplit, bf16);
  if (a.cache.head_dim == 128) return (int)launch_kernel(merge_kernel<128>, grid, block, s, a, nsplit, bf16);
  return (int)launch_kernel(merge_kernel<256>, grid, block, s, a, nsplit, bf16);
}

}  // namespace bq
