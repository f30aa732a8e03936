// k_attn_merge.hip -- joins the partial results of the splits of an attention call.
//
// A row's splits hold (M_s, l_s) and sums o_s relative to their own reference exponent M_s; with
// M = max_s M_s:  o = sum_s 2^(M_s - M) o_s / sum_s 2^(M_s - M) l_s, in a fixed order.
//
// WPR waves take a row: wave w its splits w, w + WPR, ..., lane by lane over head_dim, eight loads in
// flight.  Bound by latency: a call's partial sums are a small part of its cache.  One wave suffices for up
// to 16 splits, and four rows to a workgroup then; more splits take four waves (64 splits of one row
// one after another took 20 us, 4.5 us so).
#include <hip/hip_runtime.h>

#include "bq_attn.h"
#include "bq_internal.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kWaves = 4;

// New tokens of the sequence that a row of q belongs to (0: none).  The wave looks at 64 sequences at a time.
__device__ __forceinline__ int tokens_beside(const KvAttendArgs& aa, int64_t token, int lane) {
  for (int s0 = 0; s0 < aa.num_seqs; s0 += 64) {
    const int s = min(s0 + lane, aa.num_seqs - 1);
    const int first = max(aa.q_start[s], 0);
    const int last = (int)min((int64_t)aa.q_start[s + 1], aa.tokens);
    const int nq = min(last - first, aa.max_q_len);
    const uint64_t mine = __ballot(token >= first && token < (int64_t)first + nq);
    if (mine != 0) return __builtin_amdgcn_readlane(nq, __builtin_ctzll(mine));
  }
  return 0;
}

template <int D, int WPR>
__global__ __launch_bounds__(64 * kWaves) void merge_kernel(KvAttendArgs aa, MergeArgs ma, int bf16) {
  constexpr int kPer = D / 64;
  __shared__ float s_sum[WPR > 1 ? kWaves : 1][D];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = WPR > 1 ? wave : 0;
  const int64_t at = WPR > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kWaves + wave;  // token * heads + head
  if (at >= aa.tokens * aa.heads) return;
  const int64_t token = at / aa.heads, head = at - token * aa.heads;
  const int nq = tokens_beside(aa, token, lane);
  if (nq == 0) return;
  const int kind = ma.both ? many_rows(nq, aa.heads / aa.cache.kv_heads, aa.num_seqs) : ma.kind;
  const int nsplit = ma.nsplit[kind];
  if (nsplit <= 1) return;
  const float* sums = ma.partial[kind] + at * nsplit * D;
  const Partial* parts = reinterpret_cast<const Partial*>(ma.partial[kind] + aa.tokens * aa.heads * nsplit * D) + at * nsplit;
  const Partial mine = lane < nsplit ? parts[lane] : Partial{-INFINITY, 0.0f};
  float top = mine.m;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float f = mine.m == -INFINITY ? 0.0f : exp2_hw(mine.m - top);
  float l = f * mine.l;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
  float v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] = 0.0f;
  // splits past the last repeat it with weight zero, so that no load sits under a condition
  constexpr int kFlight = D <= 128 ? 8 : 4;
  for (int s0 = part; s0 < nsplit; s0 += kFlight * WPR) {
    float x[kFlight][kPer];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const float* src = sums + (int64_t)min(s0 + i * WPR, nsplit - 1) * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[i][k] = src[k];
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int s = s0 + i * WPR;
      const float fs = s < nsplit ? bits_f32(__builtin_amdgcn_readlane(f32_bits(f), min(s, 63))) : 0.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = fmaf(fs, x[i][k], v[k]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) s_sum[wave][lane * kPer + k] = v[k];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int d = lane * kPer + k;
      v[k] = (s_sum[0][d] + s_sum[1][d]) + (s_sum[2][d] + s_sum[3][d]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  uint16_t* out = static_cast<uint16_t*>(aa.out) + token * aa.out_stride + head * D + lane * kPer;
  if constexpr (kPer == 1) {
    *out = (uint16_t)pack16(v[0] * inv, 0.0f, bf16);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; k += 2) reinterpret_cast<uint32_t*>(out)[k / 2] = pack16(v[k] * inv, v[k + 1] * inv, bf16);
  }
  if (aa.lse != nullptr && lane == 0) aa.lse[at] = log_sum(top, l);
}

template <int D>
hipError_t launch_dim(const KvAttendArgs& a, const MergeArgs& m, int bf16, hipStream_t s) {
  const int64_t rows = a.tokens * a.heads;
  if (m.nsplit[0] > 16 || m.nsplit[1] > 16)
    return launch_kernel(merge_kernel<D, kWaves>, dim3((unsigned)rows), dim3(64 * kWaves), s, a, m, bf16);
  return launch_kernel(merge_kernel<D, 1>, dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(64 * kWaves), s, a, m, bf16);
}

}  // namespace

int launch_kv_merge(const KvAttendArgs& a, int dtype, const MergeArgs& m, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int bf16 = dtype == BF16;
  if (a.tokens * a.heads > INT32_MAX) {
    g_launch_refused_for_size = true;
    return (int)hipErrorInvalidConfiguration;
  }
  if (a.cache.head_dim == 64) return (int)launch_dim<64>(a, m, bf16, s);
  if (a.cache.head_dim == 128) return (int)launch_dim<128>(a, m, bf16, s);
  return (int)launch_dim<256>(a, m, bf16, s);
}

}  // namespace bq
