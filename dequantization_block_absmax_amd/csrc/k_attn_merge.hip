// k_attn_merge.hip -- joins the partial results of the splits of an attention call.
//
// A row's splits hold (M_s, l_s) and sums o_s relative to their own reference exponent M_s; with
// M = max_s M_s:  o = sum_s 2^(M_s - M) o_s / sum_s 2^(M_s - M) l_s, in a fixed order.
//
// Few splits (up to 16): D / 4 lanes take a row, 4 / (D / 64) rows to a wave.  More: four waves take a row, wave
// w its splits w, w + 4, ..., lane by lane over head_dim, eight loads in flight (64 splits of one row
// one after another took 20 us, 4.5 us so).  Bound by latency where few rows were split (3 to
// 5 us); by the partial sums' bytes where many were: 6216 rows of 256 over 5 splits (32 MB, written and read once) take
// 7.6 us here, 4.2 TB/s, and about 6 us of the kernel before.
#include <hip/hip_runtime.h>

#include "bq_attn.h"
#include "bq_kv.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kWaves = 4;

// New tokens beside each of N rows of q in their sequences (0: in none).  The wave looks at 64 sequences at a
// time.
template <int N>
__device__ __forceinline__ void tokens_beside(const KvAttendArgs& aa, const int64_t (&token)[N], int lane, int (&count)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) count[k] = 0;
  for (int s0 = 0; s0 < aa.num_seqs; s0 += 64) {
    const int s = min(s0 + lane, aa.num_seqs - 1);
    const int first = row_number(aa, aa.q_start[s]);
    const int nq = min(row_number(aa, aa.q_start[s + 1]) - first, aa.max_q_len);
    bool all = true;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint64_t mine = __ballot(token[k] >= first && token[k] < (int64_t)first + nq);
      if (mine != 0 && count[k] == 0) count[k] = __builtin_amdgcn_readlane(nq, __builtin_ctzll(mine));
      all = all && count[k] != 0;
    }
    if (all) break;
  }
}

// Where a row's partial results are; nsplit 0: nothing to join.
struct Source {
  const float* sums;
  const Partial* parts;
  int nsplit;
};

template <int D>
__device__ __forceinline__ Source source(const KvAttendArgs& aa, const MergeArgs& ma, int64_t at, int nq) {
  const int kind = ma.both ? many_rows(nq, aa.heads / aa.cache.kv_heads, aa.num_seqs) : ma.kind;
  const int n = kind ? ma.nsplit[1] : ma.nsplit[0];
  const float* base = kind ? ma.partial[1] : ma.partial[0];
  Source s;
  s.nsplit = nq > 0 && n > 1 ? n : 0;
  s.sums = base + at * n * D;
  s.parts = reinterpret_cast<const Partial*>(base + aa.tokens * aa.heads * n * D) + at * n;
  return s;
}

__device__ __forceinline__ float inverse(float l) { return l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l); }

template <int D>
__global__ __launch_bounds__(64 * kWaves) void merge_few_kernel(KvAttendArgs aa, MergeArgs ma, int bf16) {
  constexpr int kLanes = D / 4, kRows = 64 / kLanes;  // lanes of a row, rows of a wave
  const int lane = threadIdx.x & 63;
  const int64_t rows = aa.tokens * aa.heads;
  const int64_t at0 = ((int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kRows;
  if (at0 >= rows) return;
  int64_t token[kRows];
  int count[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) token[k] = min(at0 + k, rows - 1) / aa.heads;
  tokens_beside(aa, token, lane, count);
  const int64_t at = at0 + lane / kLanes;  // token * heads + head
  int nq = 0;
  int64_t mine = 0;
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (lane / kLanes == k) {
      nq = count[k];
      mine = token[k];
    }
  const Source src = source<D>(aa, ma, at, at < rows ? nq : 0);
  if (src.nsplit == 0) return;
  const int d = lane % kLanes * 4;
  float top = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < src.nsplit; ++s) top = fmaxf(top, src.parts[s].m);
  float l = 0.0f, exact = 0.0f;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < src.nsplit; ++s) {
    const Partial p = src.parts[s];
    const f32x4 x = *reinterpret_cast<const f32x4*>(src.sums + (int64_t)s * D + d);
    const float f = p.m == -INFINITY ? 0.0f : exp2_hw(p.m - top);
    l += lower(p.l, p.m, top);
    exact += lower(p.exact, p.m, top);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(f, x[k], v[k]);
  }
  const float inv = inverse(l);
  const int64_t head = at - mine * aa.heads;
  const u32x2 o = {pack16(v[0] * inv, v[1] * inv, bf16), pack16(v[2] * inv, v[3] * inv, bf16)};
  *reinterpret_cast<u32x2*>(static_cast<char*>(aa.out) + (mine * aa.out_stride + head * D + d) * 2) = o;
  if (aa.lse != nullptr && d == 0) aa.lse[at] = log_sum(top, exact);
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void merge_kernel(KvAttendArgs aa, MergeArgs ma, int bf16) {
  constexpr int kPer = D / 64;
  __shared__ float s_sum[kWaves][D];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t at = blockIdx.x;  // token * heads + head
  const int64_t token[1] = {at / aa.heads};
  int nq[1];
  tokens_beside(aa, token, lane, nq);
  const Source src = source<D>(aa, ma, at, nq[0]);
  if (src.nsplit == 0) return;
  const Partial mine = lane < src.nsplit ? src.parts[lane] : Partial{-INFINITY, 0.0f, 0.0f};
  float top = mine.m;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float f = mine.m == -INFINITY ? 0.0f : exp2_hw(mine.m - top);
  float l = lower(mine.l, mine.m, top), exact = lower(mine.exact, mine.m, top);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    l += __shfl_xor(l, x);
    exact += __shfl_xor(exact, x);
  }
  float v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] = 0.0f;
  // splits past the last repeat it with weight zero, so that no load sits under a condition
  constexpr int kFlight = D <= 128 ? 8 : 4;
  for (int s0 = wave; s0 < src.nsplit; s0 += kFlight * kWaves) {
    float x[kFlight][kPer];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const float* at_split = src.sums + (int64_t)min(s0 + i * kWaves, src.nsplit - 1) * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[i][k] = at_split[k];
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int s = s0 + i * kWaves;
      const float fs = s < src.nsplit ? bits_f32(__builtin_amdgcn_readlane(f32_bits(f), min(s, 63))) : 0.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = fmaf(fs, x[i][k], v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) s_sum[wave][lane * kPer + k] = v[k];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int d = lane * kPer + k;
    v[k] = (s_sum[0][d] + s_sum[1][d]) + (s_sum[2][d] + s_sum[3][d]);
  }
  const float inv = inverse(l);
  const int64_t head = at - token[0] * aa.heads;
  uint16_t* out = static_cast<uint16_t*>(aa.out) + token[0] * aa.out_stride + head * D + lane * kPer;
  if constexpr (kPer == 1) {
    *out = (uint16_t)pack16(v[0] * inv, 0.0f, bf16);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; k += 2) reinterpret_cast<uint32_t*>(out)[k / 2] = pack16(v[k] * inv, v[k + 1] * inv, bf16);
  }
  if (aa.lse != nullptr && lane == 0) aa.lse[at] = log_sum(top, exact);
}

// A launch counts threads in 32 bits.
constexpr int64_t kMostWorkgroups = (int64_t)UINT32_MAX / (64 * kWaves);

// Workgroups of merge_few_kernel.
int64_t few_workgroups(const KvAttendArgs& a) {
  const int64_t per = kWaves * (64 / (a.cache.head_dim / 4));
  return (a.tokens * a.heads + per - 1) / per;
}

template <int D>
hipError_t launch_dim(const KvAttendArgs& a, const MergeArgs& m, int bf16, hipStream_t s) {
  const int64_t rows = a.tokens * a.heads;
  if ((m.nsplit[0] > 16 || m.nsplit[1] > 16) && rows <= kMostWorkgroups)
    return launch_kernel(merge_kernel<D>, dim3((unsigned)rows), dim3(64 * kWaves), s, a, m, bf16);
  return launch_kernel(merge_few_kernel<D>, dim3((unsigned)few_workgroups(a)), dim3(64 * kWaves), s, a, m, bf16);
}

}  // namespace

bool kv_merge_fits(const KvAttendArgs& a) { return few_workgroups(a) <= kMostWorkgroups; }

int launch_kv_merge(const KvAttendArgs& a, int dtype, const MergeArgs& m, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int bf16 = dtype == BF16;
  if (a.cache.head_dim == 64) return (int)launch_dim<64>(a, m, bf16, s);
  if (a.cache.head_dim == 128) return (int)launch_dim<128>(a, m, bf16, s);
  return (int)launch_dim<256>(a, m, bf16, s);
}

}  // namespace bq
