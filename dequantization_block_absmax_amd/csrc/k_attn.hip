// k_attn.hip -- attention of new tokens over a paged key/value cache held in blockwise codes.
//
//   o_i = sum_j p_ij v_j,   p_ij = exp(s_ij) / sum_j exp(s_ij),   s_ij = scale * (q_i . k_j)
// over the keys j that row i sees; k and v are the cached values fl32(c[code] * absmax).
//
// One wave per (token, query head): 64 keys at a time, a lane to a key for the scores, then lanes
// over head_dim for the sum of values, with the running maximum and sum of the softmax.
#include <hip/hip_runtime.h>

#include "bq_internal.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <int DT>
__device__ __forceinline__ float load16(const uint16_t* p) {
  if constexpr (DT == BF16) return bits_f32((uint32_t)*p << 16);
  else return (float)__builtin_bit_cast(_Float16, *p);
}

template <int DT>
__device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (DT == BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <int KB>
__device__ __forceinline__ float value(const uint8_t* packed, const float* absmax, int64_t flat, int log2b,
                                       const float* s_c) {
  uint32_t q;
  if constexpr (KB == 4) q = (packed[flat >> 1] >> ((flat & 1) ? 0 : 4)) & 15u;
  else q = packed[flat];
  return s_c[q] * absmax[flat >> log2b];
}

template <int DT, int KB>
__global__ __launch_bounds__(64 * kWaves) void attend_kernel(KvAttendArgs aa, DequantArgs da) {
  __shared__ float s_c[256];
  __shared__ float s_q[kWaves][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  s_c[tid] = da.c[tid];
  const int seq = blockIdx.z;
  const int D = aa.cache.head_dim;
  const int group = aa.heads / aa.cache.kv_heads;
  const int64_t row = (int64_t)blockIdx.x * kWaves + wave;
  const int i = (int)(row / aa.heads), head = (int)(row % aa.heads);
  const int q0 = max(aa.q_start[seq], 0);
  const int q1 = (int)min((int64_t)aa.q_start[seq + 1], aa.tokens);
  const bool live = i < min(q1 - q0, aa.max_q_len);
  const int64_t token = live ? q0 + i : 0;
  const uint16_t* q = static_cast<const uint16_t*>(aa.q) + token * aa.q_stride + (int64_t)head * D;
  if (live)
    for (int d = lane; d < D; d += 64) s_q[wave][d] = load16<DT>(q + d);
  __syncthreads();
  if (!live) return;

  const int kv = (int)min((int64_t)max(min(aa.kv_len[seq], aa.max_kv_len), 0), aa.table_stride << aa.cache.log2_page);
  const int pos = kv - (q1 - q0) + i;
  const int hi = aa.causal ? min(kv, pos + 1) : kv;
  const int lo = aa.window > 0 && pos >= aa.window ? pos - aa.window + 1 : 0;
  const int ps = 1 << aa.cache.log2_page;
  const int kvh = head / group;

  float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane;
    float s = -INFINITY;
    int64_t flat = 0;
    if (j < hi) {
      const int page = aa.page_table[seq * aa.table_stride + (j >> aa.cache.log2_page)];
      if (page >= 0 && page < aa.cache.num_pages) {
        flat = (((int64_t)page * aa.cache.kv_heads + kvh) * ps + (j & (ps - 1))) * D;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d)
          dot = fmaf(s_q[wave][d], value<KB>(aa.cache.packed[0], aa.cache.absmax[0], flat + d, aa.cache.log2b, s_c), dot);
        s = dot * aa.scale;
      }
    }
    const float mn = fmaxf(m, wave_max(s));
    if (mn == -INFINITY) continue;
    const float alpha = expf(m - mn);
    const float p = s == -INFINITY ? 0.0f : expf(s - mn);
    l = l * alpha + wave_sum(p);
    m = mn;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= alpha;
    for (int t = 0; t < 64; ++t) {
      const float pt = __shfl(p, t);
      const int64_t ft = __shfl(flat, t);
      if (pt == 0.0f) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane + 64 * k < D)
          acc[k] = fmaf(pt, value<KB>(aa.cache.packed[1], aa.cache.absmax[1], ft + lane + 64 * k, aa.cache.log2b, s_c),
                        acc[k]);
    }
  }
  uint16_t* out = static_cast<uint16_t*>(aa.out) + token * aa.out_stride + (int64_t)head * D;
  const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (lane + 64 * k < D) out[lane + 64 * k] = to16<DT>(acc[k] * inv);
  if (aa.lse != nullptr && lane == 0) aa.lse[token * aa.heads + head] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv_attend_workspace(const KvAttendArgs&, int) { return 0; }

int launch_kv_attend(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(((int64_t)a.max_q_len * a.heads + kWaves - 1) / kWaves), 1, (unsigned)a.num_seqs);
  const dim3 block(64 * kWaves);
  if (dtype == BF16)
    return (int)(da.K == 16 ? launch_kernel(attend_kernel<BF16, 4>, grid, block, s, a, da)
                            : launch_kernel(attend_kernel<BF16, 8>, grid, block, s, a, da));
  return (int)(da.K == 16 ? launch_kernel(attend_kernel<F16, 4>, grid, block, s, a, da)
                          : launch_kernel(attend_kernel<F16, 8>, grid, block, s, a, da));
}

}  // namespace bq
