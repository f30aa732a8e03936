// k_kv_append.hip -- appending tokens to the paged cache with the rotation by position on the way, and rotating their
// queries, in one launch.
//
//   (x, y) of pair i at position t -> (fl32(fl32(x c) - fl32(y s)), fl32(fl32(y c) + fl32(x s))), c and s from the tables
//   keys: absmax, normalize and nearest rules of bq.h on the rotated binary32 values; values: the same as they are
//   queries: rounded once to their type
//
// Work decomposition.  The first workgroups take the keys' units of 8 elements, as kv_write_kernel does, the next ones the
// values', the others the queries'.  A key's lane needs the other elements of its pairs beside its own 8: where pairs lie
// rotary_dim / 2 apart it loads those 8 too (they come from the cache that the other lane fills).  A lane of the
// queries takes both sides of 8 pairs, so that q may be rotated in place, and of several heads, which share its cosines
// and sines.
//
// What bounds it.  Few tokens: the launch (48 tokens, 32 heads over 8 of 128, bf16, 4-bit: 3.8 us).  Many: memory, beside the places
// and searches of 8 elements that each lane works out: 16384 tokens, 32 over 8 of 128, bf16, 8-bit, B = 128: 91.6 us for 379 MB (projections
// and angles read, queries and codes written), 4.1 TB/s where a large copy reaches 5.0; 4099, 15 over 5 of 64, fp32, 4-bit, half of each
// head in neighbouring pairs: 12.5 us, 44 MB, 3.5 TB/s.
#include <hip/hip_runtime.h>

#include "bq_kv_device.h"
#include "bq_launch.h"

namespace bq {
namespace {

struct Angles {
  const float *cos, *sin;
  int64_t stride, max_positions;
  const int64_t* positions;
  uint32_t rotary, half;  // elements that rotate; pairs
  int32_t interleaved;
};

struct KvAppendKernelArgs {
  const uint8_t* in[2];
  int64_t stride[2];  // bytes between tokens
  float* absmax[2];
  uint8_t* packed[2];
  const uint8_t* q;
  uint8_t* q_out;
  int64_t q_stride, q_out_stride;  // bytes
  uint32_t kv_blocks;              // workgroups of the keys, and of the values
  // Items of the queries: (token, group of heads, place in the head), the last place fastest; places are 8 pairs each,
  // then (for another q_out) 8 elements each that stay.
  uint32_t items, row_items, head_items, heads, per;
  Divider by_row, by_head;
};

// The 8 floats at p (16-byte aligned).
__device__ __forceinline__ void load8(float (&v)[8], const float* p) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const u32x4 w = reinterpret_cast<const u32x4*>(p)[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * k + e] = bits_f32(w[e]);
  }
}

template <int DT>
__device__ __forceinline__ Unit<DT> load_unit(const uint8_t* p) {
  Unit<DT> x;
#pragma unroll
  for (int k = 0; k < (DT == F32 ? 2 : 1); ++k) {
    const u32x4 v = reinterpret_cast<const u32x4*>(p)[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) x.w[4 * k + e] = v[e];
  }
  return x;
}

// Rounded to DT (nearest, ties to even) and stored.
template <int DT>
__device__ __forceinline__ void store_unit(uint8_t* p, const float (&v)[8]) {
  Unit<DT> x;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (DT == F32) {
      x.w[e] = f32_bits(v[e]);
    } else {
      uint16_t h;
      if constexpr (DT == BF16) h = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
      else h = __builtin_bit_cast(uint16_t, (_Float16)v[e]);
      x.w[e >> 1] = e & 1 ? x.w[e >> 1] | (uint32_t)h << 16 : h;
    }
  }
#pragma unroll
  for (int k = 0; k < (DT == F32 ? 2 : 1); ++k)
    reinterpret_cast<u32x4*>(p)[k] = (u32x4){x.w[4 * k], x.w[4 * k + 1], x.w[4 * k + 2], x.w[4 * k + 3]};
}

__device__ __forceinline__ bool at_position(const Angles& an, uint32_t token, int64_t& t) {
  t = an.positions[token];
  const bool listed = t >= 0 && t < an.max_positions;
  t = listed ? t : 0;
  return listed;
}

// U heads of one item of the queries.
template <int DT, int U>
__device__ __forceinline__ void rotate_queries(const KvAppendKernelArgs& ka, const Angles& an, uint32_t head_bytes,
                                               uint32_t item) {
  constexpr uint32_t size = DT == F32 ? 4 : 2;
  const uint32_t token = divide(item, ka.by_row);
  const uint32_t c = item - token * ka.row_items;
  const uint32_t group = divide(c, ka.by_head), p = c - group * ka.head_items;
  int64_t t;
  if (!at_position(an, token, t)) return;
  const uint32_t head = group * U;
  const uint8_t* src = ka.q + (int64_t)token * ka.q_stride + (int64_t)head * head_bytes;
  uint8_t* dst = ka.q_out + (int64_t)token * ka.q_out_stride + (int64_t)head * head_bytes;
  const uint32_t pairs = an.rotary / 16;  // places of 8 pairs
  if (p >= pairs) {                       // 8 elements that stay
    const uint32_t d = (an.rotary + 8 * (p - pairs)) * size;
    if (src == dst || d >= head_bytes) return;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (head + u < ka.heads) {
#pragma unroll
        for (uint32_t k = 0; k < size / 2; ++k)
          reinterpret_cast<u32x4*>(dst + u * head_bytes + d)[k] = reinterpret_cast<const u32x4*>(src + u * head_bytes + d)[k];
      }
    return;
  }
  const uint32_t da = (an.interleaved ? 16 * p : 8 * p) * size, db = (an.interleaved ? 16 * p + 8 : 8 * p + an.half) * size;
  Unit<DT> a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {  // heads past the last repeat it
    const uint32_t at = (min(head + u, ka.heads - 1) - head) * head_bytes;
    a[u] = load_unit<DT>(src + at + da);
    b[u] = load_unit<DT>(src + at + db);
  }
  float cs[8], sn[8];
  load8(cs, an.cos + t * an.stride + 8 * p);
  load8(sn, an.sin + t * an.stride + 8 * p);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (head + u >= ka.heads) break;
    float x[8], y[8];
    if (an.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x0 = element<DT>(a[u], e), y0 = element<DT>(a[u], e + 1);
        const float x1 = element<DT>(b[u], e), y1 = element<DT>(b[u], e + 1);
        const int i = e / 2;
        x[e] = x0 * cs[i] - y0 * sn[i];
        x[e + 1] = y0 * cs[i] + x0 * sn[i];
        y[e] = x1 * cs[i + 4] - y1 * sn[i + 4];
        y[e + 1] = y1 * cs[i + 4] + x1 * sn[i + 4];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x0 = element<DT>(a[u], e), y0 = element<DT>(b[u], e);
        x[e] = x0 * cs[e] - y0 * sn[e];
        y[e] = y0 * cs[e] + x0 * sn[e];
      }
    }
    store_unit<DT>(dst + u * head_bytes + da, x);
    store_unit<DT>(dst + u * head_bytes + db, y);
  }
}

template <int DT, int KB, int MODE, int M>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendKernelArgs ka, KvShape sh, Angles an, QuantArgs qa) {
  using E = typename Entry<M>::type;
  constexpr uint32_t size = DT == F32 ? 4 : 2;
  __shared__ float s_thr[260];
  __shared__ E s_lut[LutLayout<MODE, M>::kSize];
  const int tid = threadIdx.x;
  if (blockIdx.x >= 2 * ka.kv_blocks) {
    const uint32_t item = (blockIdx.x - 2 * ka.kv_blocks) * (uint32_t)kThreads + tid;
    if (item >= ka.items) return;
    if (ka.per == 4) rotate_queries<DT, 4>(ka, an, sh.head_units * 8 * size, item);
    else rotate_queries<DT, 1>(ka, an, sh.head_units * 8 * size, item);
    return;
  }
  const int side = blockIdx.x >= ka.kv_blocks;
  const auto lw = lut_fetch<MODE, M, kThreads>(qa, tid);
  const uint32_t u = (blockIdx.x - (side ? ka.kv_blocks : 0)) * (uint32_t)kThreads + tid;
  Place at = place(min(u, sh.units - 1), sh);
  // lanes past the end repeat the last unit; whole blocks of them (units come in whole rows)
  if (u >= sh.units) at.flat = -1;
  const uint8_t* src = ka.in[side] + at.token * ka.stride[side] + (int64_t)at.col * size;
  const Unit<DT> x = load_unit<DT>(src);
  int64_t t;
  if (!at_position(an, at.token, t)) at.flat = -1;
  float v[8];
  if (side == 0 && at.d < an.rotary) {
    const float *cos = an.cos + t * an.stride, *sin = an.sin + t * an.stride;
    if (an.interleaved) {
      const u32x4 c4 = *reinterpret_cast<const u32x4*>(cos + at.d / 2), s4 = *reinterpret_cast<const u32x4*>(sin + at.d / 2);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x0 = element<DT>(x, e), y0 = element<DT>(x, e + 1), c = bits_f32(c4[e / 2]), s = bits_f32(s4[e / 2]);
        v[e] = x0 * c - y0 * s;
        v[e + 1] = y0 * c + x0 * s;
      }
    } else {
      const bool first = at.d < an.half;
      const uint32_t pair = first ? at.d : at.d - an.half;
      const Unit<DT> o = load_unit<DT>(first ? src + an.half * size : src - an.half * size);
      float cs[8], sn[8];
      load8(cs, cos + pair);
      load8(sn, sin + pair);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = element<DT>(o, e) * sn[e];
        v[e] = element<DT>(x, e) * cs[e] + (first ? -other : other);  // x - y as x + (-y)
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = element<DT>(x, e);
  }
  lut_fill<MODE, M, kThreads>(qa, lw, s_lut, s_thr, tid);
  quantize_unit<KB, MODE, M>([&](int e) { return v[e]; }, at.flat, sh.log2b, qa, s_lut, s_thr, ka.packed[side],
                             ka.absmax[side], tid);
}

// ---- launches -----------------------------------------------------------------------------

struct Launch {
  KvAppendKernelArgs ka;
  KvShape sh;
  Angles an;
  unsigned grid;
};

template <int DT, int KB, int MODE, int M>
hipError_t append_units(const Launch& l, const QuantArgs& qa, hipStream_t s) {
  return launch_kernel(kv_append_kernel<DT, KB, MODE, M>, dim3(l.grid), dim3(kThreads), s, l.ka, l.sh, l.an, qa);
}

template <int DT, int KB>
hipError_t append_mode(const Launch& l, const PreparedTable& t, hipStream_t s) {
  if (t.mode == LIN) {
    if (t.M <= 1) return append_units<DT, KB, LIN, 1>(l, t.qa, s);
    if (t.M == 2) return append_units<DT, KB, LIN, 2>(l, t.qa, s);
    return append_units<DT, KB, LIN, 3>(l, t.qa, s);
  }
  if (t.mode == F16B) return append_units<DT, KB, F16B, 1>(l, t.qa, s);
  if (t.mode == LOG) {
    if (t.M <= 1) return append_units<DT, KB, LOG, 1>(l, t.qa, s);
    if (t.M == 2) return append_units<DT, KB, LOG, 2>(l, t.qa, s);
    return append_units<DT, KB, LOG, 3>(l, t.qa, s);
  }
  return append_units<DT, KB, SEARCH, 1>(l, t.qa, s);
}

template <int DT>
hipError_t append_dt(const Launch& l, const PreparedTable& t, hipStream_t s) {
  return t.K == 16 ? append_mode<DT, 4>(l, t, s) : append_mode<DT, 8>(l, t, s);
}

}  // namespace

int launch_kv_append(const KvAppendArgs& a, int dtype, const PreparedTable& t, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t size = dtype == F32 ? 4 : 2;
  Launch l = {};
  l.sh = make_shape(a.cache, a.tokens, a.slots);
  l.an = {a.cos, a.sin, a.angle_stride, a.max_positions, a.positions, (uint32_t)a.rotary_dim, (uint32_t)a.rotary_dim / 2, a.interleaved};
  l.ka = {{static_cast<const uint8_t*>(a.k), static_cast<const uint8_t*>(a.v)},
          {a.k_stride * size, a.v_stride * size},
          {a.cache.absmax[0], a.cache.absmax[1]},
          {a.cache.packed[0], a.cache.packed[1]}};
  l.ka.kv_blocks = (l.sh.units + kThreads - 1) / kThreads;
  int64_t grid = 2 * (int64_t)l.ka.kv_blocks;
  if (a.q != nullptr) {
    const bool in_place = a.q == a.q_out;
    const uint32_t pairs = (uint32_t)a.rotary_dim / 16, stay = ((uint32_t)a.cache.head_dim - a.rotary_dim) / 8;
    l.ka.q = static_cast<const uint8_t*>(a.q);
    l.ka.q_out = static_cast<uint8_t*>(a.q_out);
    l.ka.q_stride = a.q_stride * size;
    l.ka.q_out_stride = a.q_out_stride * size;
    l.ka.heads = (uint32_t)a.heads;
    // at least two places to a head: the division's least
    l.ka.head_items = in_place ? (pairs < 2 ? 2 : pairs) : pairs + stay;
    // four heads to a lane once they fill the device
    l.ka.per = a.tokens * a.heads * l.ka.head_items >= (int64_t)cu_count() * 16 * kThreads ? 4 : 1;
    l.ka.row_items = (l.ka.heads + l.ka.per - 1) / l.ka.per * l.ka.head_items;
    l.ka.items = (uint32_t)(a.tokens * l.ka.row_items);
    l.ka.by_row = make_divider(l.ka.row_items);
    l.ka.by_head = make_divider(l.ka.head_items);
    grid += ((int64_t)l.ka.items + kThreads - 1) / kThreads;
  }
  if (grid > UINT32_MAX / kThreads) {
    g_launch_refused_for_size = true;
    return (int)hipErrorInvalidConfiguration;
  }
  l.grid = (unsigned)grid;
  if (dtype == F32) return (int)append_dt<F32>(l, t, s);
  if (dtype == F16) return (int)append_dt<F16>(l, t, s);
  return (int)append_dt<BF16>(l, t, s);
}

}  // namespace bq
