// k_kv.hip -- writing tokens into a paged key/value cache held in blockwise codes, and reading
// them back.
//
//   write   a = max |x| over the finite elements of a block, q = nearest code of x / a (the absmax,
//           normalize and nearest rules of bq.h), for the keys and the values of each token
//   read    out = RN(fl32(c[q] * a))
//
// The pool is the blockwise array of its elements (page, head, slot, d); B divides head_dim, so a
// block holds elements of one token's head, and a token's head is consecutive in the pool.
//
// Work decomposition.  A unit is 8 consecutive elements of one token's head.  Lane `tid` of a
// 256-lane workgroup handles units (tile * U + u) * 256 + tid, u < U, of the tokens' units in
// (token, head, d) order; grid row 0 takes the keys, row 1 the values.  A block is B / 8 = 4 .. 32
// neighbouring lanes, whose maximum is joined by lane permutes.  Both kernels stream; a decoding step is bound by the
// launch (3 us).  On MI355X:
//   write  one unit per lane, ordinary loads: 16384 tokens of 8 x 128 bf16 into 8-bit codes, B = 128, take 28.8 us from
//          HBM (3.5 TB/s of input and cache; about 22 vector instructions per element), 22.0 with the input in the last-level
//          cache; there two units 22.4, four 25.0, four with non-temporal loads 27.0
//   read   two units per lane where that leaves every CU several workgroups: 32768 tokens of 8 x 128 from
//          4-bit codes, B = 64, to bf16 take 28 us by themselves, 42 back to back on buffers in turn (4.1 TB/s,
//          3/4 of it writes; the codes' lines, two tokens of a head each, are fetched 1.4 times); by themselves, cached,
//          25.9, one unit 32.5, four 27.3, eight 29.9
#include <hip/hip_runtime.h>

#include "bq_device.h"
#include "bq_kv.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kThreads = 256;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// n / d for n < 2^31 by one multiplication: mul = ceil(2^(31+l) / d), l = ceil(log2 d), d >= 2.
struct Divider {
  uint32_t mul, shift;
};

Divider make_divider(uint32_t d) {
  uint32_t l = 1;
  while ((1u << l) < d) ++l;
  const uint64_t p = 1ull << (31 + l);
  return {(uint32_t)((p + d - 1) / d), l - 1};
}

__device__ __forceinline__ uint32_t divide(uint32_t n, Divider d) { return __umulhi(n, d.mul) >> d.shift; }

struct KvShape {
  uint32_t units;          // tokens * row_units, < 2^31
  uint32_t row_units;      // kv_heads * head_units
  uint32_t head_units;     // head_dim / 8
  Divider by_row, by_head;
  int32_t kv_heads, log2_page, log2b;
  int64_t slots;           // num_pages * page_size
  const int64_t* slot;     // one per token
};

// Where a unit lives: its token, its offset in the token's row (elements) and its flat element in
// the pool (-1: no such slot).
struct Place {
  uint32_t token, col;
  int64_t flat;
};

__device__ __forceinline__ Place place(uint32_t u, const KvShape& sh) {
  Place p;
  p.token = divide(u, sh.by_row);
  const uint32_t c = u - p.token * sh.row_units;
  p.col = c * 8;
  const uint32_t head = divide(c, sh.by_head);
  const uint32_t d = (c - head * sh.head_units) * 8;
  const int64_t slot = sh.slot[p.token];
  const int64_t page = slot >> sh.log2_page;
  const int64_t in_page = slot & ((1 << sh.log2_page) - 1);
  const int64_t row = ((page * sh.kv_heads + head) << sh.log2_page) + in_page;
  p.flat = slot >= 0 && slot < sh.slots ? row * (int64_t)(sh.head_units * 8) + d : -1;
  return p;
}

// ---- write --------------------------------------------------------------------------------

template <int DT>
struct Unit {
  uint32_t w[DT == F32 ? 8 : 4];
};

template <int DT>
__device__ __forceinline__ float element(const Unit<DT>& x, int e) {
  if constexpr (DT == F32) {
    return bits_f32(x.w[e]);
  } else if constexpr (DT == BF16) {
    return bits_f32((e & 1) ? (x.w[e >> 1] & 0xffff0000u) : (x.w[e >> 1] << 16));
  } else {
    const uint32_t v = x.w[e >> 1];
    return (float)__builtin_bit_cast(_Float16, (unsigned short)((e & 1) ? v >> 16 : v & 0xffffu));
  }
}

struct KvWriteArgs {
  const uint8_t* in[2];
  int64_t stride[2];  // bytes between tokens
  float* absmax[2];
  uint8_t* packed[2];
};

template <int DT, int KB, int MODE, int M>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvWriteArgs ka, KvShape sh, QuantArgs qa) {
  using E = typename Entry<M>::type;
  __shared__ float s_thr[260];
  __shared__ E s_lut[LutLayout<MODE, M>::kSize];
  const int tid = threadIdx.x;
  const int side = blockIdx.y;
  const uint8_t* in = ka.in[side];
  const int64_t stride = ka.stride[side];

  const auto lw = lut_fetch<MODE, M, kThreads>(qa, tid);
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + tid;
  Place at = place(min(u, sh.units - 1), sh);
  // lanes past the end repeat the last unit; whole blocks of them (units come in whole rows)
  if (u >= sh.units) at.flat = -1;
  const u32x4* src = reinterpret_cast<const u32x4*>(in + at.token * stride + (int64_t)at.col * (DT == F32 ? 4 : 2));
  Unit<DT> x;
#pragma unroll
  for (int k = 0; k < (DT == F32 ? 2 : 1); ++k) {
    const u32x4 v = src[k];
    x.w[4 * k] = v.x;
    x.w[4 * k + 1] = v.y;
    x.w[4 * k + 2] = v.z;
    x.w[4 * k + 3] = v.w;
  }
  lut_fill<MODE, M, kThreads>(qa, lw, s_lut, s_thr, tid);

  // Block maximum over finite elements, as the bits of |x| (ordered like the values).
  const int lanes = 1 << (sh.log2b - 3);  // lanes of a block
  uint32_t m = 0;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = f32_bits(element<DT>(x, e)) & 0x7fffffffu;
    finite = finite && b < 0x7f800000u;
    m = max(m, b < 0x7f800000u ? b : 0u);
  }
  m = group_max_u32(m, lanes);
  const float a = bits_f32(m);
  const float s = a < 0x1p-64f ? 0x1p64f : (a > 0x1p64f ? 0x1p-64f : 1.0f);
  const float r = 1.0f / (a * s);
  uint32_t q[8];
  if (__builtin_expect(__all(finite && s == 1.0f && a > 0.0f), 1)) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      nearest_pair<MODE, M>(element<DT>(x, e) * r, element<DT>(x, e + 1) * r, qa, s_lut, s_thr, q[e], q[e + 1]);
  } else {
    // a non-finite element and every element of a zero block take y = 0, whose code is z
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = element<DT>(x, e);
      const float y = (v * s) * r;
      q[e] = nearest_code<MODE, M>(a > 0.0f && fabsf(v) <= 0x1.fffffep127f ? y : 0.0f, qa, s_lut, s_thr);
    }
  }
  if (at.flat >= 0) {
    if constexpr (KB == 4) {
      *reinterpret_cast<uint32_t*>(ka.packed[side] + (at.flat >> 1)) = pack_word<4>(q);
    } else {
      const u32x2 w = {pack_word<8>(q), pack_word<8>(q + 4)};
      *reinterpret_cast<u32x2*>(ka.packed[side] + at.flat) = w;
    }
    if ((tid & (lanes - 1)) == 0) ka.absmax[side][at.flat >> sh.log2b] = a;
  }
}

// ---- read ---------------------------------------------------------------------------------

struct KvReadArgs {
  uint8_t* out[2];
  int64_t stride[2];  // bytes between tokens
  const float* absmax[2];
  const uint8_t* packed[2];
};

template <int DT, int KB, int U>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs ka, KvShape sh, DequantArgs da) {
  __shared__ float s_c[256];
  const int tid = threadIdx.x;
  const int side = blockIdx.y;
  const uint8_t* packed = ka.packed[side];
  const float* absmax = ka.absmax[side];
  const float c = da.c[tid];  // entries past K are zero
  Place at[U];
  u32x2 raw[U];
  float a[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = (blockIdx.x * U + i) * (uint32_t)kThreads + tid;
    at[i] = place(min(u, sh.units - 1), sh);
    const int64_t f = max(at[i].flat, (int64_t)0);  // a slot outside the pool reads the first, and gives zeros
    if constexpr (KB == 4) {
      raw[i] = (u32x2){*reinterpret_cast<const uint32_t*>(packed + (f >> 1)), 0u};
    } else {
      raw[i] = *reinterpret_cast<const u32x2*>(packed + f);
    }
    a[i] = absmax[f >> sh.log2b];
  }
  s_c[tid] = c;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = (blockIdx.x * U + i) * (uint32_t)kThreads + tid;
    if (u >= sh.units) break;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t q;
      if constexpr (KB == 4) q = (raw[i].x >> (8 * (e >> 1) + ((e & 1) ? 0 : 4))) & 15u;
      else q = ((e < 4 ? raw[i].x : raw[i].y) >> (8 * (e & 3))) & 255u;
      v[e] = at[i].flat >= 0 ? s_c[q] * a[i] : 0.0f;
      // rounded to binary32 before the conversion (a fused mixed-precision fma would round once)
      if constexpr (DT == F16) asm("" : "+v"(v[e]));
    }
    uint8_t* dst = ka.out[side] + at[i].token * ka.stride[side] + (int64_t)at[i].col * (DT == F32 ? 4 : 2);
    if constexpr (DT == F32) {
      const u32x4 lo = {f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])};
      const u32x4 hi = {f32_bits(v[4]), f32_bits(v[5]), f32_bits(v[6]), f32_bits(v[7])};
      __builtin_nontemporal_store(lo, reinterpret_cast<u32x4*>(dst));
      __builtin_nontemporal_store(hi, reinterpret_cast<u32x4*>(dst + 16));
    } else {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint16_t lo, hi;
        if constexpr (DT == BF16) {
          lo = __builtin_bit_cast(uint16_t, (__bf16)v[2 * k]);
          hi = __builtin_bit_cast(uint16_t, (__bf16)v[2 * k + 1]);
        } else {
          lo = __builtin_bit_cast(uint16_t, (_Float16)v[2 * k]);
          hi = __builtin_bit_cast(uint16_t, (_Float16)v[2 * k + 1]);
        }
        w[k] = (uint32_t)lo | ((uint32_t)hi << 16);
      }
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(dst));
    }
  }
}

// ---- launches -----------------------------------------------------------------------------

KvShape make_shape(const KvCacheArgs& c, int64_t tokens, const int64_t* slots) {
  KvShape sh;
  sh.head_units = (uint32_t)c.head_dim / 8;
  sh.row_units = (uint32_t)c.kv_heads * sh.head_units;
  sh.units = (uint32_t)(tokens * sh.row_units);
  sh.by_row = make_divider(sh.row_units);
  sh.by_head = make_divider(sh.head_units);
  sh.kv_heads = c.kv_heads;
  sh.log2_page = c.log2_page;
  sh.log2b = c.log2b;
  sh.slots = (int64_t)c.num_pages << c.log2_page;
  sh.slot = slots;
  return sh;
}

// Units per lane of a read: 2 once tiles of 2 give every CU four workgroups.
int units_per_lane(const KvShape& sh) { return (int64_t)sh.units >= (int64_t)cu_count() * 4 * kThreads ? 2 : 1; }

dim3 kv_grid(const KvShape& sh, int u) {
  return dim3((unsigned)(((int64_t)sh.units + u * kThreads - 1) / (u * kThreads)), 2);
}

template <int DT, int KB, int MODE, int M>
hipError_t write_units(const KvWriteArgs& ka, const KvShape& sh, const QuantArgs& qa, hipStream_t s) {
  return launch_kernel(kv_write_kernel<DT, KB, MODE, M>, kv_grid(sh, 1), dim3(kThreads), s, ka, sh, qa);
}

template <int DT, int KB>
hipError_t write_mode(const KvWriteArgs& ka, const KvShape& sh, const PreparedTable& t, hipStream_t s) {
  if (t.mode == LIN) {
    if (t.M <= 1) return write_units<DT, KB, LIN, 1>(ka, sh, t.qa, s);
    if (t.M == 2) return write_units<DT, KB, LIN, 2>(ka, sh, t.qa, s);
    return write_units<DT, KB, LIN, 3>(ka, sh, t.qa, s);
  }
  if (t.mode == F16B) return write_units<DT, KB, F16B, 1>(ka, sh, t.qa, s);
  if (t.mode == LOG) {
    if (t.M <= 1) return write_units<DT, KB, LOG, 1>(ka, sh, t.qa, s);
    if (t.M == 2) return write_units<DT, KB, LOG, 2>(ka, sh, t.qa, s);
    return write_units<DT, KB, LOG, 3>(ka, sh, t.qa, s);
  }
  return write_units<DT, KB, SEARCH, 1>(ka, sh, t.qa, s);
}

template <int DT>
hipError_t write_dt(const KvWriteArgs& ka, const KvShape& sh, const PreparedTable& t, hipStream_t s) {
  return t.K == 16 ? write_mode<DT, 4>(ka, sh, t, s) : write_mode<DT, 8>(ka, sh, t, s);
}

template <int DT, int KB>
hipError_t read_units(const KvReadArgs& ka, const KvShape& sh, const DequantArgs& da, hipStream_t s) {
  if (units_per_lane(sh) == 2)
    return launch_kernel(kv_read_kernel<DT, KB, 2>, kv_grid(sh, 2), dim3(kThreads), s, ka, sh, da);
  return launch_kernel(kv_read_kernel<DT, KB, 1>, kv_grid(sh, 1), dim3(kThreads), s, ka, sh, da);
}

template <int DT>
hipError_t read_dt(const KvReadArgs& ka, const KvShape& sh, const DequantArgs& da, hipStream_t s) {
  return da.K == 16 ? read_units<DT, 4>(ka, sh, da, s) : read_units<DT, 8>(ka, sh, da, s);
}

}  // namespace

int launch_kv_write(const KvCacheArgs& c, int dtype, const void* k, const void* v, int64_t tokens, int64_t k_stride,
                    int64_t v_stride, const int64_t* slots, const PreparedTable& t, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t size = dtype == F32 ? 4 : 2;
  const KvWriteArgs ka = {{static_cast<const uint8_t*>(k), static_cast<const uint8_t*>(v)},
                          {k_stride * size, v_stride * size},
                          {c.absmax[0], c.absmax[1]},
                          {c.packed[0], c.packed[1]}};
  const KvShape sh = make_shape(c, tokens, slots);
  if (dtype == F32) return (int)write_dt<F32>(ka, sh, t, s);
  if (dtype == F16) return (int)write_dt<F16>(ka, sh, t, s);
  return (int)write_dt<BF16>(ka, sh, t, s);
}

int launch_kv_read(const KvCacheArgs& c, int dtype, void* k, void* v, int64_t tokens, int64_t k_stride,
                   int64_t v_stride, const int64_t* slots, const DequantArgs& da, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t size = dtype == F32 ? 4 : 2;
  const KvReadArgs ka = {{static_cast<uint8_t*>(k), static_cast<uint8_t*>(v)},
                         {k_stride * size, v_stride * size},
                         {c.absmax[0], c.absmax[1]},
                         {c.packed[0], c.packed[1]}};
  const KvShape sh = make_shape(c, tokens, slots);
  if (dtype == F32) return (int)read_dt<F32>(ka, sh, da, s);
  if (dtype == F16) return (int)read_dt<F16>(ka, sh, da, s);
  return (int)read_dt<BF16>(ka, sh, da, s);
}

}  // namespace bq
