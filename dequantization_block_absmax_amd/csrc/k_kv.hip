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

#include "bq_kv_device.h"
#include "bq_launch.h"

namespace bq {
namespace {

// ---- write --------------------------------------------------------------------------------

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

  quantize_unit<KB, MODE, M>([&](int e) { return element<DT>(x, e); }, at.flat, sh.log2b, qa, s_lut, s_thr, ka.packed[side],
                             ka.absmax[side], tid);
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
