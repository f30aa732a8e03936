// bq_kv_device.h -- what the kernels that write tokens into the paged cache and read them back share (k_kv.hip,
// k_kv_append.hip): units of 8 elements, where they live, and their quantization.
#pragma once

#include <hip/hip_runtime.h>

#include "bq_device.h"
#include "bq_kv.h"

namespace bq {
namespace {

constexpr int kThreads = 256;  // of a workgroup of these kernels

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// n / d for n < 2^31 by one multiplication: mul = ceil(2^(31+l) / d), l = ceil(log2 d), d >= 2.
struct Divider {
  uint32_t mul, shift;
};

inline Divider make_divider(uint32_t d) {
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

// Where a unit lives: its token, its offset in the token's row and in its head (elements) and its flat
// element in the pool (-1: no such slot).
struct Place {
  uint32_t token, col, d;
  int64_t flat;
};

__device__ __forceinline__ Place place(uint32_t u, const KvShape& sh) {
  Place p;
  p.token = divide(u, sh.by_row);
  const uint32_t c = u - p.token * sh.row_units;
  p.col = c * 8;
  const uint32_t head = divide(c, sh.by_head);
  p.d = (c - head * sh.head_units) * 8;
  const int64_t slot = sh.slot[p.token];
  const int64_t page = slot >> sh.log2_page;
  const int64_t in_page = slot & ((1 << sh.log2_page) - 1);
  const int64_t row = ((page * sh.kv_heads + head) << sh.log2_page) + in_page;
  p.flat = slot >= 0 && slot < sh.slots ? row * (int64_t)(sh.head_units * 8) + p.d : -1;
  return p;
}

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

// Quantizes the 8 elements x(0) .. x(7) of the unit at `flat` of a side's pool (below 0: its lanes take part only).  The
// lanes of a block, `1 << (log2b - 3)`, call this together.
template <int KB, int MODE, int M, typename X>
__device__ __forceinline__ void quantize_unit(X x, int64_t flat, int log2b, const QuantArgs& qa,
                                              const typename Entry<M>::type* s_lut, const float* s_thr, uint8_t* packed,
                                              float* absmax, int tid) {
  // Block maximum over finite elements, as the bits of |x| (ordered like the values).
  const int lanes = 1 << (log2b - 3);  // lanes of a block
  uint32_t m = 0;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = f32_bits(x(e)) & 0x7fffffffu;
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
      nearest_pair<MODE, M>(x(e) * r, x(e + 1) * r, qa, s_lut, s_thr, q[e], q[e + 1]);
  } else {
    // a non-finite element and every element of a zero block take y = 0, whose code is z
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = x(e);
      const float y = (v * s) * r;
      q[e] = nearest_code<MODE, M>(a > 0.0f && fabsf(v) <= 0x1.fffffep127f ? y : 0.0f, qa, s_lut, s_thr);
    }
  }
  if (flat >= 0) {
    if constexpr (KB == 4) {
      *reinterpret_cast<uint32_t*>(packed + (flat >> 1)) = pack_word<4>(q);
    } else {
      const u32x2 w = {pack_word<8>(q), pack_word<8>(q + 4)};
      *reinterpret_cast<u32x2*>(packed + flat) = w;
    }
    if ((tid & (lanes - 1)) == 0) absmax[flat >> log2b] = a;
  }
}

inline KvShape make_shape(const KvCacheArgs& c, int64_t tokens, const int64_t* slots) {
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

}  // namespace
}  // namespace bq
