// bq_attn.h -- device helpers shared by the attention kernels (k_attn.hip, k_attn_chunk.hip, k_attn_merge.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "bq_kv.h"

namespace bq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 2^x and log2 x by the hardware instructions (about one unit in the last place; results below the
// normal range are zero).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }

// A sum of weights relative to the reference `from`, relative to the larger one `to`.  In units of one reference the
// weights of zero values may be 2^99 and those of the largest values 2^-101: the sums stay in range where
// 2^(from - to), below 2^-126, does not, so it is taken in two halves.  No reference yet: the sum is zero, or
// NaN from q.
__device__ __forceinline__ float lower(float sum, float from, float to) {
  const float h = exp2_hw(0.5f * (from - to));
  return from == -INFINITY ? sum : (sum * h) * h;
}

// Maximum and sum over the four 16-lane rows of a wave (lanes l, l ^ 16, l ^ 32, l ^ 48), in every lane.
__device__ __forceinline__ float rows_max(float v) {
  u32x2 s = __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false);
  v = fmaxf(bits_f32(s.x), bits_f32(s.y));
  s = __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false);
  return fmaxf(bits_f32(s.x), bits_f32(s.y));
}

__device__ __forceinline__ float rows_sum(float v) {
  u32x2 s = __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false);
  v = bits_f32(s.x) + bits_f32(s.y);
  s = __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false);
  return bits_f32(s.x) + bits_f32(s.y);
}

// Larger of three in one instruction (fmaxf of values that may be signalling NaNs, as the compiler has to take
// a product's, adds an instruction for each).
__device__ __forceinline__ float max3_hw(float a, float b, float c) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}

// Weights may grow by 2^kSlack over the running reference of a row before its sums are rescaled: binary16
// holds them up to 2^16, and with little slack the rows of a wave between them rescale in every other
// step (slack 2^6: 777 tokens over 6000 keys, head 256: 74 us, 2^12: 65).
constexpr float kSlack = 12.0f;

// Cached values enter the matrix cores multiplied by a power of two that puts the largest just below
// 2^kTopBit, so that binary16 (down to 2^-14 in full precision) keeps 11 bits of small ones too.
constexpr int kTopBit = 14;

// Two binary32 values as a pair of 16-bit ones (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  return bf16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

// A sequence's rows and keys, clamped to what the call allows.
struct Sequence {
  int q0, nq;  // first row of q, new tokens
  int kv;      // keys
};

// An entry of q_start as a row that q and out have, or their end (the difference of two is then in range too).
__device__ __forceinline__ int row_number(const KvAttendArgs& aa, int row) {
  return max((int)min((int64_t)row, aa.tokens), 0);
}

__device__ __forceinline__ Sequence sequence(const KvAttendArgs& aa, int seq) {
  Sequence s;
  s.q0 = row_number(aa, __builtin_amdgcn_readfirstlane(aa.q_start[seq]));
  // positions count all new tokens; rows past max_q_len are left out by the grid
  s.nq = max(row_number(aa, __builtin_amdgcn_readfirstlane(aa.q_start[seq + 1])) - s.q0, 0);
  s.kv = max(min(__builtin_amdgcn_readfirstlane(aa.kv_len[seq]), aa.max_kv_len), 0);
  return s;
}

// Keys [lo, hi) that the new token i of the sequence sees.
__device__ __forceinline__ int first_key(const KvAttendArgs& aa, const Sequence& s, int i) {
  const int pos = s.kv - s.nq + i;
  return aa.window > 0 && pos >= aa.window ? pos - aa.window + 1 : 0;
}

__device__ __forceinline__ int end_key(const KvAttendArgs& aa, const Sequence& s, int i) {
  return aa.causal ? max(min(s.kv, s.kv - s.nq + i + 1), 0) : s.kv;
}

// Partial results of a row over one split of its keys, relative to the reference exponent m:
// sum of weights l and the weighted sum of values (head_dim binary32), kept in the workspace.  l is the
// sum that belongs to the weighted one, of weights as they were rounded; `exact`, for lse, that of the
// unrounded ones.
struct Partial {
  float m, l, exact;
};

constexpr int kMaxSplits = 64;

// Which sequences a launch takes.  A call whose sequences may bring many rows to a key/value head goes
// through two sets of kernels: those of k_attn_chunk.hip for sequences with more than kFewRows rows (any, if
// it is the only one), and the splitting kernel of k_attn.hip for the others.  Its grid has room for kFewRows rows of
// every sequence, so more of them cost calls in which most bring one (48 single tokens beside 200 of one
// prompt, 32 heads over 8 of 128: 139 us, 180 with 64 rows, 265 with 128) and gain little elsewhere (the ragged
// batch of 9: 69, 71, 73).
enum Rows : int { kAllRows = 0, kFewOnly = 1, kManyRows = 2 };
constexpr int kFewRows = 32;

__device__ __forceinline__ bool many_rows(int nq, int group, int num_seqs) {
  return num_seqs == 1 || (int64_t)nq * group > kFewRows;
}

__device__ __forceinline__ bool takes(int rows, int nq, int group, int num_seqs) {
  return rows == kAllRows || many_rows(nq, group, num_seqs) == (rows == kManyRows);
}

// Natural logarithm of l 2^m: the integer part of log2 l joins m before the sum is rounded.
__device__ __forceinline__ float log_sum(float m, float l) {
  if (!(l > 0.0f)) return l == 0.0f ? -INFINITY : l;
  const int e = __builtin_amdgcn_frexp_expf(l);
  return ((m + (float)e) + log2_hw(__builtin_amdgcn_frexp_mantf(l))) * 0.693147180559945309f;
}

}  // namespace bq
