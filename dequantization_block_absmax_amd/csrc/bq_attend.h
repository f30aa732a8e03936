// bq_attend.h -- the kernel of attention of new tokens over a paged key/value cache held in blockwise codes.
//
//   o_i = sum_j p_ij v_j,   p_ij = exp(s_ij) / sum_j exp(s_ij),   s_ij = scale * (q_i . k_j)
// over the keys j that row i sees; k and v are the cached values c[code] * a, one pass over the keys
// with the running maximum and sum of the softmax.
//
// Factored form.  The matrix cores (v_mfma_f32_16x16x32_f16) multiply the codes' table entries,
// times 2^14 (binary16 then keeps 11 bits of every entry down to its least, 2^-20) and rounded once to
// binary16; the block maxima enter in binary32:
//   s_ij = R_i sum_b a_jb (sum_{d in b} q'_id c_jd)   q' = q 2^-e_i exact in binary16, R_i = scale 2^e_i
//   o_i  = sum_j (p_ij a'_jb) c'_jd                    for d in block b of the values
// so no cached value is formed: a code byte indexes a table in LDS that holds its two binary16
// entries side by side.  Rounded to 16 bits are: c (2^-11 relative at most), the weights p a' (2^-11, and 2^-25 of the
// largest of their row), q' where it falls 2^-14 below its row's largest element, and the result.  With q
// in binary16, whose result keeps three more bits than a bfloat16's, c enters in two parts and the weights, where registers
// allow, too (Operand, Occupancy): the error is the result's own rounding, or sqrt(2) times that.  e_i is the
// exponent of the row's largest |q|.  Weights are kept in range by the reference
//   M_i = max_j (log2-domain s_ij + E_j),   E_j the exponent of token j's largest value maximum,
// in place of the plain running maximum: the weights p a' = 2^(s - M) a' then stay below 2^14 whatever
// the size of the values, and sum and weighted sum carry the same factor, which cancels.
//
// Decomposition.  Work is split over (16 RT rows: new token x query head of one key/value head) x
// (key/value head) x (sequence) x (splits of the keys).  A workgroup's eight waves (four for 256-wide heads in
// blocks of 32, whose block maxima fill the registers) take groups of 32 keys in turn, each on its own, and
// join their sums through LDS at the end; with more than one split
// the partial sums go to the workspace and k_attn_merge.hip joins them.  For one group of 32 keys, with
// lane l = 16 g + m:
//   scores  S^T = K Q^T: A = K, lane (m, g) decodes 8 codes of key m per step of 32 d; the result's lane
//           holds, for row m, the keys 4g .. 4g+3 of each 16.
//   sums    O^T = V^T P^T: B = P^T takes exactly those keys from the same lane (the order of the 32 keys
//           in the product is free), and A = V^T the lane's d's for the same 8 keys: its codes are a
//           few consecutive bytes of each key's row, so nothing crosses lanes on the way and
//           neither operand passes through LDS.
// With several blocks to a head (NB > 1) an A tile must hold d's of one block only; lanes exchange
// halves of their bytes (spread) so that each holds some d's of every block.
//
// What bounds it.  For single tokens and drafts the bytes of codes and maxima; beside them the lookups (a permute and an
// LDS read per code byte and use) and the exchange keep the vector units and LDS about as busy, so that the
// kernels take 1.1 to 1.3 times what loads alone take with the same schedule (timed with the buffers in the last-level
// cache: 71 of 91 us, 31 of 39, 23.5 of 26.2 for the first three).  On MI355X, median of a call's kernels, buffers in turn
// past that cache:
//   64 sequences of up to 8192 keys, 32 heads over 8 of 128, 4-bit, B = 64, bf16: 94 us, 4.0 TB/s
//   3 of up to 131072 keys, 16 over 2 of 128, 8-bit, B = 128, f16: 44.5 us + join 4.7, 4.1 TB/s
//   24 x 6 tokens, window 4000, 20 over 5 of 64, 8-bit, B = 32, f16: 32.3 us + join 4.7, 1.8 TB/s: a wave has one group of
//   keys in flight and about eight in all
//   1 of 1000 keys, 32 over 8 of 128, 4-bit, B = 64, bf16: 8.3 us + join 3.5: the chain of loads from the arguments to
//   the sequence, its pages and its keys, each about 1 us, and two launches
// Eight waves of a workgroup share one table in LDS (four: 114 us in the first case, 43 in the second; sixteen: 98
// and 43).  Workgroups that each take an equal share of all keys, whatever the sequence, gained nothing (84 us
// against 83, and a longer join) over the splits below.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "bq_attn.h"
#include "bq_kv.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kGroup = 32;        // keys per wave and step
constexpr int kEntryBytes = 256;  // of the LDS table: copies for 64 lanes (32 where an entry takes 8 bytes), side
                                  // by side over the banks: no lookup waits for another

template <int D, int NB, int KB>
struct Shape {
  static constexpr int kB = D / NB;             // block size
  static constexpr int kRow = D * KB / 8;       // bytes of a key's codes
  static constexpr int kLane = kRow / 16;       // bytes of a value's codes per lane: 2, 4, 8 or 16
  static constexpr int kWords = kLane < 4 ? 1 : kLane / 4;
  static constexpr int kSteps = D / 32;         // products of 32 d
  static constexpr int kStepWords = KB / 4;     // words of a key's codes per lane and step: 1 or 2
  static constexpr int kTiles = D / 16;         // tiles of 16 d of the result
  static constexpr int kPerLane = D / 16;       // d's per lane
  static constexpr int kPerBlock = kPerLane / NB;
  static constexpr int kMaxima = NB > 2 ? NB / 2 : 1;  // block maxima of a group that a lane loads
};

// What a lane holds of one group of 32 keys: of the keys and of the values.  The group's 32 NB block
// maxima are spread over the wave, in order, and go through LDS when they are used (held where they
// are used they would take 16 NB registers).
template <int D, int NB, int KB>
struct Keys {
  using S = Shape<D, NB, KB>;
  uint32_t code[2][S::kSteps * S::kStepWords];
  float a[S::kMaxima];
};

template <int D, int NB, int KB>
struct Values {
  using S = Shape<D, NB, KB>;
  uint32_t code[8][S::kWords];
  float a[S::kMaxima];
};

// Where the pages of a group of 32 keys lie; a page outside the pool reads page 0 and hides its keys.
struct Pages {
  int id[2];
};

typedef const __attribute__((address_space(1))) uint8_t* Global;

// Keeps a uniform address in scalar registers, apart from the lane's offset: loads then take a scalar
// base and a 32-bit offset (the compiler would else keep base plus offset of every array in vector
// registers through the loop).
__device__ __forceinline__ Global scalar_base(const void* p) {
  uint64_t a = (uint64_t)(uintptr_t)p;
  asm("" : "+s"(a));
  return (Global)(uintptr_t)a;
}

// The N words at src (N = 1, 2, 4 or 8, aligned to min(N, 4) words).
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, Global src) {
  if constexpr (N == 1) {
    w[0] = *(const __attribute__((address_space(1))) uint32_t*)src;
  } else if constexpr (N == 2) {
    const u32x2 t = *(const __attribute__((address_space(1))) u32x2*)src;
    w[0] = t.x;
    w[1] = t.y;
  } else {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const u32x4 t = *(const __attribute__((address_space(1))) u32x4*)(src + 16 * k);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * k + e] = t[e];
    }
  }
}

// LDS offset of the lane's copy of the entry for byte b of w: byte << 8 | copy, one permute (copy: the
// lane's offset in a row of copies).
__device__ __forceinline__ uint32_t entry_of(uint32_t w, int b, uint32_t copy) {
  return __builtin_amdgcn_perm(w, copy, 0x0c0c0000u | (uint32_t)(4 + b) << 8);
}

// How a table entry enters the products.  One part (q in bfloat16): its binary16 rounding, 2^-11 relative, far
// below what the result's rounding leaves.  Two parts (q in binary16): the rounding and, beside it, the
// rounded rest, 2^-22 relative together; the other operand repeats, and the sum over k adds both.
//   entries in LDS, by byte: 4-bit codes the pair (low nibble, high nibble), then the rests' pair; 8-bit codes
//   one entry, then its rest
template <int KB, bool HL>
struct Operand {
  static constexpr int kParts = HL ? 2 : 1;          // products for 8 consecutive operands
  static constexpr int kLookups = KB == 4 ? 4 : 8;   // bytes that hold their codes
  static constexpr int kCopyBytes = HL && KB == 4 ? 8 : 4;

  // The 8 entries of the codes at bytes by[] of wd[].
  static __device__ __forceinline__ void look_up(const char* lut, uint32_t copy, const uint32_t (&wd)[kLookups],
                                                 const int (&by)[kLookups], f16x8 (&a)[kParts]) {
    u32x4 x[kParts];
#pragma unroll
    for (int i = 0; i < kLookups; ++i) {
      const char* at = lut + entry_of(wd[i], by[i], copy);
      if constexpr (KB == 4 && HL) {
        const u32x2 e = *reinterpret_cast<const u32x2*>(at);
        x[i / 2][2 * (i & 1)] = e.x;
        x[i / 2][2 * (i & 1) + 1] = e.y;
      } else if constexpr (KB == 4) {
        x[0][i] = *reinterpret_cast<const uint32_t*>(at);
      } else if constexpr (HL) {
        x[i / 4][i & 3] = *reinterpret_cast<const uint32_t*>(at);
      } else if ((i & 1) == 0) {
        const f16x2 pair = {*reinterpret_cast<const _Float16*>(at),
                            *reinterpret_cast<const _Float16*>(lut + entry_of(wd[i + 1], by[i + 1], copy))};
        x[0][i / 2] = __builtin_bit_cast(uint32_t, pair);
      }
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) a[k] = __builtin_bit_cast(f16x8, x[k]);
  }

  // The other operand, from pairs of its 8 values.  `repeat` sets each beside an entry and beside the entry's rest;
  // `beside` beside the entry only.
  static __device__ __forceinline__ void repeat(const u32x4& pairs, f16x8 (&b)[kParts]) {
    if constexpr (!HL) {
      b[0] = __builtin_bit_cast(f16x8, pairs);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t p0 = pairs[2 * k], p1 = pairs[2 * k + 1];
        u32x4 x;
        if constexpr (KB == 4) x = (u32x4){p0, p0, p1, p1};
        else
          x = (u32x4){__builtin_amdgcn_perm(p0, p0, 0x01000100u), __builtin_amdgcn_perm(p0, p0, 0x03020302u),
                      __builtin_amdgcn_perm(p1, p1, 0x01000100u), __builtin_amdgcn_perm(p1, p1, 0x03020302u)};
        b[k] = __builtin_bit_cast(f16x8, x);
      }
    }
  }
  static __device__ __forceinline__ void beside(const u32x4& pairs, f16x8 (&b)[kParts]) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const uint32_t p0 = pairs[(2 * k) & 3], p1 = pairs[(2 * k + 1) & 3];
      u32x4 x;
      if constexpr (KB == 4) x = (u32x4){p0, 0u, p1, 0u};
      else x = (u32x4){p0 & 0xffffu, p0 >> 16, p1 & 0xffffu, p1 >> 16};
      b[k] = __builtin_bit_cast(f16x8, x);
    }
  }
};

// Exchange between lanes m and p of a row of 16: of the lane's bytes in w (two halves), the lane with
// `upper` false keeps its first half and takes the partner's first half as its second; the other
// takes the partner's second half as its first and keeps its own second.
constexpr int kXor8 = 0x128;    // row rotate by 8: lane m ^ 8
constexpr int kXor2 = 0x4E;     // quad permute [2, 3, 0, 1]: lane m ^ 2
constexpr int kXor4 = -4;       // rotate by 12 for the even quads (from m + 4), by 4 for the odd ones (from m - 4)

template <int DPP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (DPP == kXor4) {
    const int even = __builtin_amdgcn_update_dpp(0, (int)v, 0x12C, 0xF, 0x5, false);
    return (uint32_t)__builtin_amdgcn_update_dpp(even, (int)v, 0x124, 0xF, 0xA, false);
  } else {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, DPP, 0xF, 0xF, false);
  }
}

template <int DPP>
__device__ __forceinline__ void exchange_words(uint32_t& a, uint32_t& b, bool upper) {
  const uint32_t got = partner<DPP>(upper ? a : b);
  a = upper ? got : a;
  b = upper ? b : got;
}

// Halves of 16 bits in one word (sel: per-lane byte selectors), or of 8 bits in each 16.
template <int DPP>
__device__ __forceinline__ uint32_t exchange_bytes(uint32_t w, uint32_t sel) {
  return __builtin_amdgcn_perm(partner<DPP>(w), w, sel);
}

// Spreads a lane's kPerLane consecutive d's (bytes w of each key) over the blocks: afterwards block b's
// kPerBlock d's of the lane stand at bytes [b, b + 1) * kLane / NB.
template <int D, int NB, int KB>
struct Spread {
  using S = Shape<D, NB, KB>;
  bool up[3];
  uint32_t sel16[3], sel8[3];  // selectors for halves of 16 bits, and of 8 bits in both halves of a word

  __device__ __forceinline__ explicit Spread(int m) {
    up[0] = m & 8;
    up[1] = m & 4;
    up[2] = m & 2;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      sel16[i] = up[i] ? 0x03020706u : 0x05040100u;
      sel8[i] = up[i] ? 0x03070105u : 0x06020400u;
    }
  }

  // One halving of pieces of `bytes` bytes (a piece: what the lane holds of one group of blocks).
  template <int STAGE, int BYTES>
  __device__ __forceinline__ void halve(uint32_t* w) const {
    constexpr int dpp = STAGE == 0 ? kXor8 : STAGE == 1 ? kXor4 : kXor2;
    if constexpr (BYTES >= 8) {
      constexpr int n = BYTES / 4;
#pragma unroll
      for (int p = 0; p < S::kWords; p += n)
#pragma unroll
        for (int i = 0; i < n / 2; ++i) exchange_words<dpp>(w[p + i], w[p + n / 2 + i], up[STAGE]);
    } else if constexpr (BYTES == 4) {
#pragma unroll
      for (int i = 0; i < S::kWords; ++i) w[i] = exchange_bytes<dpp>(w[i], sel16[STAGE]);
    } else {
#pragma unroll
      for (int i = 0; i < S::kWords; ++i) w[i] = exchange_bytes<dpp>(w[i], sel8[STAGE]);
    }
  }

  __device__ __forceinline__ void apply(uint32_t* w) const {
    if constexpr (NB >= 2) halve<0, S::kLane>(w);
    if constexpr (NB >= 4) halve<1, S::kLane / 2>(w);
    if constexpr (NB >= 8) halve<2, S::kLane / 4>(w);
  }

  // The d at place e of block b in lane m after apply().
  static __device__ __forceinline__ int d_of(int m, int b, int e) {
    // back through the stages: which half of the piece it was, and whose
    int half = 0, weight = 1;
    if constexpr (NB >= 8) {
      half += weight * ((m >> 1) & 1);
      m = (m & ~2) | ((b & 1) << 1);
      b >>= 1;
      weight *= 2;
    }
    if constexpr (NB >= 4) {
      half += weight * ((m >> 2) & 1);
      m = (m & ~4) | ((b & 1) << 2);
      b >>= 1;
      weight *= 2;
    }
    if constexpr (NB >= 2) {
      half += weight * ((m >> 3) & 1);
      m = (m & ~8) | ((b & 1) << 3);
    }
    return m * S::kPerLane + half * S::kPerBlock + e;
  }
};

// Keeps loads where they are written, before and after.
__device__ __forceinline__ void load_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Waves per workgroup and per SIMD.  Four per SIMD, two workgroups to a CU, where 128 registers hold a form; else one
// workgroup: among the forms at the limit 64 wide with 32 rows and two blocks (24 x 6 tokens, 8-bit, windows of 4000, buffers
// in turn: 38.1 us at four with 12 to 15 registers spilled, 35.9 at two with the weights' rests besides; bf16
// 33.5 and 29.4) and 128 wide in 8 bits with two blocks (64 single tokens over up to 4096 keys, bf16: 100 us with 7
// spilled, 90).  Of the others <128, 4, 8, 2> and <64, 1, 8, 2> with q in binary16 spill one register.  What a
// tree adds costs more: with q in binary16 <64, 1, 8, 2> spills 18, <64, 1, 4, 2> 14, <128, 4, 8, 2> 7 (in bfloat16 6), <64, 2, 4, 4> 6
// and <128, 1, 8, 1> 4.
constexpr bool wide_form(int head_dim, int nb, int bits, int rt) {
  return nb == 2 && rt * head_dim == 128 && (head_dim == 64 || bits == 8);
}

template <int D, int NB, int KB, int RT>
struct Occupancy {
  static constexpr int kWaves = D == 256 && NB == 8 ? 4 : 8;
  static constexpr int kPerSimd = D == 256 && NB == 8 ? 1 : RT * D <= 128 && NB <= 2 && !wide_form(D, NB, KB, RT) ? 4 : 2;
  // room for the weights' rests too (q in binary16; without them the weights are rounded once, 2^-11)
  static constexpr bool kRests = kPerSimd == 4 ? RT * NB * D <= 128 : kPerSimd == 2 && (NB <= 2 || RT * D == 128);
};

// What a tree of new tokens adds in LDS: the parents (as numbers of new tokens; -1: follows the context, -2: sees nothing),
// and as words of 32 new tokens, a word of zeros before and behind them, which of them are seen at all and which each
// token of the tile sees.
constexpr int kTreeWords = kMostNodes / 32 + 2;

template <int ROWS>
struct TreeShared {
  int16_t parent[kMostNodes];
  uint32_t used[kTreeWords];
  uint32_t seen[ROWS][kTreeWords];
  int depth[ROWS];  // or -1: sees nothing
};
struct NoTree {};

// Fills the shared tree of a tile with the new tokens i_first .. i_last; `parent` is token tid's.  The last 256 threads, each
// with a token of its own, follow its path to the root, a load from LDS for each ancestor: drafts level by level are a few deep, a chain of
// 256 tokens takes some 20 us more in each workgroup (one over 1024 keys 41 us, a shallow tree of as many 19).  Every thread
// takes part; a barrier has to follow.
template <int THREADS, int ROWS>
__device__ __forceinline__ void read_tree(const KvAttendArgs& aa, TreeShared<ROWS>& tree, int parent, int tid, int i_first,
                                          int i_last) {
  if (tid < kMostNodes) tree.parent[tid] = (int16_t)(parent >= -1 && parent < tid ? parent : -2);
  if (tid < kTreeWords) tree.used[tid] = 0;
  __syncthreads();
  const int node = tid - (THREADS - kMostNodes);  // whole waves
  if (node < 0) return;
  const bool mine = node >= i_first && node <= i_last;
  uint32_t* const seen = tree.seen[mine ? node - i_first : 0];
  int at = node, depth = 0, word = node >> 5;
  uint32_t bits = 0;
  if (mine)
    for (int k = 0; k < kTreeWords; ++k) seen[k] = 0;
  if (node <= i_last)
    for (int n = 0; n < kMostNodes; ++n) {  // ancestors come in descending order: a word is done when another begins
      if (at >> 5 != word) {
        if (mine) seen[word + 1] = bits;
        word = at >> 5;
        bits = 0;
      }
      if (aa.window == 0 || depth < aa.window) bits |= 1u << (at & 31);
      at = tree.parent[at];
      if (at < 0) break;
      ++depth;
    }
  const bool sees = node <= i_last && at == -1;
  if (mine) {
    seen[word + 1] = bits;
    tree.depth[node - i_first] = sees ? depth : -1;
    if (!sees)
      for (int k = 0; k < kTreeWords; ++k) seen[k] = 0;
  }
  const uint64_t all = __ballot(sees);
  if ((node & 31) == 0) tree.used[(node >> 5) + 1] = (uint32_t)(all >> (node & 63));
}

// Whether any of these tokens sees anything (the same in every lane).
template <int ROWS>
__device__ __forceinline__ bool any_node(const TreeShared<ROWS>& tree, int i_first, int i_last) {
  uint32_t any = 0;  // tokens past i_last are not marked
  for (int k = i_first >> 5; k <= i_last >> 5; ++k) any |= tree.used[k + 1] & (k == i_first >> 5 ? ~0u << (i_first & 31) : ~0u);
  return __builtin_amdgcn_readfirstlane(any) != 0;
}

// Which part of a call a workgroup takes: of one sequence and key/value head a block of rows and one of n_splits runs of `per` units of
// keys.
struct Part {
  int seq, kvh, block, split, per, n_splits;
};

__device__ __forceinline__ int from_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Divides sequences of different lengths into parts of ROWS rows by a number of units of UNIT keys, from the ALIGN-th key that they
// begin at.  Every part is as long as leaves each of `workgroups`, which the device holds at once, one, or half of that where
// less then stands idle: a part costs its units and about `extra` more.  What is left over of each sequence is a part too.
// With the kernel of k_tree.hip 24 sequences of 32 drafted tokens and up to 8192 keys took 152 us in halves and 173 in wholes, two
// of 48 and up to 131072 keys 196 and 185.  Parts are numbered in a row, since workgroups without one between the others would
// leave compute units without work: the hardware deals them out in turn.  The lengths are known on the device only, so every
// workgroup works this out, a lane to a sequence.  False: there is no such part.
template <int ROWS, int UNIT, int ALIGN>
__device__ __forceinline__ bool find_part(const KvAttendArgs& aa, int group, int nsplit, int workgroups, int least, int extra, Part& part) {
  const int lane = threadIdx.x & 63;
  int blocks = 0, units = 0;  // of the lane's sequence; of all heads
  auto load = [&](int s) {
    blocks = units = 0;
    if (s >= aa.num_seqs) return;
    const int q0 = row_number(aa, aa.q_start[s]), nq = max(row_number(aa, aa.q_start[s + 1]) - q0, 0);
    const int kv = max(min(aa.kv_len[s], aa.max_kv_len), 0);
    blocks = (int)((min(nq, aa.max_q_len) * (int64_t)group + ROWS - 1) / ROWS) * aa.cache.kv_heads;
    units = max((int)((kv - (node_first(aa, kv - nq, 0) & ~(ALIGN - 1)) + (int64_t)UNIT - 1) / UNIT), 0);
  };
  const int rounds = (aa.num_seqs + 63) / 64, lanes = min(aa.num_seqs, 64);
  int64_t work = 0;
  for (int i = 0; i < rounds; ++i) {
    load(64 * i + lane);
    work += (int64_t)blocks * units;
  }
  for (int x = 1; x < lanes; x <<= 1) work += __shfl_xor(work, x);
  work = (int64_t)(uint32_t)from_lane((int)work, 0) | (int64_t)from_lane((int)(work >> 32), 0) << 32;
  const int of_whole = max((int)((work + workgroups - 1) / workgroups), least);
  const int of_half = max((int)((work + 2 * workgroups - 1) / (2 * workgroups)), least);
  int per = of_whole;
  if (rounds == 1) {
    // lanes 0 .. 31 look for the length of a whole, the others for that of a half
    const int goal = lane < 32 ? workgroups : 2 * workgroups, from = lane < 32 ? of_whole : of_half;
    const int mine = from + (from * (lane & 31) + 15) / 16;
    const float inv = 1.0f / (float)mine;
    int n = 0;
    for (int s = 0; s < aa.num_seqs; ++s)
      n += from_lane(blocks, s) * max((int)ceilf((float)from_lane(units, s) * inv), 1);
    const uint64_t fits = __ballot(n <= goal) | 1ull << 31 | 1ull << 63;
    const int whole = from_lane(mine, __builtin_ctzll(fits)), half = from_lane(mine, 32 + __builtin_ctzll(fits >> 32));
    per = 2 * (half + extra) < whole + extra ? half : whole;
  }
  auto per_of = [&]() { return max(per, (units + nsplit - 1) / nsplit); };
  auto splits_of = [&]() { return max((units + per_of() - 1) / per_of(), 1); };
  auto up_to = [&]() {  // parts of this lane's sequence and those before it
    int n = blocks * splits_of();
    for (int x = 1; x < lanes; x <<= 1) {
      const int before = __shfl_up(n, x);
      n += lane >= x ? before : 0;
    }
    return n;
  };
  int at = blockIdx.x;
  for (int i = 0; i < rounds; ++i) {
    if (rounds > 1) load(64 * i + lane);
    const int n = up_to(), all = from_lane(n, lanes - 1);
    if (at < all) {
      const int who = __builtin_ctzll(__ballot(at < n));
      const int mine = from_lane(blocks, who);
      part.seq = 64 * i + who;
      part.per = from_lane(per_of(), who);
      part.n_splits = from_lane(splits_of(), who);
      at -= from_lane(n, who) - mine * part.n_splits;
      part.split = at / mine;
      at -= part.split * mine;
      part.kvh = at % aa.cache.kv_heads;
      part.block = at / aa.cache.kv_heads;
      return true;
    }
    at -= all;
  }
  return false;
}

// Splits of row r that no part takes: the join passes over them.
template <int D>
__device__ __forceinline__ void no_parts(const KvAttendArgs& aa, const Part& part, const Sequence& sq, int nrows, int nsplit, int r,
                                         float* partial) {
  if (r >= nrows) return;
  const int group = aa.heads / aa.cache.kv_heads;
  const int64_t row = (int64_t)(sq.q0 + r / group) * aa.heads + part.kvh * group + r % group;
  for (int x = part.n_splits; x < nsplit; ++x)
    reinterpret_cast<Partial*>(partial + aa.tokens * aa.heads * nsplit * D)[row * nsplit + x] = {-INFINITY, 0.0f, 0.0f};
}

// TREE: the new tokens are a tree (aa.parents).  Token i sees the context (the keys before the new tokens), itself and
// the tokens on its path from the root, by its depth within the window.  The words are worked out once for a tile, beside
// the first loads, each token's path by a lane of its own; they are looked at for the groups that reach past the
// context only.  `rows`: what takes() goes by or, of a tree, the workgroups that the device holds at once where the
// parts are found from the lengths (find_part), and else 0.
template <int D, int NB, int KB, int RT, bool HL, bool TREE>
__global__ __launch_bounds__((64 * Occupancy<D, NB, KB, RT>::kWaves), (Occupancy<D, NB, KB, RT>::kPerSimd)) void attend_kernel(
    KvAttendArgs aa, DequantArgs da, int nsplit, float* partial, int rows) {
  using O = Operand<KB, HL>;
  constexpr bool bf16 = !HL;  // the type of q and out
  constexpr int W = Occupancy<D, NB, KB, RT>::kWaves;
  using S = Shape<D, NB, KB>;
  constexpr int kThreads = 64 * W;
  constexpr int kRows = 16 * RT;
  constexpr int kPitch = D + 4;  // of a row of partial sums in LDS
  constexpr int kLut = 256 * kEntryBytes;
  constexpr int kQueries = RT * S::kSteps * O::kParts * 64 * 16;  // in the order the lanes read them
  constexpr int kMaxima = 32 * NB * 4;                   // one side of a wave's group
  constexpr int kLoop = kLut + kQueries + 2 * W * kMaxima, kSums = W * 16 * kPitch * 4;
  // table, queries and block maxima; after the keys, the waves' sums
  __shared__ __attribute__((aligned(16))) char s_mem[kLoop > kSums ? kLoop : kSums];
  __shared__ Partial s_part[W][kRows];
  __shared__ std::conditional_t<TREE, TreeShared<kRows>, NoTree> s_tree;
  __shared__ float s_scale[kRows];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  // The table's entries are asked for first: they come with the arguments, beside the chain of loads from the
  // sequence to its pages to its keys.
  float entry_lo = 0.0f, entry_hi = 0.0f;
  if (tid < 256) {
    entry_lo = da.c[KB == 4 ? tid & 15 : tid];
    entry_hi = da.c[KB == 4 ? tid >> 4 : tid];
  }
  load_fence();
  const int group = aa.heads / aa.cache.kv_heads;
  Part part = {(int)blockIdx.z, (int)blockIdx.y, (int)blockIdx.x / nsplit, (int)blockIdx.x % nsplit, 0, nsplit};
  if constexpr (TREE) {
    constexpr int kPartUnits = 3;  // that a part costs besides its own
    if (rows != 0 && !find_part<kRows, kGroup * W, kGroup>(aa, group, nsplit, rows, 1, kPartUnits, part)) return;
  }
  const int split = part.split, tile = part.block, kvh = part.kvh, seq = part.seq;
  const Sequence sq = sequence(aa, seq);
  const int nrows = min(sq.nq, aa.max_q_len) * group;  // rows of the sequence for this key/value head
  if (tile * kRows >= nrows || (!TREE && !takes(rows, min(sq.nq, aa.max_q_len), group, aa.num_seqs))) return;
  if constexpr (TREE) {
    if (split == 0 && tid < kRows) no_parts<D>(aa, part, sq, nrows, nsplit, tile * kRows + tid, partial);
  }

  // Keys of the tile's rows together, this split's groups of 32 of them, and this wave's: groups
  // wave, wave + W, ... of the split.
  const int last_row = min(tile * kRows + kRows, nrows) - 1;
  const int i_first = tile * kRows / group, i_last = last_row / group;
  const int context = sq.kv - sq.nq;
  // of a tree, whose depths are not known yet, from the least depth there is to the greatest there could be
  const int first = TREE ? node_first(aa, context, 0) : first_key(aa, sq, i_first), begin = first & ~(kGroup - 1);
  int end = TREE ? max(min(sq.kv, context + i_last + 1), 0) : end_key(aa, sq, i_last);
  const int lo_all = TREE ? node_first(aa, context, i_last) : first_key(aa, sq, i_last);  // seen by every row
  int hi_all = TREE ? context : end_key(aa, sq, i_first);
  const int groups = end > begin ? (end - begin + kGroup - 1) / kGroup : 0;
  const int per = TREE && rows != 0 ? part.per * W : (groups + nsplit - 1) / nsplit;
  const int g_end = min((split + 1) * per, groups);
  int gi = split * per + wave;

  const int lps = aa.cache.log2_page;
  // read through scalar loads: the numbers are the same for the whole wave, and waiting for them
  // does not wait for the cache's vector loads before them
  typedef const __attribute__((address_space(4))) int32_t* ScalarTable;
  const ScalarTable pages = (ScalarTable)(uintptr_t)(aa.page_table + (int64_t)seq * aa.table_stride);
  const int last_page = sq.kv > 0 ? (sq.kv - 1) >> lps : 0;
  auto find = [&](int i) {
    Pages p;
#pragma unroll
    for (int u = 0; u < 2; ++u) p.id[u] = pages[min((begin + i * kGroup + 16 * u) >> lps, last_page)];
    return p;
  };
  auto listed = [&](int id) { return (uint32_t)id < (uint32_t)aa.cache.num_pages; };
  auto row_of = [&](int i, const Pages& p, int u) {  // the pool's row (page, head, slot) of the half group
    const int j = begin + i * kGroup + 16 * u;
    return (((int64_t)(listed(p.id[u]) ? p.id[u] : 0) * aa.cache.kv_heads + kvh) << lps) + (j & ((1 << lps) - 1));
  };
  // The maxima of the group's first 16 keys, then of the others: lane l takes the l-th few.
  auto load_maxima = [&](int i, const Pages& p, int side, float* a) {
    constexpr int half = NB == 1 ? 16 : 32;  // lanes of 16 keys (NB = 1: the wave's upper half repeats the lower)
    const Global src0 = scalar_base(aa.cache.absmax[side] + row_of(i, p, 0) * NB);
    const Global src1 = scalar_base(aa.cache.absmax[side] + row_of(i, p, 1) * NB);
    load_words<S::kMaxima>(reinterpret_cast<uint32_t*>(a),
                           (lane & half ? src1 : src0) + (uint32_t)((lane & (half - 1)) * S::kMaxima * 4));
  };
  float* const s_maxima = reinterpret_cast<float*>(s_mem + kLut + kQueries) + wave * 2 * (kMaxima / 4);
  auto put_maxima = [&](int side, const float* a) {
    float* dst = s_maxima + side * (kMaxima / 4) + (NB == 1 ? lane & 31 : lane) * S::kMaxima;
#pragma unroll
    for (int k = 0; k < S::kMaxima; ++k) dst[k] = a[k];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  // of the lane's keys 4g .. 4g+3 of the half group u, block by block
  auto get_maxima = [&](int side, int u, float (&a)[4][NB]) {
    const float* src = s_maxima + side * (kMaxima / 4) + (16 * u + 4 * g) * NB;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(src + 4 * k);
#pragma unroll
      for (int e = 0; e < 4; ++e) a[(4 * k + e) / NB][(4 * k + e) % NB] = v[e];
    }
  };
  // A lane takes a quarter of each block's codes of key m: d = b * B + g * B / 4 + 0 .. B / 4 - 1.
  constexpr int kQuarter = S::kB / 4 * KB / 8;  // bytes
  auto load_keys = [&](int i, const Pages& p, Keys<D, NB, KB>& x) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(i, p, u);
      const Global src = scalar_base(aa.cache.packed[0] + row * S::kRow);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        load_words<kQuarter / 4>(&x.code[u][b * (kQuarter / 4)], src + (uint32_t)(m * S::kRow + g * kQuarter) + b * 4 * kQuarter);
    }
    load_maxima(i, p, 0, x.a);
  };
  // A lane takes bytes m * kLane .. of the codes of keys 4g .. 4g+3 of each 16.
  auto load_values = [&](int i, const Pages& p, Values<D, NB, KB>& x) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(i, p, u);
      const Global src = scalar_base(aa.cache.packed[1] + row * S::kRow) + (uint32_t)(4 * g * S::kRow + m * S::kLane);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (S::kLane == 2) x.code[4 * u + r][0] = *(const __attribute__((address_space(1))) uint16_t*)(src + r * S::kRow);
        else load_words<S::kWords>(x.code[4 * u + r], src + r * S::kRow);
      }
    }
    load_maxima(i, p, 1, x.a);
  };

  int parent = -2;  // of new token tid
  if constexpr (TREE) {
    if (tid <= i_last && tid < kMostNodes) parent = aa.parents[sq.q0 + tid];
    load_fence();
  }
  Keys<D, NB, KB> xk;
  Values<D, NB, KB> xv;
  Pages now = {{0, 0}}, next = {{0, 0}};
  if (gi < g_end) {  // the first group is on its way while the table and the queries are set up
    now = find(gi);
    next = find(min(gi + W, groups - 1));
    load_keys(gi, now, xk);
    load_values(gi, now, xv);
  }

  // Table (see Operand).
  if (tid < 256) {
    const float x0 = __builtin_ldexpf(entry_lo, kTopBit), x1 = __builtin_ldexpf(entry_hi, kTopBit);
    const float r0 = (float)(_Float16)x0, r1 = (float)(_Float16)x1;
    const uint32_t e = KB == 8 && HL ? pack_f16(x0, x0 - r0) : pack_f16(x0, x1);
    const uint32_t rest = KB == 4 && HL ? pack_f16(x0 - r0, x1 - r1) : e;
    const u32x4 e4 = {e, rest, e, rest};
#pragma unroll
    for (int i = 0; i < kEntryBytes / 16; ++i)  // in turn over the banks
      *reinterpret_cast<u32x4*>(s_mem + tid * kEntryBytes + ((i + tid) & (kEntryBytes / 16 - 1)) * 16) = e4;
  }
  const uint32_t copy = (lane * O::kCopyBytes) & (kEntryBytes - 1);
  if constexpr (TREE) read_tree<kThreads, kRows>(aa, s_tree, parent, tid, i_first, i_last);

  // Queries: wave t sets up the 16 rows of tile t, as the products' operands and a scale per row.
  f16x8* const s_q = reinterpret_cast<f16x8*>(s_mem + kLut);
  if (wave < RT) {
    const int r = tile * kRows + wave * 16 + m;
    const int i = r < nrows ? r / group : 0;
    const int head = kvh * group + (r < nrows ? r - i * group : 0);
    const char* src = static_cast<const char*>(aa.q) + ((int64_t)(sq.q0 + i) * aa.q_stride + (int64_t)head * D) * 2;
    u32x4 w[S::kSteps];
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      constexpr int per_block = S::kSteps / NB;
      const int d = s / per_block * S::kB + g * (S::kB / 4) + s % per_block * 8;
      w[s] = *reinterpret_cast<const u32x4*>(src + d * 2);
    }
    float x[S::kSteps][8];
    if (bf16) {
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[s][e] = bits_f32(e & 1 ? w[s][e >> 1] & 0xffff0000u : w[s][e >> 1] << 16);
    } else {
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[s][e] = (float)__builtin_bit_cast(f16x8, w[s])[e];
    }
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, f32_bits(x[s][e]) & 0x7fffffffu);
    const float tf = rows_max(bits_f32(top < 0x7f800000u ? top : 0u));
    const int ex = tf > 0.0f ? __builtin_amdgcn_frexp_expf(tf) : 0;  // |q| < 2^ex
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __builtin_ldexpf(x[s][2 * k], -ex), b = __builtin_ldexpf(x[s][2 * k + 1], -ex);
        // 4-bit codes: the first element of a byte is its high nibble, the high half of the table's pair
        o[k] = KB == 4 ? pack_f16(b, a) : pack_f16(a, b);
      }
      f16x8 b[O::kParts];
      O::repeat(o, b);
#pragma unroll
      for (int k = 0; k < O::kParts; ++k) s_q[((wave * S::kSteps + s) * O::kParts + k) * 64 + lane] = b[k];
    }
    if (g == 0) s_scale[wave * 16 + m] = __builtin_ldexpf(aa.scale * 1.44269504088896341f, ex - kTopBit);
  }
  __syncthreads();  // table and queries are in place
  if constexpr (TREE) {
    if (!any_node(s_tree, i_first, i_last)) end = hi_all = 0;  // no row of the tile sees any key: theirs may hold anything
  }

  // Rows of this lane (column m of the products): the keys they see, their scales.
  int lo[RT], hi[RT];
  float scale[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = tile * kRows + t * 16 + m;
    const int i = r / group;
    if constexpr (TREE) {  // of the context
      const int depth = r < nrows ? s_tree.depth[i - i_first] : -1;
      lo[t] = node_first(aa, context, depth);
      hi[t] = depth >= 0 ? context : 0;
    } else {
      lo[t] = r < nrows ? first_key(aa, sq, i) : 0;
      hi[t] = r < nrows ? end_key(aa, sq, i) : 0;
    }
    scale[t] = s_scale[t * 16 + m];
  }

  const Spread<D, NB, KB> spread(m);
  float ref[RT], sum[RT];  // reference M, sum of weights (this lane's keys)
  f32x4 acc[RT][S::kTiles];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    ref[t] = -INFINITY;
    sum[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < S::kTiles; ++i) acc[t][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Scores of the group, in the log2 domain: the lane's keys 4g .. 4g+3 of each 16.
  float s[RT][2][4];
  auto scores = [&](const Keys<D, NB, KB>& x) {
    put_maxima(0, x.a);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float ka[4][NB];
      get_maxima(0, u, ka);
      f32x4 z[RT];
#pragma unroll
      for (int k = 0; k < S::kSteps; ++k) {
        uint32_t wd[O::kLookups];
        int by[O::kLookups];
#pragma unroll
        for (int b = 0; b < O::kLookups; ++b) {
          wd[b] = x.code[u][k * S::kStepWords + b / 4];
          by[b] = b & 3;
        }
        f16x8 a[O::kParts];
        O::look_up(s_mem, copy, wd, by, a);
        constexpr int per_block = S::kSteps / NB;
        const int b = k / per_block;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (k % per_block == 0) z[t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int h = 0; h < O::kParts; ++h)
            z[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[h], s_q[((t * S::kSteps + k) * O::kParts + h) * 64 + lane], z[t], 0, 0, 0);
          if (k % per_block == per_block - 1) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              s[t][u][r] = b == 0 ? z[t][r] * ka[r][b] : fmaf(z[t][r], ka[r][b], s[t][u][r]);
            // The scaled score is rounded here, once, and not inside fused multiply-adds below: the key
            // that sets the reference then has the weight 2^-E exactly.
            if (k == S::kSteps - 1) {
#pragma unroll
              for (int r = 0; r < 4; ++r) s[t][u][r] *= scale[t];
            }
          }
        }
      }
    }
  };

  // Weights of the lane's 8 keys, block by block, as pairs of binary16.
  constexpr bool kRests = HL && Occupancy<D, NB, KB, RT>::kRests;
  u32x4 w[RT][NB], rest[RT][kRests ? NB : 1];  // and what rounding them left
  auto weights = [&](int j0, const Pages& p, const Values<D, NB, KB>& x) {
    float va[2][4][NB];
    put_maxima(1, x.a);
    get_maxima(1, 0, va[0]);
    get_maxima(1, 1, va[1]);
    if (!(j0 >= lo_all && j0 + kGroup <= hi_all && listed(p.id[0]) && listed(p.id[1]))) {  // uniform
      // Some row does not see some key.  Keys that no row of the tile sees may have any maxima: zeros.
      uint32_t used = 0, seen[RT];  // of the group's keys: new tokens that are seen, and by whom
#pragma unroll
      for (int t = 0; t < RT; ++t) seen[t] = 0;
      if constexpr (TREE) {
        const int from = j0 - context;
        if (from > -kGroup) {
          const int k = (from + 32) >> 5;
          used = __builtin_amdgcn_alignbit(s_tree.used[k + 1], s_tree.used[k], from & 31) >> (4 * g);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int i = min(tile * kRows + t * 16 + m, last_row) / group - i_first;
            seen[t] = __builtin_amdgcn_alignbit(s_tree.seen[i][k + 1], s_tree.seen[i][k], from & 31) >> (4 * g);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = j0 + 16 * u + 4 * g + r;
          const bool node = TREE && j >= context;
          const bool none = j < first || j >= end || !listed(p.id[u]) || (node && !(used >> (16 * u + r) & 1));
#pragma unroll
          for (int b = 0; b < NB; ++b) va[u][r][b] = none ? 0.0f : va[u][r][b];
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const bool hidden = node ? !(seen[t] >> (16 * u + r) & 1) : j < lo[t] || j >= hi[t];
            s[t][u][r] = none || hidden ? -INFINITY : s[t][u][r];
          }
        }
    }
    // exponents of the keys' largest value maximum (at least -99; a of zero counts as 2^-100)
    float ev[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float a = max3_hw(0x1p-100f, fabsf(va[u][r][0]), fabsf(va[u][r][NB > 1 ? 1 : 0]));
#pragma unroll
        for (int b = 2; b + 1 < NB; b += 2) a = max3_hw(a, fabsf(va[u][r][b]), fabsf(va[u][r][b + 1]));
        ev[u][r] = (float)__builtin_amdgcn_frexp_expf(a);
      }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; r += 2) top = max3_hw(top, s[t][u][r] + ev[u][r], s[t][u][r + 1] + ev[u][r + 1]);
      if (__any(top > ref[t] + kSlack)) {  // rare after the first groups: raise the reference
        const float up = fmaxf(ref[t], rows_max(top));
        const float f = ref[t] == -INFINITY ? 0.0f : exp2_hw(ref[t] - up);
        sum[t] = lower(sum[t], ref[t], up);
        ref[t] = up;
#pragma unroll
        for (int i = 0; i < S::kTiles; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][i][r] *= f;
      }
      const float safe = fmaxf(ref[t], -0x1p120f);  // no key yet: -infinity - safe is still -infinity
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const float p0 = exp2_hw(s[t][u][r] - safe), p1 = exp2_hw(s[t][u][r + 1] - safe);
          sum[t] += p0 + p1;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float w0 = p0 * va[u][r][b], w1 = p1 * va[u][r + 1][b];
            const uint32_t pair = pack_f16(w0, w1);
            w[t][b][2 * u + r / 2] = pair;
            if constexpr (kRests) {
              const f16x2 h = __builtin_bit_cast(f16x2, pair);
              rest[t][b][2 * u + r / 2] = pack_f16(w0 - (float)h.x, w1 - (float)h.y);
            }
          }
        }
    }
  };

  auto add_values = [&](Values<D, NB, KB>& x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) spread.apply(x.code[e]);
#pragma unroll
    for (int wd = 0; wd < S::kWords; ++wd) {
      uint32_t pair[4][2];  // 4-bit: both keys' codes of a pair in one byte (even and odd d's)
      if constexpr (KB == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x0 = x.code[2 * k][wd], x1 = x.code[2 * k + 1][wd];
          pair[k][0] = ((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
          pair[k][1] = (x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u);
        }
      }
      constexpr int kBytes = S::kLane < 4 ? S::kLane : 4;
      constexpr int kPer = KB == 4 ? 2 : 1;  // d's per byte
#pragma unroll
      for (int by = 0; by < kBytes; ++by)
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
          uint32_t wds[O::kLookups];
          int bys[O::kLookups];
#pragma unroll
          for (int k = 0; k < O::kLookups; ++k) {
            wds[k] = KB == 4 ? pair[k & 3][h] : x.code[k][wd];
            bys[k] = by;
          }
          f16x8 a[O::kParts];
          O::look_up(s_mem, copy, wds, bys, a);
          const int i = (4 * wd + by) * kPer + h;  // tile: place i of the lane's d's
          const int b = i / S::kPerBlock;
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            f16x8 p[O::kParts];
            O::repeat(w[t][b], p);
#pragma unroll
            for (int k = 0; k < O::kParts; ++k) acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[k], p[k], acc[t][i], 0, 0, 0);
            if constexpr (kRests) {
              O::beside(rest[t][b], p);
#pragma unroll
              for (int k = 0; k < O::kParts; ++k) acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[k], p[k], acc[t][i], 0, 0, 0);
            }
          }
        }
    }
  };

  // A group's keys are used before its values: the next group's keys are loaded into the same
  // registers in between, its values at the end, and the page numbers come one group further ahead.
  if (gi < g_end) {
    while (gi + W < g_end) {
      const Pages later = find(min(gi + 2 * W, groups - 1));
      scores(xk);
      load_fence();
      load_keys(gi + W, next, xk);
      load_fence();
      weights(begin + gi * kGroup, now, xv);
      add_values(xv);
      load_fence();
      load_values(gi + W, next, xv);
      load_fence();
      now = next;
      next = later;
      gi += W;
    }
    scores(xk);
    weights(begin + gi * kGroup, now, xv);
    add_values(xv);
  }

  // Join the waves: common reference, then their scaled sums in wave order.
  bool sees[RT];  // a row of a tree that sees nothing went along through the context
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    sees[t] = true;
    if constexpr (TREE) {
      sees[t] = s_tree.depth[min(tile * kRows + t * 16 + m, last_row) / group - i_first] >= 0;
      if (!sees[t]) {
        ref[t] = -INFINITY;
        sum[t] = 0.0f;
      }
    }
    sum[t] = rows_sum(sum[t]);
    if (g == 0) s_part[wave][t * 16 + m] = {ref[t], sum[t], sum[t]};
  }
  __syncthreads();  // also: every lookup is done, the table's memory is free
  float* s_sum = reinterpret_cast<float*>(s_mem);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < W; ++v) top = fmaxf(top, s_part[v][t * 16 + m].m);
    const float f = ref[t] == -INFINITY ? 0.0f : __builtin_ldexpf(exp2_hw(ref[t] - top), -kTopBit);
#pragma unroll
    for (int i = 0; i < S::kTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = Spread<D, NB, KB>::d_of(4 * g + r, i / S::kPerBlock, i % S::kPerBlock);
        s_sum[(wave * 16 + m) * kPitch + d] = sees[t] ? acc[t][i][r] * f : 0.0f;
      }
    __syncthreads();
#pragma unroll
    for (int c0 = 0; c0 < 16 * D / 4; c0 += kThreads) {  // groups of 4 d of the 16 rows
      const int c = c0 + tid;
      const int row = c / (D / 4), d = c % (D / 4) * 4;
      const int r = tile * kRows + t * 16 + row;
      if ((16 * D / 4) % kThreads != 0 && c >= 16 * D / 4) break;
      if (r >= nrows) continue;
      const int i = r / group, head = kvh * group + (r - i * group);
      const int64_t token = sq.q0 + i;
      float m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) m_all = fmaxf(m_all, s_part[v][t * 16 + row].m);
#pragma unroll
      for (int v = 0; v < W; ++v) {
        const Partial p = s_part[v][t * 16 + row];
        l_all += lower(p.l, p.m, m_all);
      }
      f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < W; ++v) o += *reinterpret_cast<const f32x4*>(&s_sum[(v * 16 + row) * kPitch + d]);
      if (nsplit == 1) {
        const float inv = l_all > 0.0f ? 1.0f / l_all : (l_all == 0.0f ? 0.0f : l_all);
        const u32x2 o16 = {pack16(o[0] * inv, o[1] * inv, bf16), pack16(o[2] * inv, o[3] * inv, bf16)};
        *reinterpret_cast<u32x2*>(static_cast<char*>(aa.out) + (token * aa.out_stride + (int64_t)head * D + d) * 2) = o16;
        if (d == 0 && aa.lse != nullptr) aa.lse[token * aa.heads + head] = log_sum(m_all, l_all);
      } else {
        const int64_t part = (token * aa.heads + head) * nsplit + split;
        *reinterpret_cast<f32x4*>(partial + part * D + d) = o;
        if (d == 0) reinterpret_cast<Partial*>(partial + aa.tokens * aa.heads * nsplit * D)[part] = {m_all, l_all, l_all};
      }
    }
    if (t + 1 < RT) __syncthreads();
  }
}

}  // namespace

}  // namespace bq
