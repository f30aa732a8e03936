// k_attn_chunk.hip -- attention of longer runs of new tokens over the cache.
//
// With many rows to a key the arithmetic of the products bounds the call, and decoding the codes anew
// for every tile of rows would double the vector work.  So the keys and values of the sequences that bring
// many rows are first expanded once into the workspace (expand_kernel), as binary16 in the order in which
// the matrix cores take them, and chunk_kernel multiplies from there:
//   K' = RN16(fl32(c a) 2^(14-ek)), V' = RN16(fl32(c a) 2^(14-ev)), per tile of 64 keys of a head
// with 2^ek, 2^ev powers of two above the tile's largest maximum.  Where the keys of a tile are of very different
// size (kKeySpread, kValueSpread) each key has powers of its own, so that every cached value keeps 11 bits,
// whatever the type of q and the size of the values beside it (down to 2^-16 of the largest of its key).  ek joins
// the scale of the scores.  ev joins the softmax: weights are taken relative to
//   M_i = max_j (log2-domain s_ij + ev_j)   as   w_ij = 2^(s_ij + ev_j - M_i + 3),
// so that w V' has the same unit, 2^(M - 17), in every tile, and a weight is rounded relative to the largest
// weight times value of its row and not to the largest weight.  The denominator is sum_j w_ij 2^-ev_j.
// Exponents of their own, and denominators of unrounded weights, cost where they occur: 2048 tokens over 18432 keys
// take 655 us as a rule, 935 where every tile's values are apart, 789 where the first tile's values are 2^9
// times the others' and matter to the rows (in one run).
//
// chunk_kernel: a workgroup of four waves takes 128 rows (new token x query head of one key/value
// head) and walks the tiles of 64 keys with the running maximum and sum of the softmax.  A wave takes
// 32 rows, with v_mfma_f32_32x32x16_f16; lane l = 32 g + n:
//   S^T = K' Q^T   A = K' from LDS, B = Q in registers; the result holds row n's scores of the keys
//                  8 (v / 4) + 4 g + v % 4 of each 32 (element v)
//   O^T = V'^T P^T B = P^T: 8 keys per lane and step, taken in just that order, so the weights stay where
//                  they were computed; V' is stored with its keys in the same order.
//
// What is rounded.  K', V' and the weights to binary16, each 2^-11 at most; with q in bfloat16 that is a fraction of the
// result's own rounding.  With q in binary16 (kFine) it would be four times that rounding (8.5e-4 of the result's
// norm against 2.1e-4), the keys most of it, and a sequence's bits would depend on whether a long piece stands
// beside it in the call, since bq_attend.h keeps two parts of its operands.  So what rounding left of K'
// follows in 6 bits, multiplied with q in 6 bits by v_mfma_scale_f32_32x32x64_f8f6f4 (an eighth more time on the
// matrix cores, 3/8 more key bytes), and what it left of the weights as a second binary16 product with the same V'.  V' stays
// once rounded, as bq_kv_read in that type gives it: 3.0e-4, sqrt(2) times the result's own rounding.
//
// What bounds it.  Each product of a wave reads 1 KB of LDS per 32 cycles, and four such waves are all
// that LDS delivers: matrix cores and LDS have the same least time, and neither is reached while the exponentials and
// the barrier stand between.  On MI355X (the largest library product of this type: 1189 TFLOP/s):
//   2048 tokens over 18432 keys, 32 heads over 8 of 128, bf16: 600-650 us by the box's clock (900-970 TFLOP/s), matrix
//   cores busy 52%, expansion 24 us; f16, with the rests, 910-990 us
//   777 over 6000, 8 heads over 1 of 256, bf16: 59.5 us (600 TFLOP/s, matrix cores 25%; 245 workgroups: about 13 us are
//   start and end of a workgroup, not its tiles), expansion 7.5, join 8.1; f16 91 us
//   9 sequences of up to 700 over up to 5000, 16 over 4 of 64, f16: 58 us (340 TFLOP/s, matrix cores 24%, vector units
//   about 35%: short workgroups of unequal length), expansion 13; bf16 42
#include <hip/hip_runtime.h>

#include <type_traits>

#include "bq_attn.h"
#include "bq_kv.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kTile = 64;   // keys

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x32 __attribute__((ext_vector_type(32)));
typedef int i32x6 __attribute__((ext_vector_type(6)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// What a tile's expansion leaves beside its values: exponents, whether its keys have exponents of their own (in
// an array of bytes, keys then values, tile after tile), and which of its keys some row sees.
struct TileInfo {
  int16_t ek, k_apart, ev, v_apart;
  uint64_t keys;
};

// Exponents of a tile's keys may differ by this much before each has its own.  A value 2^n below its tile's
// power of two has 11 bits while n <= 28, so keys have room to spare; a weight is rounded relative to the
// tile's largest value, 2^n too coarsely.
constexpr int kKeySpread = 12, kValueSpread = 4;
// Least exponents; a tile's zeros have it.  Sums of 2^30 weights 2^(s - M + 3) <= 2^(15 - ev) stay in range.
constexpr int kLeastKey = -100, kLeastValue = -80;

// ---- expansion ----------------------------------------------------------------------------
//
// Workgroup: the keys or the values of one tile of one head.  Fragment order of a tile (16-byte pieces of 8 binary16):
//   K' piece ((kb * D/16 + s) * 64 + 32 g + n): key 32 kb + n, d = 16 s + 8 g + 0 .. 7
//   V' piece ((db * 4 + ks) * 64 + 32 g + n):   d = 32 db + n, keys 16 ks + 8 (e / 4) + 4 g + e % 4, e = 0 .. 7
// FINE adds what rounding left of K', in 6 bits (2 of exponent, 3 of mantissa; at most 4 in magnitude): 24 bytes for
// the 32 d = 64 S + 16 i + 8 g + 0 .. 7, i = 0 .. 3, of key 32 kb + n, the first 16 of each lane before the last 8
//   words ((S * 2 + kb) * 64) * 6 + 4 (32 g + n) .. + 3 and ((S * 2 + kb) * 64) * 6 + 256 + 2 (32 g + n) .. + 1
constexpr int kRestWords(int head_dim) { return 12 * head_dim; }  // of a tile

template <int D, int KB, bool FINE>
__global__ __launch_bounds__(256) void expand_kernel(KvAttendArgs aa, DequantArgs da, int ntiles, u32x4* tiles,
                                                     TileInfo* infos, int8_t* exponents, uint32_t* rests) {
  __shared__ float s_c[256];
  __shared__ float s_a[kTile * 8];       // block maxima of the tile's keys or values; zero (theirs may be NaN) where no row sees the key
  __shared__ int64_t s_row[kTile];       // pool row of each key
  __shared__ float s_factor[kTile];      // 2^(14 - exponent) of each key, where they are apart
  __shared__ uint32_t s_listed[2];
  __shared__ u32x4 s_out[kTile * D / 8]; // values' pieces, in their order
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = blockIdx.x, kvh = blockIdx.y >> 1, side = blockIdx.y & 1, seq = blockIdx.z;
  const float entry = da.c[tid];
  const Sequence sq = sequence(aa, seq);
  const int group = aa.heads / aa.cache.kv_heads;
  if (!many_rows(min(sq.nq, aa.max_q_len), group, aa.num_seqs)) return;
  const int i_last = min(sq.nq, aa.max_q_len) - 1;
  const int first = first_key(aa, sq, 0), end = end_key(aa, sq, i_last);  // keys that some row sees
  if (tile * kTile >= end || (tile + 1) * kTile <= first) return;         // not read
  const int log2nb = __builtin_ctz(D) - aa.cache.log2b, nb = 1 << log2nb;

  s_c[tid] = entry;
  if (wave == 0) {
    const int j = tile * kTile + lane;
    const int id = j >= first && j < end ? aa.page_table[(int64_t)seq * aa.table_stride + (j >> aa.cache.log2_page)] : -1;
    const bool listed = (uint32_t)id < (uint32_t)aa.cache.num_pages;
    s_row[lane] = listed ? (((int64_t)id * aa.cache.kv_heads + kvh) << aa.cache.log2_page) +
                               (j & ((1 << aa.cache.log2_page) - 1))
                         : -1;
    const uint64_t all = __ballot(listed);
    if (lane < 2) s_listed[lane] = (uint32_t)(all >> (32 * lane));
  }
  __syncthreads();
  constexpr int kRow = D * KB / 8;
  const uint8_t* const packed = aa.cache.packed[side];
  // The codes are on their way while the maxima are worked out.
  // keys: a unit is 8 d of one key; values: 4 d of the 8 keys of a piece
  constexpr int kKeyUnits = kTile * D / 8 / 256, kValueUnits = (kTile * D / 32 + 255) / 256;
  u32x2 key_code[kKeyUnits];
  uint32_t value_code[kValueUnits][8];
  auto key_unit = [&](int p, int& key, int& d8) {
    const int s = (p >> 6) % (D / 16);
    d8 = 2 * s + ((p >> 5) & 1);
    key = (p >> 6) / (D / 16) * 32 + (p & 31);
  };
  auto value_unit = [&](int p, int e, int& key, int& d4) {
    const int oct = p / (D / 4), g = oct & 1, ks = oct >> 1;
    d4 = p % (D / 4);
    key = 16 * ks + 8 * (e >> 2) + 4 * g + (e & 3);
  };
  if (side == 0) {
#pragma unroll
    for (int k = 0; k < kKeyUnits; ++k) {
      int key, d8;
      key_unit(256 * k + tid, key, d8);
      const uint8_t* src = packed + max(s_row[key], (int64_t)0) * kRow + d8 * KB;
      if constexpr (KB == 4) key_code[k] = (u32x2){*reinterpret_cast<const uint32_t*>(src), 0u};
      else key_code[k] = *reinterpret_cast<const u32x2*>(src);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kValueUnits; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        int key, d4;
        value_unit(min(256 * k + tid, kTile * D / 32 - 1), e, key, d4);
        const uint8_t* src = packed + max(s_row[key], (int64_t)0) * kRow + d4 * KB / 2;
        value_code[k][e] = KB == 4 ? *reinterpret_cast<const uint16_t*>(src) : *reinterpret_cast<const uint32_t*>(src);
      }
  }
  for (int e = tid; e < kTile << log2nb; e += 256) {
    const int64_t row = s_row[e >> log2nb];
    s_a[e] = row >= 0 ? aa.cache.absmax[side][(row << log2nb) + (e & (nb - 1))] : 0.0f;
  }
  __syncthreads();
  // Exponents, |a| < 2^e: lane l of every wave takes key l.  Keys that no row sees have no say, nor do zero
  // keys, whose scores are zero at any scale (zero values have: their weights count).
  uint32_t top = 0;
  for (int b = 0; b < nb; ++b) top = max(top, f32_bits(s_a[(lane << log2nb) + b]) & 0x7fffffffu);
  const int least = side == 0 ? kLeastKey : kLeastValue;
  int own = min(max((int)(top >> 23) - 126, least), 120);
  const bool counts = s_row[lane] >= 0 && (side == 1 || top != 0);
  s16x2 ends = counts ? (s16x2){(short)own, (short)-own} : (s16x2){-128, -128};
#pragma unroll
  for (int x = 1; x < 64; x <<= 1)
    ends = __builtin_elementwise_max(ends, __builtin_bit_cast(s16x2, __shfl_xor(__builtin_bit_cast(int, ends), x)));
  const int ex = __builtin_amdgcn_readfirstlane(max((int)ends.x, least));
  // the same in every wave; false if no key counts
  const bool apart = __builtin_amdgcn_readfirstlane(ends.x + ends.y > (side == 0 ? kKeySpread : kValueSpread));
  const float f = __builtin_ldexpf(1.0f, kTopBit - ex);
  const int64_t at = ((int64_t)seq * aa.cache.kv_heads + kvh) * ntiles + tile;
  if (!apart || !counts) own = ex;
  if (wave == 0) exponents[(2 * at + side) * kTile + lane] = (int8_t)own;
  if (tid == 0) {
    if (side == 0) infos[at].ek = (int16_t)ex, infos[at].k_apart = apart;
    else infos[at].ev = (int16_t)ex, infos[at].v_apart = apart;
    if (side == 0) infos[at].keys = s_listed[0] | (uint64_t)s_listed[1] << 32;
  }
  if (apart) {
    if (wave == 0) s_factor[lane] = __builtin_ldexpf(1.0f, kTopBit - own);
    __syncthreads();
  }
  auto factor = [&](int key) { return apart ? s_factor[key] : f; };
  u32x4* const out = tiles + at * (2 * kTile * D / 8) + side * (kTile * D / 8);

  if (side == 0) {
#pragma unroll
    for (int k = 0; k < kKeyUnits; ++k) {
      int key, d8;
      key_unit(256 * k + tid, key, d8);
      const float a = s_a[(key << log2nb) + (d8 * 8 >> aa.cache.log2b)], to = factor(key);
      const u32x2 c = key_code[k];
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t q0 = KB == 4 ? (c.x >> (8 * i + 4)) & 15u : ((i < 2 ? c.x : c.y) >> (16 * (i & 1))) & 255u;
        const uint32_t q1 = KB == 4 ? (c.x >> (8 * i)) & 15u : ((i < 2 ? c.x : c.y) >> (16 * (i & 1) + 8)) & 255u;
        w[i] = pack_f16((s_c[q0] * a) * to, (s_c[q1] * a) * to);
      }
      out[256 * k + tid] = w;
    }
    if constexpr (FINE) {
#pragma unroll 1
      for (int u = tid; u < 2 * D; u += 256) {  // whole waves: 64 lanes of one (S, kb)
        const int key = (u >> 6 & 1) * 32 + (u & 31), g = u >> 5 & 1, S = u >> 7;
        const float to = factor(key);
        f16x32 left;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d8 = 8 * S + 2 * i + g;
          const float a = s_a[(key << log2nb) + (d8 * 8 >> aa.cache.log2b)];
          const uint8_t* src = packed + max(s_row[key], (int64_t)0) * kRow + d8 * KB;
          u32x2 c;
          if constexpr (KB == 4) c = (u32x2){*reinterpret_cast<const uint32_t*>(src), 0u};
          else c = *reinterpret_cast<const u32x2*>(src);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t q = KB == 4 ? (c.x >> (8 * (e >> 1) + ((e & 1) ? 0 : 4))) & 15u
                                       : ((e < 4 ? c.x : c.y) >> (8 * (e & 3))) & 255u;
            const float v = (s_c[q] * a) * to;
            left[8 * i + e] = (_Float16)(v - (float)(_Float16)v);
          }
        }
        const i32x6 w = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(left, 1.0f);
        uint32_t* const dst = rests + at * kRestWords(D) + (u >> 6) * 384;
        *reinterpret_cast<u32x4*>(dst + 4 * (u & 63)) = (u32x4){(uint32_t)w[0], (uint32_t)w[1], (uint32_t)w[2], (uint32_t)w[3]};
        *reinterpret_cast<u32x2*>(dst + 256 + 2 * (u & 63)) = (u32x2){(uint32_t)w[4], (uint32_t)w[5]};
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < kValueUnits; ++k) {
    const int p = 256 * k + tid;
    if (kTile * D / 32 < 256 && p >= kTile * D / 32) break;
    float v[8][4];
    int key, d4;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      value_unit(p, e, key, d4);
      const float a = s_a[(key << log2nb) + (d4 * 4 >> aa.cache.log2b)], to = factor(key);
      const uint32_t c = value_code[k][e];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t q = KB == 4 ? (c >> (8 * (i >> 1) + ((i & 1) ? 0 : 4))) & 15u : (c >> (8 * i)) & 255u;
        v[e][i] = (s_c[q] * a) * to;
      }
    }
    const int d = d4 * 4, oct = p / (D / 4);
    u32x4* dst = s_out + ((d >> 5) * 4 + (oct >> 1)) * 64 + 32 * (oct & 1) + (d & 31);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dst[i] = (u32x4){pack_f16(v[0][i], v[1][i]), pack_f16(v[2][i], v[3][i]), pack_f16(v[4][i], v[5][i]),
                       pack_f16(v[6][i], v[7][i])};
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTile * D / 8 / 256; ++k) out[256 * k + tid] = s_out[256 * k + tid];
}

// ---- attention ----------------------------------------------------------------------------

// How the products are taken: kFine with q in binary16 (below); else as rounded, with or without lse.
enum Form : int { kPlain, kLse, kFine };

// Workgroups per CU (= waves per SIMD) by registers and LDS.
template <int D, bool FINE>
constexpr int kChunkPerCu = D == 64 ? (FINE ? 2 : 3) : D == 128 ? 2 : 1;

// Weights begin at 2^kHead and grow to 2^(kHead + kSlack), the last power of two below binary16's largest: as far
// above its least step, 2^-24, as they can be.
constexpr float kHead = 3.0f;

template <int D, int FORM>
__global__ __launch_bounds__(256, (kChunkPerCu<D, FORM == kFine>)) void chunk_kernel(
    KvAttendArgs aa, int ntiles, const u32x4* tiles, const TileInfo* infos, const int8_t* exponents, const uint32_t* rests,
    int nblocks, int nsplit, float* partial) {
  constexpr bool LSE = FORM == kLse, FINE = FORM == kFine, bf16 = !FINE;
  constexpr int kSteps = D / 16, kBlocks = D / 32;
  constexpr int kPieces = kTile * D / 8;          // of keys, and of values, in a tile
  constexpr int kStage = kPieces / 256;           // pieces of each that a thread stages
  __shared__ u32x4 s_key[2][kPieces];
  __shared__ u32x4 s_value[2][kPieces];
  constexpr int kRest = kRestWords(D) / 3 / 256;  // words of the rests that a thread stages at a time
  typedef uint32_t RestWords __attribute__((ext_vector_type(kRest)));
  __shared__ __attribute__((aligned(16))) uint32_t s_rest[2][FINE ? kRestWords(D) : 4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, g = lane >> 5;
  // fastest the key/value head: with 8 of them each stays on one XCD, whose L2 its tiles share
  const int kvh = blockIdx.x % aa.cache.kv_heads, rest = blockIdx.x / aa.cache.kv_heads;
  const int split = rest % nsplit;
  const int seq = blockIdx.z;
  const int group = aa.heads / aa.cache.kv_heads;
  const Sequence sq = sequence(aa, seq);
  const int nq = min(sq.nq, aa.max_q_len);
  const int nrows = nq * group;
  const int block = nblocks - 1 - rest / nsplit;  // later rows see more keys: first
  if (block * kChunkRows >= nrows || !many_rows(nq, group, aa.num_seqs)) return;

  // Tiles of the block's rows together, and this split's.
  const int last_row = min(block * kChunkRows + kChunkRows, nrows) - 1;
  const int begin = first_key(aa, sq, block * kChunkRows / group) / kTile;
  const int end = (end_key(aa, sq, last_row / group) + kTile - 1) / kTile;
  const int count = max(end - begin, 0), per = (count + nsplit - 1) / nsplit;
  const int t_first = begin + split * per, t_end = min(t_first + per, end);
  // keys that every row of the wave sees
  const int w_first = min(block * kChunkRows + wave * 32, last_row), w_last = min(w_first + 31, last_row);
  const int lo_all = first_key(aa, sq, w_last / group), hi_all = end_key(aa, sq, w_first / group);

  const int64_t head_at = ((int64_t)seq * aa.cache.kv_heads + kvh) * ntiles;
  u32x4 stage_k[kStage], stage_v[kStage];
  auto source = [&](int t, int side) { return tiles + (head_at + t) * (2 * kPieces) + side * kPieces + tid; };
  auto fetch = [&](u32x4* stage, int t, int side) {
    const u32x4* src = source(t, side);
#pragma unroll
    for (int k = 0; k < kStage; ++k) stage[k] = src[256 * k];
  };
  // a tile ahead and by scalar loads: waiting for them does not wait for the tiles on their way
  typedef const __attribute__((address_space(4))) uint32_t* ScalarWords;
  struct Info {
    int ek, ev;
    bool apart;
    uint64_t keys;
  };
  auto find = [&](int t) {
    const ScalarWords src = (ScalarWords)(uintptr_t)(infos + head_at + t);
    return Info{(int16_t)src[0], (int16_t)src[1], (src[0] | src[1]) >> 16 != 0, src[2] | (uint64_t)src[3] << 32};
  };
  RestWords stage_r[3];
  auto rest_source = [&](int t) { return reinterpret_cast<const RestWords*>(rests + (head_at + t) * kRestWords(D)) + tid; };
  auto fetch_rests = [&](int t) {
    if constexpr (FINE) {
      const RestWords* src = rest_source(t);
#pragma unroll
      for (int k = 0; k < 3; ++k) stage_r[k] = src[256 * k];
    }
  };
  auto put_rests = [&](int b) {
    if constexpr (FINE) {
#pragma unroll
      for (int k = 0; k < 3; ++k) reinterpret_cast<RestWords*>(s_rest[b])[256 * k + tid] = stage_r[k];
    }
  };
  Info info = {0, 0, false, 0};
  if (t_first < t_end) {  // on their way while the queries are set up
    fetch(stage_k, t_first, 0);
    fetch(stage_v, t_first, 1);
    fetch_rests(t_first);
    info = find(t_first);
  }

  // Queries as operands: binary16 relative to a power of two of the row, the scale's sign included.
  const int r = block * kChunkRows + wave * 32 + n;
  const bool live = r < nrows;
  const int row_i = live ? r / group : 0;
  const int head = kvh * group + (live ? r - row_i * group : 0);
  const int64_t token = sq.q0 + row_i;
  const int lo = live ? first_key(aa, sq, row_i) : 0, hi = live ? end_key(aa, sq, row_i) : 0;
  float scale;
  f16x8 q[kSteps];
  i32x8 q_rest[FINE ? D / 64 : 1];  // four times q, in 6 bits
  {
    const char* src = static_cast<const char*>(aa.q) + (token * aa.q_stride + (int64_t)head * D + 8 * g) * 2;
    u32x4 w[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) w[s] = *reinterpret_cast<const u32x4*>(src + 32 * s);
    // magnitudes of 16-bit floats are ordered like their bits
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) top = max(top, max(w[s][k] & 0x7fffu, (w[s][k] >> 16) & 0x7fffu));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    if (top >= (bf16 ? 0x7f80u : 0x7c00u)) top = 0;
    const float tf = bf16 ? bits_f32(top << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)top);
    const int ex = tf > 0.0f ? max(__builtin_amdgcn_frexp_expf(tf), -126) : 0;  // |q| < 2^ex
    const float unit = __builtin_ldexpf(aa.scale < 0.0f ? -1.0f : 1.0f, -ex);
    if (bf16) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[s][k] = pack_f16(bits_f32(w[s][k] << 16) * unit, bits_f32(w[s][k] & 0xffff0000u) * unit);
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = w[s][k];
          const f16x2 h = __builtin_bit_cast(f16x2, x);
          w[s][k] = pack_f16((float)h.x * unit, (float)h.y * unit);
        }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = __builtin_bit_cast(f16x8, w[s]);
    if constexpr (FINE) {
#pragma unroll
      for (int S = 0; S < D / 64; ++S) {
        f16x32 x;
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = q[4 * S + i / 8][i % 8] * (_Float16)4.0f;
        const i32x6 y = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(x, 1.0f);
        q_rest[S] = (i32x8){y[0], y[1], y[2], y[3], y[4], y[5], 0, 0};
      }
    }
    scale = __builtin_ldexpf(fabsf(aa.scale) * 1.44269504088896341f, ex);
  }

  // M of the row; sums of its weights as rounded and unrounded (this lane's keys, in units of 2^(M - 3))
  float ref = -INFINITY, sum = 0.0f, exact = 0.0f;
  float least_ev = -INFINITY;  // of tiles whose rounded weights are good for the denominator
  int most_ev = -1000;         // of the tiles so far
  f32x16 acc[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][v] = 0.0f;

  // Half steps of 32 keys, so that each has independent work for the matrix cores and the vector units:
  // while half h's weights are computed from its scores, the scores of half h + 1 and the sums with
  // the weights of half h - 1 are multiplied.
  f32x16 sc[2];            // scores of the tile's two halves
  u32x4 w[2][2];           // weights of the halves, 16 keys each
  w[1][0] = w[1][1] = (u32x4){0, 0, 0, 0};
  u32x4 left[2][FINE ? 2 : 1];  // what rounding left of them
  left[1][0] = left[1][FINE ? 1 : 0] = (u32x4){0, 0, 0, 0};
  // Adds the products with the rests of 64 d of the keys of half a tile.
  auto add_rest = [&](int half, int S, const uint32_t* rest, f32x16 z) {
    const uint32_t* src = rest + (S * 2 + half) * 384;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(src + 4 * lane);
    const u32x2 hi = *reinterpret_cast<const u32x2*>(src + 256 + 2 * lane);
    const i32x8 a = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, 0, 0};
    constexpr int kFp6 = 2, kOne = 127, kQuarter = 125;  // the type (2 + 3 bits), and scales 2^(x - 127)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, q_rest[S], z, kFp6, kFp6, 0, kOne, 0, kQuarter);
  };
  auto multiply_keys = [&](int half, const u32x4* tile, const uint32_t* rest) {
    const f16x8* kp = reinterpret_cast<const f16x8*>(tile) + lane + half * kSteps * 64;
    f32x16 z;
#pragma unroll
    for (int v = 0; v < 16; ++v) z[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) z = __builtin_amdgcn_mfma_f32_32x32x16_f16(kp[k * 64], q[k], z, 0, 0, 0);
    if constexpr (FINE) {
#pragma unroll
      for (int S = 0; S < D / 64; ++S) z = add_rest(half, S, rest, z);
    }
    return z;
  };
  auto add_values = [&](int half, const u32x4* tile) {
    const f16x8* vp = reinterpret_cast<const f16x8*>(tile) + lane + half * 2 * 64;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vp[(i * 4 + ks) * 64], __builtin_bit_cast(f16x8, w[half][ks]), acc[i], 0, 0, 0);
        if constexpr (FINE)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vp[(i * 4 + ks) * 64], __builtin_bit_cast(f16x8, left[half][ks]), acc[i], 0, 0, 0);
      }
  };
  // The half step of half `half` of tile t: next = the tile (and half) whose scores follow, prev = the
  // tile whose values the other half's weights belong to; beside every second product, move(k) passes a piece on.
  auto half_step = [&](auto half_c, int t, const Info& info, const u32x4* next, const uint32_t* next_rest,
                       const u32x4* prev, auto move) {
    constexpr int half = half_c.value;
    const float ev = (float)info.ev;
    const int j0 = t * kTile + 32 * half;
    const uint32_t keys = half ? (uint32_t)(info.keys >> 32) : (uint32_t)info.keys;
    f32x16& s = sc[half];
    // The half step's products in order: scores of the next half and sums of the previous one in turn, so
    // that no product waits for the one before it, their operands read kAhead products ahead.
    constexpr int kMul = 2 * kSteps, kAhead = 6;
    const f16x8* kp = reinterpret_cast<const f16x8*>(next) + lane + (half ^ 1) * kSteps * 64;
    const f16x8* vp = reinterpret_cast<const f16x8*>(prev) + lane + (half ^ 1) * 2 * 64;
    auto operand = [&](int z) { return z & 1 ? vp[((z >> 1) % kBlocks * 4 + (z >> 1) / kBlocks) * 64] : kp[(z >> 1) * 64]; };
    f16x8 a[kMul];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) a[z] = operand(z);
    __builtin_amdgcn_sched_barrier(0);
    // at least 2^-100: a hidden key's -infinity stays what it is
    const float f = fmaxf(__builtin_ldexpf(scale, info.ek - kTopBit), 0x1p-100f);
    // the exponents of the lane's keys 8 i + 4 g .. + 3, a byte each, where they are apart (side 0: keys)
    auto own = [&](int side, int i) {
      return reinterpret_cast<const uint32_t*>(exponents)[(2 * (head_at + t) + side) * (kTile / 4) + 8 * half + 2 * i + g];
    };
    auto byte_of = [](uint32_t x, int e) { return (int)(int8_t)(x >> (8 * e)); };
    if (info.apart) {  // rare: the scores to the tile's units, the values' exponents beside them
      const float inv = 1.0f / f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t xk = own(0, i), xv = own(1, i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[4 * i + e] = fmaf((float)(byte_of(xv, e) - info.ev), inv, __builtin_ldexpf(s[4 * i + e], byte_of(xk, e) - info.ek));
      }
    }
    if (!(j0 >= lo_all && j0 + 32 <= hi_all && keys == ~0u)) {  // some key hidden from some row
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int key = 8 * (v >> 2) + (v & 3), j = j0 + 4 * g + key;
        const uint32_t hide = (~(keys >> (4 * g)) >> key) & 1u;
        s[v] = hide | (uint32_t)(j < lo) | (uint32_t)(j >= hi) ? -INFINITY : s[v];
      }
    }
    float top = -INFINITY, p = 0.0f;
    u32x4 x[2], y[2];
    // Weights of scores v .. v + 1 as 2^(score f + c), and their sums in this half step.  `part` takes the weights
    // as rounded: a row that one key fills gives that key's value.  Where lse is asked for, `whole` takes them
    // unrounded: the rounded ones would move it by up to 2^-11.
    float part = 0.0f, whole = 0.0f;
    auto weigh = [&](int v, float c) {
      const float e = exp2_hw(fmaf(s[v], f, c));
      if (v & 1) {
        uint32_t pair = pack_f16(p, e);
        asm volatile("" : "+v"(pair));  // here, beside the products, and not on the side of the branch below
        const f16x2 h = __builtin_bit_cast(f16x2, pair);
        if constexpr (!FINE) part = __builtin_amdgcn_fdot2(h, (f16x2){(_Float16)1.0f, (_Float16)1.0f}, part, false);
        if constexpr (LSE) whole += p + e;
        if constexpr (FINE) {
          part += p + e;
          y[v >> 3][(v & 7) >> 1] = pack_f16(fmaf((float)h.x, -1.0f, p), fmaf((float)h.y, -1.0f, e));
        }
        x[v >> 3][(v & 7) >> 1] = pair;
      } else {
        p = e;
      }
    };
    auto offset = [&]() { return (ev + kHead) - fmaxf(ref, -0x1p120f); };  // no key yet: -infinity stays
    float c = offset();
    auto add_left = [&](int z) {
      const int i = (z >> 1) % kBlocks, ks = (z >> 1) / kBlocks;
      acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[z], __builtin_bit_cast(f16x8, left[half ^ 1][ks]), acc[i], 0, 0, 0);
    };
    f32x16& z_next = sc[half ^ 1];
#pragma unroll
    for (int v = 0; v < 16; ++v) z_next[v] = 0.0f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int z = 0; z < kMul; ++z) {  // kept in this order
      if (z & 1) {
        const int i = (z >> 1) % kBlocks, ks = (z >> 1) / kBlocks;
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[z], __builtin_bit_cast(f16x8, w[half ^ 1][ks]), acc[i], 0, 0, 0);
      } else {
        z_next = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[z], q[z >> 1], z_next, 0, 0, 0);
      }
      if constexpr (FINE) {
        if (z % 8 == 7) z_next = add_rest(half ^ 1, z / 8, next_rest, z_next);
        if (z & 1) add_left(z);
      }
      if (z + kAhead < kMul) a[z + kAhead] = operand(z + kAhead);
      if (z & 1) move(z >> 1);
#pragma unroll
      for (int v = z * 16 / kMul; v < (z + 1) * 16 / kMul; ++v) {
        weigh(v, c);
        if (v & 1) top = max3_hw(top, s[v - 1], s[v]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    top = fmaf(top, f, ev);
    if (__any(top > ref + kSlack)) {
      // Rare after the first tiles: a larger reference.  The sums so far move to it, and the weights are taken
      // again.
      const u32x2 o = __builtin_amdgcn_permlane32_swap(f32_bits(top), f32_bits(top), false, false);
      const float up = fmaxf(ref, fmaxf(bits_f32(o.x), bits_f32(o.y)));
      const float down = ref == -INFINITY ? 0.0f : exp2_hw(ref - up);
      sum = lower(sum, ref, up);
      if constexpr (LSE) exact = lower(exact, ref, up);
      if constexpr (!FINE) least_ev = up > ref ? ev - kHead : least_ev;
      ref = up;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][v] *= down;
      part = whole = 0.0f;
      c = offset();
#pragma unroll
      for (int v = 0; v < 16; ++v) weigh(v, c);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      w[half][ks] = x[ks];
      if constexpr (FINE) left[half][ks] = y[ks];
    }
    // The denominator.  It is at least 2^(3 - ev) of the tile that M is from, and a rounded weight, times 2^-ev of
    // its own tile, is off by up to 2^(-25 - ev) at the least: nothing beside it unless the tile's values are more than 2^3 times
    // smaller.  Then, and where the keys have exponents of their own, it takes weights that are not rounded and
    // do not hold the exponent.  (kFine sums unrounded weights anyway; these lose what counts below 2^-126 only.)
    if constexpr (FINE) most_ev = max(most_ev, info.ev);
    if (info.apart || (FINE ? info.ev < most_ev - 60 : __any(ev < least_ev))) {
      float more = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t xv = own(1, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) more += exp2_hw(fmaf(s[4 * i + e], f, c) - (float)byte_of(xv, e));
      }
      sum += more;
      if constexpr (LSE) exact += more;
    } else {
      sum += __builtin_ldexpf(part, -info.ev);
      if constexpr (LSE) exact += __builtin_ldexpf(whole, -info.ev);
    }
  };

  if (t_first < t_end) {
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      s_key[0][256 * k + tid] = stage_k[k];
      s_value[1][256 * k + tid] = (u32x4){0, 0, 0, 0};  // no weights wait at first
    }
    put_rests(0);
    fetch(stage_k, min(t_first + 1, t_end - 1), 0);
    fetch_rests(min(t_first + 1, t_end - 1));
    __syncthreads();
    sc[0] = multiply_keys(0, s_key[0], s_rest[0]);
    for (int t = t_first; t < t_end; ++t) {
      const int b = (t - t_first) & 1;
      const Info info_next = find(min(t + 1, t_end - 1));
      // The next tile's keys and this one's values go from registers to LDS, and those that follow them are
      // asked for, one piece at a time beside the products (613 us for 2048 tokens over 18432 keys, 32 heads of
      // 128, and 57.2 for 777 over 6000, 8 of 256; all at once between the half steps 657 and 65.3).  The buffers
      // written were last read before the previous barrier.
      const u32x4* src_k = source(min(t + 2, t_end - 1), 0);
      const u32x4* src_v = source(min(t + 1, t_end - 1), 1);
      auto ask = [&](int k) {
        u32x4& piece = k < kStage ? stage_k[k] : stage_v[k - kStage];
        piece = k < kStage ? src_k[256 * k] : src_v[256 * (k - kStage)];
      };
      put_rests(b ^ 1);
      half_step(std::integral_constant<int, 0>(), t, info, s_key[b], s_rest[b], s_value[b ^ 1], [&](int k) {
        u32x4& piece = k < kStage ? stage_k[k] : stage_v[k - kStage];
        u32x4* dst = k < kStage ? s_key[b ^ 1] + 256 * k : s_value[b] + 256 * (k - kStage);
        dst[tid] = piece;
        if constexpr (!FINE) ask(k);
      });
      __syncthreads();
      fetch_rests(min(t + 2, t_end - 1));
      half_step(std::integral_constant<int, 1>(), t, info, s_key[b ^ 1], s_rest[b ^ 1], s_value[b], [&](int k) {
        if constexpr (FINE) ask(k);
      });
      info = info_next;
    }
    add_values(1, s_value[(t_end - 1 - t_first) & 1]);
  }

  const u32x2 o2 = __builtin_amdgcn_permlane32_swap(f32_bits(sum), f32_bits(sum), false, false);
  const float unit = __builtin_ldexpf(1.0f, -kTopBit);  // of the sums beside those of the weights
  const float l = bits_f32(o2.x) + bits_f32(o2.y);
  if constexpr (LSE) {
    const u32x2 o3 = __builtin_amdgcn_permlane32_swap(f32_bits(exact), f32_bits(exact), false, false);
    exact = bits_f32(o3.x) + bits_f32(o3.y);
  }
  if (!live) return;
  const int64_t part = (token * aa.heads + head) * nsplit + split;
  const float inv = nsplit > 1 ? unit : (l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l)) * unit;
#pragma unroll
  for (int k = 0; k < kBlocks; ++k)
#pragma unroll
    for (int v = 0; v < 16; v += 4) {
      const int d = 32 * k + 2 * v + 4 * g;
      const f32x4 o = {acc[k][v] * inv, acc[k][v + 1] * inv, acc[k][v + 2] * inv, acc[k][v + 3] * inv};
      if (nsplit > 1) {
        *reinterpret_cast<f32x4*>(partial + part * D + d) = o;
      } else {
        const u32x2 o16 = {pack16(o[0], o[1], bf16), pack16(o[2], o[3], bf16)};
        *reinterpret_cast<u32x2*>(static_cast<char*>(aa.out) + (token * aa.out_stride + (int64_t)head * D + d) * 2) = o16;
      }
    }
  if (g == 0) {
    if (nsplit > 1) reinterpret_cast<Partial*>(partial + aa.tokens * aa.heads * nsplit * D)[part] = {ref - kHead, l, FINE ? l : exact};
    else if (LSE || (FINE && aa.lse != nullptr)) aa.lse[token * aa.heads + head] = log_sum(ref - kHead, FINE ? l : exact);
  }
}

template <int D, int KB>
hipError_t launch_expand(const KvAttendArgs& a, const ChunkPlan& p, bool fine, const DequantArgs& da, hipStream_t s) {
  char* const ws = static_cast<char*>(a.workspace);
  const dim3 grid((unsigned)p.ntiles, (unsigned)a.cache.kv_heads * 2, (unsigned)a.num_seqs);
  return launch_kernel(fine ? expand_kernel<D, KB, true> : expand_kernel<D, KB, false>, grid, dim3(256), s, a, da, p.ntiles,
                       reinterpret_cast<u32x4*>(ws), reinterpret_cast<TileInfo*>(ws + p.info_at),
                       reinterpret_cast<int8_t*>(ws + p.exponents_at), reinterpret_cast<uint32_t*>(ws + p.rest_at));
}

template <int D>
hipError_t launch_chunk(const KvAttendArgs& a, const ChunkPlan& p, bool fine, const DequantArgs& da, hipStream_t s) {
  const hipError_t e = da.K == 16 ? launch_expand<D, 4>(a, p, fine, da, s) : launch_expand<D, 8>(a, p, fine, da, s);
  if (e != hipSuccess) return e;
  char* const ws = static_cast<char*>(a.workspace);
  const dim3 grid((unsigned)(a.cache.kv_heads * p.nsplit * p.blocks), 1u, (unsigned)a.num_seqs);
  const auto kernel = fine ? chunk_kernel<D, kFine> : a.lse != nullptr ? chunk_kernel<D, kLse> : chunk_kernel<D, kPlain>;
  return launch_kernel(kernel, grid, dim3(256), s, a, p.ntiles, reinterpret_cast<const u32x4*>(ws),
                       reinterpret_cast<const TileInfo*>(ws + p.info_at), reinterpret_cast<const int8_t*>(ws + p.exponents_at),
                       reinterpret_cast<const uint32_t*>(ws + p.rest_at), p.blocks, p.nsplit,
                       reinterpret_cast<float*>(ws + p.partial_at));
}

template <bool FINE>
int slots(int head_dim) {
  return cu_count() * (head_dim == 64 ? kChunkPerCu<64, FINE> : head_dim == 128 ? kChunkPerCu<128, FINE> : kChunkPerCu<256, FINE>);
}

}  // namespace

// Workgroups of the attention kernel that the device holds at once.
int chunk_slots(int head_dim, int dtype) { return dtype == F16 ? slots<true>(head_dim) : slots<false>(head_dim); }

// Bytes of a tile beside its 256 head_dim: the rests.
int64_t chunk_rest_bytes(int head_dim, int dtype) { return dtype == F16 ? 4 * kRestWords(head_dim) : 0; }

static_assert(sizeof(TileInfo) == kTileInfoBytes && kTile == 64, "workspace layout");

int launch_kv_chunk(const KvAttendArgs& a, int dtype, const ChunkPlan& p, const DequantArgs& da, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool fine = dtype == F16;
  if (a.cache.head_dim == 64) return (int)launch_chunk<64>(a, p, fine, da, s);
  if (a.cache.head_dim == 128) return (int)launch_chunk<128>(a, p, fine, da, s);
  return (int)launch_chunk<256>(a, p, fine, da, s);
}

}  // namespace bq
