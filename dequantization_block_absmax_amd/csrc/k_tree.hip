// k_tree.hip -- attention of a tree of drafted tokens over the cache, for drafts with many rows to a key/value head.
//
//   o_i = sum_j p_ij v_j,   p_ij = exp(s_ij) / sum_j exp(s_ij),   s_ij = scale * (q_i . k_j)
// over the keys j that row i sees: the context within its window, its ancestors and itself; one pass with the running maximum
// and sum of the softmax.
//
// Work decomposition.  A workgroup takes 128 rows (new token x query head of one key/value head) and a run of tiles of 64 keys
// (find_part).  Waves 0 to 3 multiply, 32 rows each, on v_mfma_f32_32x32x16_f16; waves 4 to 7 decode: a lane takes a quarter of a
// key's head, looks its codes up in a table in LDS, multiplies by the block maximum and rounds once to binary16, relative to a power
// of two of the tile (of the key, where keys differ too much).  So each code is decoded once for 128 rows, where the kernel of
// bq_attend.h decodes it once for 16 to 64.  Keys go to LDS in the order of the first product's operands, values by rows,
// their 16-byte chunks permuted so that neither the stores nor the transposed loads (ds_read_b64_tr_b16) of the second product's
// operands meet in a bank.  Both have two buffers, so that one barrier a tile is enough: while tile t is multiplied, the keys of
// t + 1 and the values of t are decoded and the exponents of t + 2 found.  A multiplying wave takes half a tile at a time: the
// products of the next half's scores, those of the last half's weights with their values, and this half's exponentials
// stand in turn, in an order that is kept.  With q in binary16 what rounding left of the keys follows in 6 bits through
// v_mfma_scale_f32_32x32x64_f8f6f4, and what it left of the weights as second products; values are rounded once.
//
// What bounds it.  Nothing alone: in the steady state a tile takes about 3900 cycles of a compute unit, of which the matrix cores have
// work for 1024, LDS for about 1800 and the vector units for about 2200; decoding alone, without the products, took 129 us of 188 in
// the first case below and 179 of 266 in the third (before two of its waves looked a tile ahead).  On MI355X, a call's time with its join
// after some 30 ms of such calls (12% more in the first few, until the clock has risen), and the kernel's own:
//   24 drafts of up to 32 tokens over up to 8192 keys, 32 heads over 8, 4-bit, B = 64, bf16: 150 us, 366 TFLOP/s; 138, 396
//   2 of 48 over up to 131072, 16 over 2, 8-bit, B = 128, f16: 178 us, 383 TFLOP/s; 170, 402
//   2 of 256 over up to 18432, 32 over 4, 4-bit, B = 64, bf16: 213 us, 499 TFLOP/s; 202, 526
// With q in binary16 <128, 8> spills 16 registers and <128, 4> 10, in the loop.
// Other forms, same cases: four waves that decode between their own products, two workgroups to a compute unit, 155, 272 and 232 us;
// all eight waves in both roles with keys held in registers spilled; loads four tiles ahead instead of one 189, 194 and 268 against
// 188, 188 and 266; one workgroup to each run of a fixed length, without numbering, 169, 354 and 210.  Against
// 148, 175 and 210: the decoding waves at a higher priority 158, 181 and 228, the others at one no change; a half's first operands asked for
// at the end of the half before 148, 259 (registers spilled) and 210.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "bq_attend.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kTile = 64;   // keys
constexpr int kRows = kTreeBlockRows;  // new token x query head of one key/value head
constexpr int kLeastTiles = 4;  // of a workgroup, where the keys are split
constexpr int kPartTiles = 8;   // that a part costs besides its own
constexpr int kThreads = 512;  // four waves with 32 rows each, and four that decode

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x32 __attribute__((ext_vector_type(32)));
typedef int i32x6 __attribute__((ext_vector_type(6)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// A tile's keys are apart where their largest block maxima differ by more than 2^kKeySpread: then binary16 would lose bits of the
// small ones relative to the largest.  The same of values by 2^kValueSpread, whose weights have to stay in binary16's range too.
// Exponents end at the least that the sums' scale allows.  kHead: log2 of the room above a weight of 1 that the reference may
// fall short by, kSlack of it before it moves.
constexpr int kKeySpread = 12, kValueSpread = 4;
constexpr int kLeastKey = -100, kLeastValue = -80;
constexpr float kHead = 3.0f;

// A decoding thread takes D / 4 consecutive d of one key: lane = key, wave = quarter of the head.
template <int D, int KB, bool FINE>
struct Decode {
  static constexpr int kPart = D / 4;
  static constexpr int kPieces = kPart / 8;          // of 8 d, 16 bytes of binary16
  static constexpr int kRow = D * KB / 8;            // bytes of a key's codes
  static constexpr int kWords = kPart * KB / 32;     // of a thread's codes
  static constexpr int kPieceWords = KB / 4;
  static constexpr int kBlocks = D / 32;             // most blocks of a head
  static constexpr int kEntry = FINE && KB == 4 ? 8 : 4;  // bytes of a table entry
  static constexpr int kLookups = KB == 4 ? 4 : 8;   // of a piece
  typedef std::conditional_t<FINE && KB == 4, f32x2, uint32_t> Entry;
};

// What a decoding thread loads of its key for one interval: codes of a tile's keys and of the values of the tile before, and the
// block maxima of its own d; and, ahead of that, the maxima of the whole head for what there is to know of a later tile.
template <int D, int KB, bool FINE>
struct Raw {
  uint32_t code[2][Decode<D, KB, FINE>::kWords];
  float own[2], all[Decode<D, KB, FINE>::kBlocks];
};

// What there is to know of a tile, left in LDS for the waves that multiply: of its keys and of its values 2^e above the largest
// maximum and, where they are apart, every key's own exponents; which keys some row sees.
struct Info {
  int e[2], apart[2];
  uint64_t keys;
  int8_t own[2][kTile];
};
constexpr int kInfos = 4;  // while one is written, those of the three tiles before may be read

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  u32x2 s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = max(s.x, s.y);
  s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)max(s.x, s.y));
}

__device__ __forceinline__ int exponent(uint32_t bits, int least) { return min(max((int)(bits >> 23) - 126, least), 120); }

template <int D, int KB, bool FINE>
__global__ __launch_bounds__(kThreads, 2) void tree_kernel(KvAttendArgs aa, DequantArgs da, int nsplit, int workgroups, float* partial) {
  using C = Decode<D, KB, FINE>;
  constexpr bool bf16 = !FINE;
  constexpr int kSteps = D / 16, kBlocks = D / 32;
  constexpr int kTilePieces = kTile * D / 8;
  __shared__ u32x4 s_key[2][kTilePieces];
  __shared__ __attribute__((aligned(16))) char s_value[2][kTilePieces * 16];
  __shared__ __attribute__((aligned(16))) uint32_t s_rest[2][FINE ? 12 * D : 4];
  __shared__ __attribute__((aligned(16))) char s_table[256 * kEntryBytes];
  __shared__ Info s_info[kInfos];
  __shared__ TreeShared<kRows> s_tree;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const bool decodes = __builtin_amdgcn_readfirstlane(tid >> 8);
  const int n = lane & 31, g = lane >> 5;
  float entry_lo = 0.0f, entry_hi = 0.0f;
  if (decodes) {
    entry_lo = da.c[KB == 4 ? tid & 15 : tid & 255];
    entry_hi = da.c[KB == 4 ? tid >> 4 & 15 : tid & 255];
  }
  load_fence();
  const int group = aa.heads / aa.cache.kv_heads;
  Part part;
  if (!find_part<kRows, kTile, kTile>(aa, group, nsplit, workgroups, kLeastTiles, kPartTiles, part)) return;
  const int kvh = part.kvh, block = part.block, seq = part.seq, split = part.split;
  const Sequence sq = sequence(aa, seq);
  const int nrows = min(sq.nq, aa.max_q_len) * group;
  const int last_row = min(block * kRows + kRows, nrows) - 1;
  const int i_first = block * kRows / group, i_last = last_row / group;
  const int context = sq.kv - sq.nq;
  const int first = node_first(aa, context, 0);
  int last = max(min(sq.kv, context + i_last + 1), 0);  // end of the keys that some row may see
  const int begin = first / kTile, end = (last + kTile - 1) / kTile;
  const int t_first = begin + split * part.per, t_end = min(t_first + part.per, end);
  if (split == 0)
    for (int r = tid; r < kRows; r += kThreads) no_parts<D>(aa, part, sq, nrows, nsplit, block * kRows + r, partial);
  const int lo_all = node_first(aa, context, i_last);
  int hi_all = context;

  const int parent = tid <= i_last ? aa.parents[sq.q0 + tid] : -2;
  // ---- the cache: rows of the pool, codes and maxima of the thread's key of a tile
  const int lps = aa.cache.log2_page, log2b = aa.cache.log2b, nb = D >> log2b;
  const int32_t* const pages = aa.page_table + (int64_t)seq * aa.table_stride;
  const int last_page = sq.kv > 0 ? (sq.kv - 1) >> lps : 0;
  auto page_of = [&](int t) { return pages[min((min(t, t_end - 1) * kTile + lane) >> lps, last_page)]; };
  auto listed = [&](int id) { return (uint32_t)id < (uint32_t)aa.cache.num_pages; };
  auto row_of = [&](int t, int id) {
    const int j = min(t, t_end - 1) * kTile + lane;
    return (((int64_t)(listed(id) ? id : 0) * aa.cache.kv_heads + kvh) << lps) + (j & ((1 << lps) - 1));
  };
  auto fetch = [&](Raw<D, KB, FINE>& x, int64_t row, int64_t row_before) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int64_t from = side == 0 ? row : row_before;
      const uint8_t* src = aa.cache.packed[side] + from * C::kRow + wave * (C::kPart * KB / 8);
#pragma unroll
      for (int k = 0; k < C::kWords; k += 4) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(src + 4 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) x.code[side][k + e] = v[e];
      }
      x.own[side] = aa.cache.absmax[side][from * nb + (wave * C::kPart >> log2b)];
    }
  };
  auto fetch_all = [&](Raw<D, KB, FINE>& x, int64_t row) {
    if (wave < 2) {
      const float* a = aa.cache.absmax[wave] + row * nb;
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b) x.all[b] = a[min(b, nb - 1)];
    }
  };
  // Interval t takes the codes in raw[k] and the maxima there, those of tile t + 1; k takes turns.
  Raw<D, KB, FINE> raw[2];
  int id[2] = {0, 0};               // page of the lane's key of tile t + 2, in id[k]
  int64_t row0 = 0, row1 = 0;       // its rows of tiles t and t + 1
  bool listed0 = false, listed1 = false;
  if (decodes && t_first < t_end) {
    const int id0 = page_of(t_first), id1 = page_of(t_first + 1);
    id[0] = page_of(t_first + 2);
    listed0 = listed(id0);
    row0 = row_of(t_first, id0);
    fetch_all(raw[1], row0);
    fetch(raw[0], row0, row0);
    listed1 = listed(id1);
    row1 = row_of(t_first + 1, id1);
    fetch_all(raw[0], row1);
  }

  if (decodes) {  // table
    const float x0 = __builtin_ldexpf(entry_lo, kTopBit), x1 = __builtin_ldexpf(entry_hi, kTopBit);
    const uint32_t w = pack_f16(x1, x0);
    const u32x4 e = FINE && KB == 4 ? (u32x4){f32_bits(x1), f32_bits(x0), f32_bits(x1), f32_bits(x0)}
                    : FINE          ? (u32x4){f32_bits(x0), f32_bits(x0), f32_bits(x0), f32_bits(x0)}
                                    : (u32x4){w, w, w, w};
    const int to = tid & 255;
#pragma unroll
    for (int i = 0; i < kEntryBytes / 16; ++i)  // in turn over the banks
      *reinterpret_cast<u32x4*>(s_table + to * kEntryBytes + ((i + to) & (kEntryBytes / 16 - 1)) * 16) = e;
  }
  const uint32_t copy = (lane * C::kEntry) & (kEntryBytes - 1);

  // Queries as operands: binary16 relative to a power of two of the row, the scale's sign included.
  const int r = block * kRows + wave * 32 + n;
  const bool live = r < nrows;
  const int row_i = live ? r / group : i_first;
  const int head = kvh * group + (live ? r - row_i * group : 0);
  const int64_t token = sq.q0 + row_i;
  float scale = 0.0f;
  f16x8 q[kSteps];
  i32x8 q_rest[FINE ? D / 64 : 1];  // four times q, in 6 bits
  if (!decodes) {
    // d = 8 (2 s + g) .. + 7 for step s
    const char* src = static_cast<const char*>(aa.q) + (token * aa.q_stride + (int64_t)head * D + 8 * g) * 2;
    u32x4 w[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) w[s] = *reinterpret_cast<const u32x4*>(src + 32 * s);
    uint32_t top = 0;  // magnitudes of 16-bit floats are ordered like their bits
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) top = max(top, max(w[s][k] & 0x7fffu, (w[s][k] >> 16) & 0x7fffu));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    if (top >= (bf16 ? 0x7f80u : 0x7c00u)) top = 0;
    const float tf = bf16 ? bits_f32(top << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)top);
    const int ex = tf > 0.0f ? max(__builtin_amdgcn_frexp_expf(tf), -126) : 0;  // |q| < 2^ex
    const float unit = __builtin_ldexpf(aa.scale < 0.0f ? -1.0f : 1.0f, -ex);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = w[s][k];
        const f16x2 h = __builtin_bit_cast(f16x2, x);
        w[s][k] = bf16 ? pack_f16(bits_f32(x << 16) * unit, bits_f32(x & 0xffff0000u) * unit) : pack_f16((float)h.x * unit, (float)h.y * unit);
      }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = __builtin_bit_cast(f16x8, w[s]);
    if constexpr (FINE) {
      // the rests' order: lane g has d = 64 S + 32 g + 0 .. 31, of which the other half lane holds two pieces
#pragma unroll
      for (int S = 0; S < D / 64; ++S) {
        f16x32 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // piece 8 S + 4 g + i is step 4 S + 2 g + i / 2 of half lane i & 1
          u32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = __shfl((int)w[4 * S + i / 2][e], n + 32 * (i & 1));
            const uint32_t hi = __shfl((int)w[4 * S + 2 + i / 2][e], n + 32 * (i & 1));
            v[e] = g ? hi : lo;
          }
          const f16x8 p = __builtin_bit_cast(f16x8, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[8 * i + e] = p[e] * (_Float16)4.0f;
        }
        const i32x6 y = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(x, 1.0f);
        q_rest[S] = (i32x8){y[0], y[1], y[2], y[3], y[4], y[5], 0, 0};
      }
    }
    scale = __builtin_ldexpf(fabsf(aa.scale) * 1.44269504088896341f, ex);
  }
  read_tree<kThreads, kRows>(aa, s_tree, parent, tid, i_first, i_last);
  __syncthreads();  // table and tree are in place
  if (!any_node(s_tree, i_first, i_last)) last = hi_all = 0;  // no row of the block sees any key: theirs may hold anything
  const int depth = s_tree.depth[row_i - i_first];
  const uint32_t* const seen = s_tree.seen[row_i - i_first];
  const int lo = node_first(aa, context, depth), hi = depth >= 0 ? context : 0;  // of the context

  // Whether some row sees the lane's key of tile t.
  auto counts = [&](int t, bool in_pool) {
    const int j = t * kTile + lane, node = j - context;
    const bool used = node < 0 || (node < kMostNodes && (s_tree.used[(node >> 5) + 1] >> (node & 31) & 1));
    return j >= first && j < last && in_pool && used;
  };

  // ---- decoding
  // What there is to know of a tile: wave 0 finds out about its keys, wave 1 about its values.
  auto learn = [&](int t, bool in_pool, const float (&all)[C::kBlocks]) {
    if (wave > 1) return;
    Info& info = s_info[t & (kInfos - 1)];
    const uint64_t keys = __ballot(counts(min(t, t_end - 1), in_pool));
    const bool seen_key = keys >> lane & 1;
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < C::kBlocks; ++b) top = max(top, f32_bits(all[b]) & 0x7fffffffu);
    top = seen_key ? top : 0u;
    const bool say = seen_key && (wave == 1 || top != 0);  // zero keys, whose scores are zero at any scale, have none
    const int least = wave == 0 ? kLeastKey : kLeastValue;
    const uint32_t most = wave_max_bits(say ? top : 0u), low = ~wave_max_bits(say ? ~top : 0u);
    const int e = exponent(most, least);
    const bool apart = low <= most && e - exponent(low, least) > (wave == 0 ? kKeySpread : kValueSpread);
    info.own[wave][lane] = (int8_t)(apart && say ? exponent(top, least) : e);
    if (lane == 0) {
      info.e[wave] = e;
      info.apart[wave] = apart;
      info.keys = keys;  // the same of both
    }
  };
  // The block maximum of the d that the thread decodes, relative to the tile's exponent or the key's own.
  auto relative = [&](float own, int side, int t) {
    const Info& info = s_info[t & (kInfos - 1)];
    const float a = __builtin_ldexpf(own, -info.own[side][lane]);
    return info.keys >> lane & 1 ? a : 0.0f;
  };
  auto entry_at = [&](uint32_t w, int b) { return *reinterpret_cast<const typename C::Entry*>(s_table + entry_of(w, b, copy)); };
  auto look_up = [&](const uint32_t (&code)[C::kWords], int i, typename C::Entry (&e)[C::kLookups]) {
#pragma unroll
    for (int k = 0; k < C::kLookups; ++k) e[k] = entry_at(code[i * C::kPieceWords + k / 4], k & 3);
  };
  // The 8 values of piece i: rounded once to binary16, and what that left (times the tile's power of two).
  auto products = [&](float a, const typename C::Entry (&e)[C::kLookups], f16x8* left) {
    u32x4 h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (FINE) {
        float v0, v1;
        if constexpr (KB == 4) {
          v0 = e[k].x * a;
          v1 = e[k].y * a;
        } else {
          v0 = bits_f32(e[2 * k]) * a;
          v1 = bits_f32(e[2 * k + 1]) * a;
        }
        const uint32_t pair = pack_f16(v0, v1);
        h[k] = pair;
        if (left != nullptr) {
          const f16x2 y = __builtin_bit_cast(f16x2, pair);
          (*left)[2 * k] = (_Float16)(v0 - (float)y.x);
          (*left)[2 * k + 1] = (_Float16)(v1 - (float)y.y);
        }
      } else {
        f16x2 c;
        if constexpr (KB == 4) {
          const uint32_t x2 = e[k];
          c = __builtin_bit_cast(f16x2, x2);
        } else {
          const uint32_t x0 = e[2 * k], x1 = e[2 * k + 1];
          c.x = __builtin_bit_cast(f16x2, x0).x;
          c.y = __builtin_bit_cast(f16x2, x1).x;
        }
        // mixed-precision instructions: one rounding, to binary16
        const f16x2 y = {(_Float16)__builtin_fmaf((float)c.x, a, 0.0f), (_Float16)__builtin_fmaf((float)c.y, a, 0.0f)};
        h[k] = __builtin_bit_cast(uint32_t, y);
      }
    }
    return h;
  };
  const int key_to = (lane >> 5) * kSteps * 64 + (lane & 31);
  const int turn = 2 * (lane & 3) + (lane >> 2 & 1);  // see value_at
  auto put_key = [&](int b, int i, const u32x4& h) {
    const int d8 = wave * C::kPieces + i;
    s_key[b][key_to + (d8 >> 1) * 64 + 32 * (d8 & 1)] = h;
  };
  auto put_value = [&](int b, int i, const u32x4& h) {
    *reinterpret_cast<u32x4*>(s_value[b] + lane * (2 * D) + ((wave * C::kPieces + i) ^ turn) * 16) = h;
  };
  f16x32 left;  // of 32 d of the key
  auto put_rest = [&](int b, int part) {  // d = 32 part .. of the head
    if constexpr (FINE) {
      const i32x6 w = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(left, 1.0f);
      // 24 bytes for lane 32 (part & 1) + n of S = part / 2, half = key / 32; the first 16 of each lane before the last 8
      const int l = 32 * (part & 1) + (lane & 31);
      const int dst = ((part >> 1) * 2 + (lane >> 5)) * 384;
      *reinterpret_cast<u32x4*>(&s_rest[b][dst + 4 * l]) = (u32x4){(uint32_t)w[0], (uint32_t)w[1], (uint32_t)w[2], (uint32_t)w[3]};
      *reinterpret_cast<u32x2*>(&s_rest[b][dst + 256 + 2 * l]) = (u32x2){(uint32_t)w[4], (uint32_t)w[5]};
    }
  };
  // Piece i of the keys from its entries, with what rounding left of it.
  auto finish_key = [&](int b, int i, float a, const typename C::Entry (&e)[C::kLookups]) {
    f16x8 l;
    put_key(b, i, products(a, e, FINE ? &l : nullptr));
    if constexpr (FINE) {
#pragma unroll
      for (int k = 0; k < 8; ++k) left[8 * (i & 3) + k] = l[k];
      if (i % 4 == 3) put_rest(b, wave * (C::kPieces / 4) + i / 4);
    }
  };
  // Where a lane reads the values' operands: rows of 16-byte chunks, chunk c of key k at place c ^ (2 (k & 3) + (k >> 2 & 1)), so that
  // neither the writes (a key to a lane) nor the transposed reads (4 keys x 16 d to 16 lanes) meet in a bank.
  const int x_of = 2 * (lane >> 4 & 1) + (lane >> 1 & 1), turn_r = 2 * (lane >> 2 & 3) + g;
  const int value_base = ((lane >> 2 & 3) + 4 * g) * (2 * D) + 8 * (lane & 1);
  const int value_at[2] = {value_base + (x_of ^ turn_r) * 16, value_base + (x_of ^ turn_r ^ 4) * 16};
  auto value_operand = [&](int b, int half, int i, int ks) {  // d = 32 i .., keys 32 half + 16 ks ..
    typedef __attribute__((address_space(3))) s16x4* Local;
    const char* at = s_value[b] + value_at[i & 1] + (i >> 1) * 128 + (32 * half + 16 * ks) * (2 * D);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Local)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Local)(at + 8 * (2 * D)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(f16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  // M of the row; sum of its weights (this lane's keys, in units of 2^(M - 3))
  float ref = -INFINITY, sum = 0.0f;
  int most_ev = -1000;  // of the tiles so far
  f32x16 acc[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][v] = 0.0f;
  f32x16 sc[2];
  u32x4 w[2][2];
  w[1][0] = w[1][1] = (u32x4){0, 0, 0, 0};
  u32x4 wl[2][FINE ? 2 : 1];  // what rounding left of them
  wl[1][0] = wl[1][FINE ? 1 : 0] = (u32x4){0, 0, 0, 0};
  auto add_rest = [&](int half, int S, const uint32_t* rest, f32x16 z) {
    const uint32_t* src = rest + (S * 2 + half) * 384;
    const u32x4 a4 = *reinterpret_cast<const u32x4*>(src + 4 * lane);
    const u32x2 a2 = *reinterpret_cast<const u32x2*>(src + 256 + 2 * lane);
    const i32x8 a = {(int)a4.x, (int)a4.y, (int)a4.z, (int)a4.w, (int)a2.x, (int)a2.y, 0, 0};
    constexpr int kFp6 = 2, kOne = 127, kQuarter = 125;
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, q_rest[S], z, kFp6, kFp6, 0, kOne, 0, kQuarter);
  };
  auto multiply_keys = [&](int half, int b) {
    const f16x8* kp = reinterpret_cast<const f16x8*>(s_key[b]) + lane + half * kSteps * 64;
    f32x16 z;
#pragma unroll
    for (int v = 0; v < 16; ++v) z[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) z = __builtin_amdgcn_mfma_f32_32x32x16_f16(kp[k * 64], q[k], z, 0, 0, 0);
    if constexpr (FINE) {
#pragma unroll
      for (int S = 0; S < D / 64; ++S) z = add_rest(half, S, s_rest[b], z);
    }
    return z;
  };

  // A tile's Info as the waves that multiply hold it.
  struct Known {
    int ek, ev, apart;
    uint64_t keys;
  };
  auto known = [&](int t) {
    const Info& x = s_info[t & (kInfos - 1)];
    return Known{__builtin_amdgcn_readfirstlane(x.e[0]), __builtin_amdgcn_readfirstlane(x.e[1]), __builtin_amdgcn_readfirstlane(x.apart[0] | x.apart[1] << 1),
                 (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)x.keys) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x.keys >> 32)) << 32};
  };
  // The half step of half `half` of tile t: next_b, prev_b: the buffers of the keys whose scores follow and of the values that
  // the other half's weights belong to.
  auto half_step = [&](auto half_c, int t, const Known& info, int next_b, int prev_b) {
    constexpr int half = half_c.value;
    const float ev = (float)info.ev;
    const int j0 = t * kTile + 32 * half;
    const uint32_t keys = half ? (uint32_t)(info.keys >> 32) : (uint32_t)info.keys;
    f32x16& s = sc[half];
    constexpr int kMul = 2 * kSteps, kAhead = 6;
    const f16x8* kp = reinterpret_cast<const f16x8*>(s_key[next_b]) + lane + (half ^ 1) * kSteps * 64;
    auto operand = [&](int z) {
      return z & 1 ? value_operand(prev_b, half ^ 1, (z >> 1) % kBlocks, (z >> 1) / kBlocks) : kp[(z >> 1) * 64];
    };
    f16x8 a[kMul];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) a[z] = operand(z);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15");  // max3_hw is no instruction that the compiler waits for a matrix product before
    float f = fmaxf(__builtin_ldexpf(scale, info.ek - kTopBit), 0x1p-100f);
    // of the lane's keys 8 i + 4 g + e, element 4 i + e
    auto own_of = [&](int side, int v) { return (int)s_info[t & (kInfos - 1)].own[side][32 * half + 8 * (v >> 2) + 4 * g + (v & 3)]; };
    if (info.apart) {  // rare: the scores to the tile's units, the values' exponents beside them
      const float inv = 1.0f / f;
#pragma unroll
      for (int v = 0; v < 16; ++v)
        s[v] = fmaf((float)(own_of(1, v) - info.ev), inv, __builtin_ldexpf(s[v], own_of(0, v) - info.ek));
    }
    if (!(j0 >= lo_all && j0 + 32 <= hi_all && keys == ~0u)) {  // some key hidden from some row
      const int from = j0 - context;
      uint32_t mine = 0;  // bit k: the row sees key j0 + k
      if (from > -32) {
        const int word = min((from + 32) >> 5, kTreeWords - 2);
        mine = __builtin_amdgcn_alignbit(seen[word + 1], seen[word], from & 31);
      }
      const int above = min(max(lo - j0, 0), 31), below = min(max(hi - j0, 0), 32);
      if (below > 0 && lo - j0 < 32) mine |= (~0u >> (32 - below)) & (~0u << above);
      mine = (mine & keys) >> (4 * g);
#pragma unroll
      for (int v = 0; v < 16; ++v) s[v] = mine >> (8 * (v >> 2) + (v & 3)) & 1 ? s[v] : -INFINITY;
    }
    float top = -INFINITY, p = 0.0f;
    u32x4 x[2], y[2];
    float part = 0.0f;
    auto weigh = [&](int v, float c) {
      const float e = exp2_hw(fmaf(s[v], f, c));
      if (v & 1) {
        uint32_t pair = pack_f16(p, e);
        asm volatile("" : "+v"(pair));  // here, beside the products, and not on the side of the branch below
        part += p + e;
        if constexpr (FINE) {
          const f16x2 h = __builtin_bit_cast(f16x2, pair);
          y[v >> 3][(v & 7) >> 1] = pack_f16(fmaf((float)h.x, -1.0f, p), fmaf((float)h.y, -1.0f, e));
        }
        x[v >> 3][(v & 7) >> 1] = pair;
      } else {
        p = e;
      }
    };
    auto offset = [&]() { return (ev + kHead) - fmaxf(ref, -0x1p120f); };  // no key yet: -infinity stays
    float c = offset();
    f32x16& z_next = sc[half ^ 1];
#pragma unroll
    for (int v = 0; v < 16; ++v) z_next[v] = 0.0f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int z = 0; z < kMul; ++z) {  // kept in this order
      if (z & 1) {
        const int i = (z >> 1) % kBlocks, ks = (z >> 1) / kBlocks;
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[z], __builtin_bit_cast(f16x8, w[half ^ 1][ks]), acc[i], 0, 0, 0);
        if constexpr (FINE)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[z], __builtin_bit_cast(f16x8, wl[half ^ 1][ks]), acc[i], 0, 0, 0);
      } else {
        z_next = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[z], q[z >> 1], z_next, 0, 0, 0);
      }
      if constexpr (FINE) {
        if (z % 8 == 7) z_next = add_rest(half ^ 1, z / 8, s_rest[next_b], z_next);
      }
      if (z + kAhead < kMul) a[z + kAhead] = operand(z + kAhead);
#pragma unroll
      for (int v = z * 16 / kMul; v < (z + 1) * 16 / kMul; ++v) {
        weigh(v, c);
        if (v & 1) top = max3_hw(top, s[v - 1], s[v]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    top = fmaf(top, f, ev);
    const bool far = __any(fabsf(top) > 0x1p14f && top != -INFINITY);
    if (far || __any(top > ref + kSlack)) {
      // Rare after the first tiles: a larger reference.  The sums so far move to it, and the weights are taken again.
      if (far) {  // scores that are rounded by as much as the slack: once, here, and not again beside the reference
        top = -INFINITY;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          s[v] *= f;
          top = fmaxf(top, s[v]);
        }
        f = 1.0f;
        top += ev;
      }
      const u32x2 o = __builtin_amdgcn_permlane32_swap(f32_bits(top), f32_bits(top), false, false);
      const float up = fmaxf(ref, fmaxf(bits_f32(o.x), bits_f32(o.y)));
      const float down = ref == -INFINITY ? 0.0f : exp2_hw(ref - up);
      sum = lower(sum, ref, up);
      ref = up;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][v] *= down;
      part = 0.0f;
      c = offset();
#pragma unroll
      for (int v = 0; v < 16; ++v) weigh(v, c);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      w[half][ks] = x[ks];
      if constexpr (FINE) wl[half][ks] = y[ks];
    }
    // The denominator, in weights that do not hold the exponent.
    most_ev = max(most_ev, info.ev);
    if (info.apart >> 1 || info.ev < most_ev - 60) {
      float more = 0.0f;
#pragma unroll
      for (int v = 0; v < 16; ++v) more += exp2_hw(fmaf(s[v], f, c) - (float)own_of(1, v));
      sum += more;
    } else {
      sum += __builtin_ldexpf(part, -info.ev);
    }
  };

  if (t_first < t_end) {
    // The decoding waves are a tile ahead: while tile t is multiplied, they decode the keys of tile t + 1 and the values of
    // tile t, and find out what there is to know of tile t + 2.  Loads are an interval ahead of that, in registers that take turns
    // (a copy would wait for them).  Both kinds of wave pass as many barriers.
    if (decodes) {
      learn(t_first, listed0, raw[1].all);
      __syncthreads();
      auto decode = [&](int t, auto set) {
        constexpr int k = set.value;
        const Raw<D, KB, FINE>& x = raw[k];
        const int b = (t - t_first) & 1;
        const float ka = relative(x.own[0], 0, t);
        const float va = t > t_first ? relative(x.own[1], 1, t - 1) : 0.0f;  // the zeros that this makes have no weights
        typename C::Entry ek[C::kPieces][C::kLookups], ev[C::kPieces][C::kLookups];
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) look_up(x.code[0], i, ek[i]);
        if constexpr (KB == 4 && !FINE) {
#pragma unroll
          for (int i = 0; i < C::kPieces; ++i) look_up(x.code[1], i, ev[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool listed2 = listed(id[k]);
        const int64_t row2 = row_of(t + 2, id[k]);
        fetch(raw[k ^ 1], row1, row0);
        fetch_all(raw[k ^ 1], row2);
        id[k ^ 1] = page_of(t + 3);
        learn(t + 1, listed1, x.all);
        row0 = row1;
        row1 = row2;
        listed1 = listed2;
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) finish_key(b, i, ka, ek[i]);
        if constexpr (!(KB == 4 && !FINE)) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < C::kPieces; ++i) look_up(x.code[1], i, ev[i]);
        }
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) put_value(b ^ 1, i, products(va, ev[i], nullptr));
        __syncthreads();
      };
      for (int t = t_first; t <= t_end; t += 2) {
        decode(t, std::integral_constant<int, 0>());
        if (t + 1 <= t_end) decode(t + 1, std::integral_constant<int, 1>());
      }
      return;
    }
    __syncthreads();
    __syncthreads();
    sc[0] = multiply_keys(0, 0);
    for (int t = t_first; t < t_end; ++t) {
      const int b = (t - t_first) & 1;
      const Known info = known(t);
      half_step(std::integral_constant<int, 0>(), t, info, b, b ^ 1);
      __syncthreads();  // the next tile's keys and this one's values are there; their buffers' last tiles are done with
      half_step(std::integral_constant<int, 1>(), t, info, b ^ 1, b);
    }
    // the last half's weights
    const int b = (t_end - 1 - t_first) & 1;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const f16x8 v = value_operand(b, 1, i, ks);
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, __builtin_bit_cast(f16x8, w[1][ks]), acc[i], 0, 0, 0);
        if constexpr (FINE)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, __builtin_bit_cast(f16x8, wl[1][ks]), acc[i], 0, 0, 0);
      }
  }
  if (decodes) return;

  const u32x2 o2 = __builtin_amdgcn_permlane32_swap(f32_bits(sum), f32_bits(sum), false, false);
  const float unit = __builtin_ldexpf(1.0f, -kTopBit);  // of the sums beside those of the weights
  const bool sees = depth >= 0;  // a row that sees nothing went along through the context
  const float l = sees ? bits_f32(o2.x) + bits_f32(o2.y) : 0.0f;
  if (!live) return;
  const int64_t to = (token * aa.heads + head) * nsplit + split;
  const float inv = nsplit > 1 ? unit : (l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l)) * unit;
#pragma unroll
  for (int k = 0; k < kBlocks; ++k)
#pragma unroll
    for (int v = 0; v < 16; v += 4) {
      const int d = 32 * k + 2 * v + 4 * g;
      f32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = sees ? acc[k][v + e] * inv : 0.0f;
      if (nsplit > 1) {
        *reinterpret_cast<f32x4*>(partial + to * D + d) = o;
      } else {
        const u32x2 o16 = {pack16(o[0], o[1], bf16), pack16(o[2], o[3], bf16)};
        *reinterpret_cast<u32x2*>(static_cast<char*>(aa.out) + (token * aa.out_stride + (int64_t)head * D + d) * 2) = o16;
      }
    }
  if (g == 0) {
    const float m = sees ? ref - kHead : -INFINITY;
    if (nsplit > 1) reinterpret_cast<Partial*>(partial + aa.tokens * aa.heads * nsplit * D)[to] = {m, l, l};
    else if (aa.lse != nullptr) aa.lse[token * aa.heads + head] = log_sum(m, l);
  }
}

template <int KB>
hipError_t launch_bits(const KvAttendArgs& a, int grid, int nsplit, int workgroups, bool fine, const DequantArgs& da, hipStream_t s) {
  return launch_kernel(fine ? tree_kernel<128, KB, true> : tree_kernel<128, KB, false>, dim3((unsigned)grid), dim3(kThreads), s, a, da,
                       nsplit, workgroups, static_cast<float*>(a.workspace));
}

}  // namespace

int tree_block_slots() { return cu_count(); }

int launch_tree_blocks(const KvAttendArgs& a, int dtype, int grid, int nsplit, int workgroups, const DequantArgs& da, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return (int)(da.K == 16 ? launch_bits<4>(a, grid, nsplit, workgroups, dtype == F16, da, s)
                          : launch_bits<8>(a, grid, nsplit, workgroups, dtype == F16, da, s));
}

}  // namespace bq
