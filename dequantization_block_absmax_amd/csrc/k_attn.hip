// k_attn.hip -- attention of new tokens over a paged key/value cache held in blockwise codes.
//
//   o_i = sum_j p_ij v_j,   p_ij = exp(s_ij) / sum_j exp(s_ij),   s_ij = scale * (q_i . k_j)
// over the keys j that row i sees; k and v are the cached values c[code] * a, one pass over the keys
// with the running maximum and sum of the softmax.
//
// Factored form.  The matrix cores (v_mfma_f32_16x16x32_f16) multiply the codes' table entries,
// rounded once to binary16; the block maxima enter in binary32:
//   s_ij = R_i sum_b a_jb (sum_{d in b} q'_id c_jd)   q' = q 2^-e_i exact in binary16, R_i = scale 2^e_i
//   o_i  = sum_j (p_ij a'_jb) c'_jd                    for d in block b of the values
// so no cached value is formed: a code byte indexes a table in LDS that holds its two binary16
// entries side by side.  Rounded to 16 bits are: c (2^-12 relative), the weights p a' (2^-12 relative
// to the largest of their row), q' where it falls 2^-14 below its row's largest element, and the
// result.  e_i is the exponent of the row's largest |q|.  Weights are kept in range by the reference
//   M_i = max_j (log2-domain s_ij + E_j),   E_j the exponent of token j's largest value maximum,
// in place of the plain running maximum: the weights p a' = 2^(s - M) a' then stay below 2^8 whatever
// the size of the values, and sum and weighted sum carry the same factor, which cancels.
//
// Decomposition.  Work is split over (16 RT rows: new token x query head of one key/value head) x
// (key/value head) x (sequence) x (splits of the keys).  A workgroup's four waves take groups of 32
// keys in turn, each on its own, and join their sums through LDS at the end; with more than one split
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
#include <hip/hip_runtime.h>

#include "bq_attn.h"
#include "bq_internal.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kWaves = 4;
constexpr int kGroup = 32;        // keys per wave and step
constexpr int kCopies = 32;       // copies of the LDS table, one per bank: no lookup waits for another
constexpr float kSlack = 6.0f;    // weights may grow by 2^6 before the sums are rescaled

template <int D, int NB, int KB>
struct Shape {
  static constexpr int kRow = D * KB / 8;       // bytes of a key's codes
  static constexpr int kLane = kRow / 16;       // bytes of a value's codes per lane: 2, 4, 8 or 16
  static constexpr int kWords = kLane < 4 ? 1 : kLane / 4;
  static constexpr int kSteps = D / 32;         // products of 32 d
  static constexpr int kTiles = D / 16;         // tiles of 16 d of the result
  static constexpr int kPerLane = D / 16;       // d's per lane
  static constexpr int kPerBlock = kPerLane / NB;
};

// One group of 32 keys as a lane loads it.
template <int D, int NB, int KB>
struct Group {
  using S = Shape<D, NB, KB>;
  uint32_t k[2][S::kSteps][KB == 4 ? 1 : 2];
  uint32_t v[8][S::kWords];
  float ka[2][4][NB], va[2][4][NB];
};

// Where the pages of a group of 32 keys lie; a page outside the pool reads page 0 and hides its keys.
struct Pages {
  int id[2];
};

template <int KB>
__device__ __forceinline__ uint32_t table_at(const char* lut, uint32_t byte_times_128, uint32_t lane4) {
  return *reinterpret_cast<const uint32_t*>(lut + (byte_times_128 | lane4));
}

// Table entry of byte b of a word: 4-bit codes, the binary16 pair (low nibble, high nibble); 8-bit codes, the
// binary16 entry in the low half.
template <int KB>
__device__ __forceinline__ uint32_t lookup(const char* lut, uint32_t w, int b, uint32_t lane4) {
  const uint32_t at = b == 0 ? w << 7 : w >> (8 * b - 7);
  return table_at<KB>(lut, at & 0x7f80u, lane4);
}

// Two 8-bit codes' entries as a pair.
__device__ __forceinline__ uint32_t join(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x05040100u); }

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
  } else
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, DPP, 0xF, 0xF, false);
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

template <int D, int NB, int KB, int RT>
__global__ __launch_bounds__(64 * kWaves, RT* D > 128 ? 1 : 2) void attend_kernel(KvAttendArgs aa, DequantArgs da,
                                                                                   int nsplit, int bf16) {
  using S = Shape<D, NB, KB>;
  constexpr int kRows = 16 * RT;
  constexpr int kPitch = D + 4;  // of a row of partial sums in LDS
  constexpr int kLut = 256 * kCopies * 4, kSums = kWaves * 16 * kPitch * 4;
  __shared__ __attribute__((aligned(16))) char s_mem[kLut > kSums ? kLut : kSums];
  __shared__ Partial s_part[kWaves][kRows];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int split = blockIdx.x;
  const int kvh = blockIdx.y % aa.cache.kv_heads, tile = blockIdx.y / aa.cache.kv_heads;
  const int seq = blockIdx.z;
  const int group = aa.heads / aa.cache.kv_heads;
  const Sequence sq = sequence(aa, seq);
  const int nrows = min(sq.nq, aa.max_q_len) * group;  // rows of the sequence for this key/value head
  if (tile * kRows >= nrows) return;

  // Table: entry b in copy c at (b * kCopies + c) * 4; a lane reads copy lane % 32.
  {
    const float lo = da.c[KB == 4 ? tid & 15 : tid], hi = da.c[KB == 4 ? tid >> 4 : tid];
    const uint32_t e = pack_f16(lo, hi);
    const u32x4 e4 = {e, e, e, e};
#pragma unroll
    for (int i = 0; i < kCopies / 4; ++i)  // in turn over the banks
      *reinterpret_cast<u32x4*>(s_mem + tid * (kCopies * 4) + ((i + tid) & (kCopies / 4 - 1)) * 16) = e4;
  }
  const uint32_t lane4 = (lane & (kCopies - 1)) * 4;

  // Rows of this lane (column m of the products), their keys and queries.
  int lo[RT], hi[RT];
  float scale[RT];
  f16x8 q[RT][S::kSteps];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = tile * kRows + t * 16 + m;
    const bool live = r < nrows;
    const int i = live ? r / group : 0;
    const int head = kvh * group + (live ? r - i * group : 0);
    lo[t] = live ? first_key(aa, sq, i) : 0;
    hi[t] = live ? end_key(aa, sq, i) : 0;
    const char* src = static_cast<const char*>(aa.q) + ((int64_t)(sq.q0 + i) * aa.q_stride + (int64_t)head * D) * 2;
    float x[S::kSteps][8];
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(src + (32 * s + 8 * g) * 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
        x[s][e] = bf16 ? bits_f32(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
        top = max(top, f32_bits(x[s][e]) & 0x7fffffffu);
      }
    }
    const float tf = rows_max(bits_f32(top < 0x7f800000u ? top : 0u));
    const int ex = tf > 0.0f ? __builtin_amdgcn_frexp_expf(tf) : 0;  // |q| < 2^ex
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __builtin_ldexpf(x[s][2 * k], -ex), b = __builtin_ldexpf(x[s][2 * k + 1], -ex);
        // 4-bit codes: the first element of a byte is its high nibble, the high half of the table's pair
        w[k] = KB == 4 ? pack_f16(b, a) : pack_f16(a, b);
      }
      q[t][s] = __builtin_bit_cast(f16x8, w);
    }
    scale[t] = __builtin_ldexpf(aa.scale * 1.44269504088896341f, ex);
  }

  // Keys of the tile's rows together, this split's groups of 32 of them, and this wave's.
  const int last_row = min(tile * kRows + kRows, nrows) - 1;
  const int i_first = tile * kRows / group, i_last = last_row / group;
  const int begin = first_key(aa, sq, i_first) & ~(kGroup - 1);
  const int end = end_key(aa, sq, i_last);
  const int lo_all = first_key(aa, sq, i_last), hi_all = end_key(aa, sq, i_first);  // seen by every row
  const int groups = end > begin ? (end - begin + kGroup - 1) / kGroup : 0;
  const int per = (groups + nsplit - 1) / nsplit;
  const int g_end = min((split + 1) * per, groups);

  const int lps = aa.cache.log2_page;
  // read through scalar loads: the numbers are the same for the whole wave, and waiting for them
  // does not wait for the cache's vector loads before them
  typedef const __attribute__((address_space(4))) int32_t* ScalarTable;
  const ScalarTable pages = (ScalarTable)(uintptr_t)(aa.page_table + (int64_t)seq * aa.table_stride);
  const int last_page = sq.kv > 0 ? (sq.kv - 1) >> lps : 0;
  auto find = [&](int gi) {
    Pages p;
#pragma unroll
    for (int u = 0; u < 2; ++u) p.id[u] = pages[min((begin + gi * kGroup + 16 * u) >> lps, last_page)];
    return p;
  };
  const uint32_t k_at = m * S::kRow + g * (KB == 4 ? 4 : 8);
  const uint32_t v_at = 4 * g * S::kRow + m * S::kLane;
  const uint32_t a_at = 4 * g * NB * 4;
  auto load = [&](int gi, const Pages& p, Group<D, NB, KB>& x) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = begin + gi * kGroup + 16 * u;
      const uint32_t id = (uint32_t)p.id[u] < (uint32_t)aa.cache.num_pages ? p.id[u] : 0;
      const int64_t row = (((int64_t)id * aa.cache.kv_heads + kvh) << lps) + (j & ((1 << lps) - 1));
      const uint8_t* kp = aa.cache.packed[0] + row * S::kRow;
      const uint8_t* vp = aa.cache.packed[1] + row * S::kRow;
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
        if constexpr (KB == 4) {
          x.k[u][s][0] = *reinterpret_cast<const uint32_t*>(kp + k_at + 16 * s);
        } else {
          const u32x2 w = *reinterpret_cast<const u32x2*>(kp + k_at + 32 * s);
          x.k[u][s][0] = w.x;
          x.k[u][s][1] = w.y;
        }
      }
      const float* kap = aa.cache.absmax[0] + row * NB;
      const float* vap = aa.cache.absmax[1] + row * NB;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const f32x4 ka = *reinterpret_cast<const f32x4*>(reinterpret_cast<const char*>(kap) + a_at + 16 * i);
        const f32x4 va = *reinterpret_cast<const f32x4*>(reinterpret_cast<const char*>(vap) + a_at + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x.ka[u][(4 * i + e) / NB][(4 * i + e) % NB] = ka[e];
          x.va[u][(4 * i + e) / NB][(4 * i + e) % NB] = va[e];
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t* src = vp + v_at + r * S::kRow;
        uint32_t* w = x.v[4 * u + r];
        if constexpr (S::kLane == 2) {
          w[0] = *reinterpret_cast<const uint16_t*>(src);
        } else if constexpr (S::kLane == 4) {
          w[0] = *reinterpret_cast<const uint32_t*>(src);
        } else if constexpr (S::kLane == 8) {
          const u32x2 t = *reinterpret_cast<const u32x2*>(src);
          w[0] = t.x;
          w[1] = t.y;
        } else {
          const u32x4 t = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = t[e];
        }
      }
    }
  };

  const Spread<D, NB, KB> spread(m);
  float ref[RT], safe[RT], sum[RT];  // reference M, M where it is finite, sum of weights (this lane's keys)
  f32x4 acc[RT][S::kTiles];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    ref[t] = -INFINITY;
    safe[t] = sum[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < S::kTiles; ++i) acc[t][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto step = [&](int gi, const Pages& p, Group<D, NB, KB>& x) {
    const int j0 = begin + gi * kGroup;
    // scores, in the log2 domain
    float s[RT][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 z[RT];
#pragma unroll
      for (int k = 0; k < S::kSteps; ++k) {
        u32x4 w;
        if constexpr (KB == 4) {
#pragma unroll
          for (int b = 0; b < 4; ++b) w[b] = lookup<4>(s_mem, x.k[u][k][0], b, lane4);
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            w[b] = join(lookup<8>(s_mem, x.k[u][k][b >> 1], 2 * (b & 1), lane4),
                        lookup<8>(s_mem, x.k[u][k][b >> 1], 2 * (b & 1) + 1, lane4));
        }
        const f16x8 a = __builtin_bit_cast(f16x8, w);
        constexpr int per_block = S::kSteps / NB;
        const int b = k / per_block;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (k % per_block == 0) z[t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
          z[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[t][k], z[t], 0, 0, 0);
          if (k % per_block == per_block - 1) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              s[t][u][r] = b == 0 ? z[t][r] * x.ka[u][r][b] : fmaf(z[t][r], x.ka[u][r][b], s[t][u][r]);
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
    // exponents of the tokens' largest value maximum (between 2^-100 and 2^100; zero counts as 2^-100)
    float ev[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float a = fabsf(x.va[u][r][0]);
#pragma unroll
        for (int b = 1; b < NB; ++b) a = fmaxf(a, fabsf(x.va[u][r][b]));
        ev[u][r] = (float)__builtin_amdgcn_frexp_expf(fminf(fmaxf(a, 0x1p-100f), 0x1p100f));
      }
    const bool listed0 = (uint32_t)p.id[0] < (uint32_t)aa.cache.num_pages;
    const bool listed1 = (uint32_t)p.id[1] < (uint32_t)aa.cache.num_pages;
    const bool masked = !(j0 >= lo_all && j0 + kGroup <= hi_all && listed0 && listed1);  // uniform
    uint32_t w[RT][NB][4];  // weights of the lane's 8 keys
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      uint32_t hide = 0;
      if (masked) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = j0 + 16 * u + 4 * g + r;
            const bool out = j < lo[t] || j >= hi[t] || !(u == 0 ? listed0 : listed1);
            hide |= out ? 1u << (4 * u + r) : 0u;
            if (out) s[t][u][r] = 0.0f;
          }
      }
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = s[t][u][r] + ev[u][r];
          top = fmaxf(top, masked && (hide >> (4 * u + r) & 1) ? -INFINITY : v);
        }
      if (__any(top > ref[t] + kSlack)) {  // rare after the first groups: raise the reference
        const float up = fmaxf(ref[t], rows_max(top));
        const float f = ref[t] == -INFINITY ? 0.0f : exp2_hw(ref[t] - up);
        ref[t] = up;
        safe[t] = up == -INFINITY ? 0.0f : up;
        sum[t] *= f;
#pragma unroll
        for (int i = 0; i < S::kTiles; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][i][r] *= f;
      }
      float pw[NB][8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int e = 4 * u + r;
          const bool out = masked && (hide >> e & 1);
          const float p2 = out ? 0.0f : exp2_hw(s[t][u][r] - safe[t]);
          sum[t] += p2;
#pragma unroll
          for (int b = 0; b < NB; ++b) pw[b][e] = out ? 0.0f : p2 * x.va[u][r][b];
        }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) w[t][b][k] = pack_f16(pw[b][2 * k], pw[b][2 * k + 1]);
    }
    // sums of values
#pragma unroll
    for (int e = 0; e < 8; ++e) spread.apply(x.v[e]);
#pragma unroll
    for (int wd = 0; wd < S::kWords; ++wd) {
      uint32_t pair[4][2];  // 4-bit: both keys' codes of a pair in one byte (even and odd d's)
      if constexpr (KB == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x0 = x.v[2 * k][wd], x1 = x.v[2 * k + 1][wd];
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
          u32x4 a;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (KB == 4) a[k] = lookup<4>(s_mem, pair[k][h], by, lane4);
            else
              a[k] = join(lookup<8>(s_mem, x.v[2 * k][wd], by, lane4), lookup<8>(s_mem, x.v[2 * k + 1][wd], by, lane4));
          }
          const int i = (4 * wd + by) * kPer + h;  // tile: place i of the lane's d's
          const int b = i / S::kPerBlock;
#pragma unroll
          for (int t = 0; t < RT; ++t)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                __builtin_bit_cast(f16x8, a),
                __builtin_bit_cast(f16x8, (u32x4){w[t][b][0], w[t][b][1], w[t][b][2], w[t][b][3]}), acc[t][i], 0, 0, 0);
        }
    }
  };

  __syncthreads();  // the table is in place
  // Groups wave, wave + 4, ... of the split: the next group's loads, and the page numbers of the one
  // after it, are issued before the current group is worked on.
  int gi = split * per + wave;
  if (gi < g_end) {
    Group<D, NB, KB> x0, x1;
    Pages p0 = find(gi), p1 = find(min(gi + kWaves, groups - 1));
    load(gi, p0, x0);
    for (;;) {
      const Pages p2 = find(min(gi + 2 * kWaves, groups - 1));
      load(min(gi + kWaves, groups - 1), p1, x1);
      step(gi, p0, x0);
      gi += kWaves;
      if (gi >= g_end) break;
      const Pages p3 = find(min(gi + 2 * kWaves, groups - 1));
      load(min(gi + kWaves, groups - 1), p2, x0);
      step(gi, p1, x1);
      gi += kWaves;
      if (gi >= g_end) break;
      p0 = p2;
      p1 = p3;
    }
  }

  // Join the waves: common reference, then their scaled sums in wave order.
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    sum[t] = rows_sum(sum[t]);
    if (g == 0) s_part[wave][t * 16 + m] = {ref[t], sum[t]};
  }
  __syncthreads();  // also: every lookup is done, the table's memory is free
  float* s_sum = reinterpret_cast<float*>(s_mem);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_part[w][t * 16 + m].m);
    const float f = ref[t] == -INFINITY ? 0.0f : exp2_hw(ref[t] - top);
#pragma unroll
    for (int i = 0; i < S::kTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = Spread<D, NB, KB>::d_of(4 * g + r, i / S::kPerBlock, i % S::kPerBlock);
        s_sum[(wave * 16 + m) * kPitch + d] = acc[t][i][r] * f;
      }
    __syncthreads();
    // 16 threads to a row, each some groups of 4 d
    const int row = tid >> 4;
    const int r = tile * kRows + t * 16 + row;
    if (r < nrows) {
      const int i = r / group, head = kvh * group + (r - i * group);
      const int64_t token = sq.q0 + i;
      float m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m_all = fmaxf(m_all, s_part[w][t * 16 + row].m);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const Partial p = s_part[w][t * 16 + row];
        l_all += p.m == -INFINITY ? 0.0f : p.l * exp2_hw(p.m - m_all);
      }
      const float inv = l_all > 0.0f ? 1.0f / l_all : (l_all == 0.0f ? 0.0f : l_all);
      const int64_t part = ((token * aa.heads + head) * nsplit + split);
      float* wsum = static_cast<float*>(aa.workspace) + part * D;
      Partial* wpart = reinterpret_cast<Partial*>(static_cast<float*>(aa.workspace) + aa.tokens * aa.heads * nsplit * D) + part;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int d = (tid & 15) * 4 + 64 * c;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(&s_sum[(w * 16 + row) * kPitch + d]);
        if (nsplit == 1) {
          const u32x2 o = {pack16(v[0] * inv, v[1] * inv, bf16), pack16(v[2] * inv, v[3] * inv, bf16)};
          *reinterpret_cast<u32x2*>(static_cast<char*>(aa.out) + (token * aa.out_stride + (int64_t)head * D + d) * 2) = o;
        } else {
          *reinterpret_cast<f32x4*>(wsum + d) = v;
        }
      }
      if ((tid & 15) == 0) {
        if (nsplit > 1) *wpart = {m_all, l_all};
        else if (aa.lse != nullptr) aa.lse[token * aa.heads + head] = log_sum(m_all, l_all);
      }
    }
    __syncthreads();
  }
}

}  // namespace

// Rows per tile and splits of the keys, by what the call's shape bounds.
struct Plan {
  int rt, tiles, nsplit;
};

static Plan make_plan(const KvAttendArgs& a) {
  Plan p;
  const int64_t rows = (int64_t)a.max_q_len * (a.heads / a.cache.kv_heads);
  p.rt = rows > 16 ? 2 : 1;
  p.tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
  const int64_t base = (int64_t)p.tiles * a.cache.kv_heads * a.num_seqs;
  const int64_t cus = cu_count();
  auto splits = [&](int64_t target, int64_t keys) {
    const int64_t most = ((int64_t)a.max_kv_len + keys - 1) / keys;
    int64_t n = (target + base - 1) / base;
    n = n < most ? n : most;
    return n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n;
  };
  int64_t n = splits(8 * cus, 256);
  if (n * base < 2 * cus) n = splits(2 * cus, 128);
  p.nsplit = (int)n;
  return p;
}

size_t kv_attend_workspace(const KvAttendArgs& a, int) {
  const Plan p = make_plan(a);
  if (p.nsplit == 1) return 0;
  return (size_t)a.tokens * a.heads * p.nsplit * (a.cache.head_dim + 2) * 4;
}

namespace {

template <int D, int NB, int KB, int RT>
hipError_t launch_rows(const KvAttendArgs& a, const Plan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  const dim3 grid((unsigned)p.nsplit, (unsigned)(p.tiles * a.cache.kv_heads), (unsigned)a.num_seqs);
  return launch_kernel(attend_kernel<D, NB, KB, RT>, grid, dim3(64 * kWaves), s, a, da, p.nsplit, dtype == BF16);
}

template <int D, int NB>
hipError_t launch_blocks(const KvAttendArgs& a, const Plan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  if (da.K == 16)
    return p.rt == 1 ? launch_rows<D, NB, 4, 1>(a, p, dtype, da, s) : launch_rows<D, NB, 4, 2>(a, p, dtype, da, s);
  return p.rt == 1 ? launch_rows<D, NB, 8, 1>(a, p, dtype, da, s) : launch_rows<D, NB, 8, 2>(a, p, dtype, da, s);
}

}  // namespace

int launch_kv_attend(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Plan p = make_plan(a);
  if ((int64_t)p.tiles * a.cache.kv_heads > 65535) {  // grid rows
    g_launch_refused_for_size = true;
    return (int)hipErrorInvalidConfiguration;
  }
  const int nb = a.cache.head_dim >> a.cache.log2b;
  hipError_t e;
  if (a.cache.head_dim == 64) {
    e = nb == 1 ? launch_blocks<64, 1>(a, p, dtype, da, s) : launch_blocks<64, 2>(a, p, dtype, da, s);
  } else if (a.cache.head_dim == 128) {
    e = nb == 1   ? launch_blocks<128, 1>(a, p, dtype, da, s)
        : nb == 2 ? launch_blocks<128, 2>(a, p, dtype, da, s)
                  : launch_blocks<128, 4>(a, p, dtype, da, s);
  } else {
    e = nb == 1   ? launch_blocks<256, 1>(a, p, dtype, da, s)
        : nb == 2 ? launch_blocks<256, 2>(a, p, dtype, da, s)
        : nb == 4 ? launch_blocks<256, 4>(a, p, dtype, da, s)
                  : launch_blocks<256, 8>(a, p, dtype, da, s);
  }
  if (e != hipSuccess || p.nsplit == 1) return (int)e;
  return launch_kv_merge(a, dtype, p.nsplit, stream);
}

}  // namespace bq
