// k_kv_accept.hip -- keeping the accepted path of a draft in the paged cache: new token path[i] moves to the place of new
// token i, its codes and block maxima as they are.
//
// A wave takes the keys or the values of one head of one sequence, 16 tokens at a time: lane l < 16 finds token l's two
// places, then the wave loads all their bytes before it stores any.  The path ascends, so path[i] >= i, and what a
// later piece reads (places from path[i + 1] on) no earlier one has written (places up to i).  A few KB to a
// sequence: bound by the chain of loads, path to page to codes.  One sequence of 8 heads of 128, 4-bit: 3.9 us; 512 sequences, paths
// of up to 9, 8-bit: 9.0 us.
#include <hip/hip_runtime.h>

#include "bq_attn.h"
#include "bq_launch.h"

namespace bq {
namespace {

constexpr int kPiece = 16;  // tokens
constexpr int kCodeUnits = kPiece * 256 / 16 / 64;  // 16 bytes each, of up to 256 bytes a token and head: per lane
constexpr int kMaxima = kPiece * 8 / 64;            // of up to 8 blocks a token and head: per lane

__global__ __launch_bounds__(64) void kv_accept_kernel(KvAcceptArgs aa) {
  const int lane = threadIdx.x;
  const int kvh = blockIdx.x >> 1, side = blockIdx.x & 1, seq = blockIdx.y;
  KvAttendArgs rows;
  rows.tokens = aa.tokens;
  rows.q_start = aa.q_start;
  rows.kv_len = aa.kv_len;
  rows.max_kv_len = aa.max_kv_len;
  const Sequence sq = sequence(rows, seq);
  const int len = max(min(__builtin_amdgcn_readfirstlane(aa.path_len[seq]), sq.nq), 0);
  const int32_t* const path = aa.path + (int64_t)seq * aa.path_stride;
  const int32_t* const pages = aa.page_table + (int64_t)seq * aa.table_stride;
  const int context = sq.kv - sq.nq, lps = aa.cache.log2_page;
  const uint32_t units = (uint32_t)(aa.cache.head_dim * aa.bits / 8) / 16;
  const uint32_t nb = (uint32_t)aa.cache.head_dim >> aa.cache.log2b;
  u32x4* const codes = reinterpret_cast<u32x4*>(aa.cache.packed[side]);
  float* const maxima = aa.cache.absmax[side];
  // the pool's row (page, head, slot) of key j, or -1
  auto row_of = [&](int j) {
    const int id = j >= 0 && j < sq.kv ? pages[j >> lps] : -1;
    return (uint32_t)id < (uint32_t)aa.cache.num_pages
               ? (((int64_t)id * aa.cache.kv_heads + kvh) << lps) + (j & ((1 << lps) - 1))
               : (int64_t)-1;
  };
  for (int i0 = 0; i0 < len; i0 += kPiece) {
    const int i = i0 + lane;
    const bool mine = lane < kPiece && i < len;
    const int from = mine ? path[i] : -1, before = mine && i > 0 ? path[i - 1] : -1;
    // an entry that does not ascend ends the row
    const uint64_t bad = __ballot(mine && !(from > before && from < sq.nq));
    const int count = bad != 0 ? __builtin_ctzll(bad) : min(len - i0, kPiece);
    const bool moves = lane < count && from != i;
    const int64_t src = moves ? row_of(context + from) : -1, to = moves ? row_of(context + i) : -1;
    u32x4 c[kCodeUnits];
    float a[kMaxima];
    int64_t c_at[kCodeUnits], a_at[kMaxima];
    auto places = [&](uint32_t token, int64_t& s, int64_t& t) {
      s = __shfl(src, (int)token);
      t = __shfl(to, (int)token);
      return token < (uint32_t)count && s >= 0 && t >= 0;
    };
#pragma unroll
    for (int k = 0; k < kCodeUnits; ++k) {
      const uint32_t u = 64 * k + lane, token = u / units, part = u - token * units;
      int64_t s, t;
      const bool ok = places(token & 63, s, t) && token < kPiece;
      c_at[k] = ok ? t * units + part : -1;
      if (ok) c[k] = codes[s * units + part];
    }
#pragma unroll
    for (int k = 0; k < kMaxima; ++k) {
      const uint32_t u = 64 * k + lane, token = u / nb, part = u - token * nb;
      int64_t s, t;
      const bool ok = places(token & 63, s, t) && token < kPiece;
      a_at[k] = ok ? t * nb + part : -1;
      if (ok) a[k] = maxima[s * nb + part];
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every load of the piece has come back
#pragma unroll
    for (int k = 0; k < kCodeUnits; ++k)
      if (c_at[k] >= 0) codes[c_at[k]] = c[k];
#pragma unroll
    for (int k = 0; k < kMaxima; ++k)
      if (a_at[k] >= 0) maxima[a_at[k]] = a[k];
    if (bad != 0) return;
  }
}

}  // namespace

int launch_kv_accept(const KvAcceptArgs& a, void* stream) {
  return (int)launch_kernel(kv_accept_kernel, dim3((unsigned)a.cache.kv_heads * 2, (unsigned)a.num_seqs), dim3(64),
                            static_cast<hipStream_t>(stream), a);
}

}  // namespace bq
