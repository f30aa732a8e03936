// k_attn.hip -- attention of new tokens over the cache: how a call is divided among the kernels of bq_attend.h (few rows
// to a key/value head) and k_attn_chunk.hip (many), and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bq_attend.h"
#include "bq_launch.h"

namespace bq {

// How a call is done: tiles of 16 rt rows and splits of the keys for the splitting kernel, for every
// sequence or for those with few rows, and the plan of the chunk kernels where some may have many.
struct Plan {
  bool few, many;
  int rt, tiles, nsplit;
  size_t partial_at, bytes;
  ChunkPlan chunk;
};

// The expanded keys and values may take this much of the workspace (with q in binary16 3/16 of it more, for the
// rests); a call that would need more is left to the splitting kernel.  Room is kept for every sequence at the
// longest length, as their row counts are known on the device only: 2048 tokens beside 63 single ones, 32 heads over 8 of 128,
// bf16, take 2.1 GiB and 0.60 ms over 8192 keys each, 4.3 GiB and 1.2 ms over 16384, and over 32768, left to the
// splitting kernel, 7.4 ms.
constexpr int64_t kMaxExpanded = (int64_t)4 << 30;

// Splits of the keys: those whose rounds of resident workgroups (`slots`; `base` without splits) take the least
// time, a workgroup costing its steps of 256 keys and about 3 more (24 windows of 4000 keys, 5 heads: 4 splits
// 24.4 us, 8 splits 30.0; 64 sequences of up to 8192 keys, 8 heads: 1 split 90.3, 2 splits and their join
// 89.3, 4 splits 92.5).  With several sequences, whose lengths may differ, a workgroup takes 8192 keys at most.
static int64_t choose_splits(int64_t base, int64_t slots, int64_t keys, int num_seqs) {
  const int64_t steps = (keys + 255) / 256;
  const int64_t least = num_seqs > 1 ? std::max((steps + 31) / 32, (int64_t)1) : 1;  // one without any keys
  int64_t best = INT64_MAX, n = 1;
  for (int64_t k = least < kMaxSplits ? least : kMaxSplits; k <= kMaxSplits && (k <= steps || k <= 1); ++k) {
    const int64_t cost = (base * k + slots - 1) / slots * ((steps + k - 1) / k + 3);
    if (cost < best) {
      best = cost;
      n = k;
    }
  }
  return n;
}

// Rows of a key/value head (new tokens x its query heads) up to which the splitting kernel alone is the
// faster way, codes decoded anew for every 32 rows against an expanded copy written and read (us, 8 sequences of
// 8192 keys, 4 heads, this kernel / the expanding ones):
//   bf16, 128 wide, 4-bit: 256 rows 75 / 91, 384 121 / 111; 64 wide: 256 50 / 63, 384 74 / 74
//   f16 (operands in two parts), 128 wide, 4-bit: 192 107 / 125, 256 121 / 117, 384 189 / 152, one sequence of 16000
//   keys 256 39 / 44, 384 53 / 55; 64 wide: 256 72 / 76, 384 105 / 95
//   256 wide (16 rows to a workgroup), 8-bit, bf16: 96 118 / 169, 128 166 / 148, one sequence of 16000 keys 43 / 57;
//   f16: 128 184 / 203, 256 341 / 261
static int64_t most_few_rows(int64_t head_dim, int dtype) { return head_dim == 256 ? 128 : dtype == F16 ? 256 : 384; }

static Plan make_plan(const KvAttendArgs& a, int dtype) {
  Plan p = {};
  const int64_t group = a.heads / a.cache.kv_heads, D = a.cache.head_dim, cus = cu_count();
  int64_t rows = a.max_q_len * group;
  const int64_t ntiles = ((int64_t)a.max_kv_len + 63) / 64;
  const int64_t heads_all = (int64_t)a.cache.kv_heads * a.num_seqs, rest = chunk_rest_bytes(a.cache.head_dim, dtype);
  const int64_t per_tile = heads_all * 64 * D * 4;  // at most 2^52
  p.many = rows > most_few_rows(D, dtype) && ntiles > 0 && ntiles <= kMaxExpanded / per_tile;
  p.few = !p.many || a.num_seqs > 1;
  if (p.many) {
    ChunkPlan& c = p.chunk;
    c.ntiles = (int)ntiles;
    c.blocks = (int)((rows + kChunkRows - 1) / kChunkRows);
    // Workgroups without splits: the rows there are, whatever their sequences.  Of the numbers of splits,
    // the one whose rounds of resident workgroups take the least time, a workgroup costing its tiles and
    // about 6 more (start, end, and its part of the join).
    const int64_t base = a.cache.kv_heads * ((a.tokens * group + kChunkRows - 1) / kChunkRows);
    const int64_t slots = chunk_slots(a.cache.head_dim, dtype);
    int64_t best = INT64_MAX;
    c.nsplit = 1;
    for (int64_t n = 1; n <= 32 && (n == 1 || n * 4 <= ntiles); ++n) {
      const int64_t cost = (base * n + slots - 1) / slots * ((ntiles + n - 1) / n + 6);
      if (cost < best) {
        best = cost;
        c.nsplit = (int)n;
      }
    }
    const size_t tiles = (size_t)(ntiles * heads_all);
    c.rest_at = tiles * 64 * D * 4;
    c.info_at = c.rest_at + tiles * rest;
    c.exponents_at = c.info_at + tiles * kTileInfoBytes;
    c.partial_at = (c.exponents_at + tiles * 2 * 64 + 255) & ~(size_t)255;
    c.end = c.partial_at + (c.nsplit > 1 ? (size_t)a.tokens * a.heads * c.nsplit * (D + 3) * 4 : 0);
    p.partial_at = (c.end + 255) & ~(size_t)255;
    rows = kFewRows;  // the splitting kernel's sequences
  }
  p.bytes = p.partial_at;
  if (!p.few) return p;
  p.rt = rows > 16 && D <= 128 ? 2 : 1;
  p.tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
  // tiles with rows in them: sequences may bring fewer tokens than the longest
  const int64_t rows_all = a.tokens * group / (16 * p.rt) + a.num_seqs;
  const int64_t base = a.cache.kv_heads * std::min((int64_t)p.tiles * a.num_seqs, rows_all);
  const int nb = a.cache.head_dim >> a.cache.log2b;
  const int64_t slots = cus * (D == 256 || nb == 4 || (p.rt == 2 && D == 128) || wide_form((int)D, nb, a.bits, p.rt) ? 1 : 2);
  // the workspace is asked for without a window, and holds for any
  int64_t n = choose_splits(base, slots, a.max_kv_len, a.num_seqs);
  if (a.window > 0 && (int64_t)a.window + a.max_q_len < a.max_kv_len) {
    const int64_t k = choose_splits(base, slots, (int64_t)a.window + a.max_q_len, a.num_seqs);
    n = k < n ? k : n;
  }
  p.nsplit = (int)n;
  if (n > 1) p.bytes += (size_t)a.tokens * a.heads * n * (D + 3) * 4;
  return p;
}

size_t kv_attend_workspace(const KvAttendArgs& a, int dtype) { return make_plan(a, dtype).bytes; }

namespace {

template <int D, int NB, int KB, int RT, bool HL>
hipError_t launch_type(const KvAttendArgs& a, const Plan& p, const DequantArgs& da, hipStream_t s) {
  const dim3 grid((unsigned)(p.tiles * p.nsplit), (unsigned)a.cache.kv_heads, (unsigned)a.num_seqs);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + p.partial_at);
  return launch_kernel(attend_kernel<D, NB, KB, RT, HL, false>, grid, dim3(64 * Occupancy<D, NB, KB, RT>::kWaves), s, a, da, p.nsplit,
                       partial, p.many ? kFewOnly : kAllRows);
}

template <int D, int NB, int KB, int RT>
hipError_t launch_rows(const KvAttendArgs& a, const Plan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  return dtype == F16 ? launch_type<D, NB, KB, RT, true>(a, p, da, s) : launch_type<D, NB, KB, RT, false>(a, p, da, s);
}

template <int D, int NB>
hipError_t launch_blocks(const KvAttendArgs& a, const Plan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  if constexpr (D <= 128) {
    if (p.rt == 2) return da.K == 16 ? launch_rows<D, NB, 4, 2>(a, p, dtype, da, s) : launch_rows<D, NB, 8, 2>(a, p, dtype, da, s);
  }
  return da.K == 16 ? launch_rows<D, NB, 4, 1>(a, p, dtype, da, s) : launch_rows<D, NB, 8, 1>(a, p, dtype, da, s);
}

hipError_t launch_few(const KvAttendArgs& a, const Plan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  const int nb = a.cache.head_dim >> a.cache.log2b;
  if (a.cache.head_dim == 64)
    return nb == 1 ? launch_blocks<64, 1>(a, p, dtype, da, s) : launch_blocks<64, 2>(a, p, dtype, da, s);
  if (a.cache.head_dim == 128)
    return nb == 1   ? launch_blocks<128, 1>(a, p, dtype, da, s)
           : nb == 2 ? launch_blocks<128, 2>(a, p, dtype, da, s)
                     : launch_blocks<128, 4>(a, p, dtype, da, s);
  return nb == 1   ? launch_blocks<256, 1>(a, p, dtype, da, s)
         : nb == 2 ? launch_blocks<256, 2>(a, p, dtype, da, s)
         : nb == 4 ? launch_blocks<256, 4>(a, p, dtype, da, s)
                   : launch_blocks<256, 8>(a, p, dtype, da, s);
}

}  // namespace

int launch_kv_attend(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream) {
  const Plan p = make_plan(a, dtype);
  // Every launch fits before the first is enqueued: threads along x in 32 bits, grid rows in 16.
  const bool join = (p.few && p.nsplit > 1) || (p.many && p.chunk.nsplit > 1);
  const int few_threads = 64 * (a.cache.head_dim == 256 && a.cache.log2b == 5 ? Occupancy<256, 8, 4, 1>::kWaves : 8);
  if ((p.few && (int64_t)p.tiles * p.nsplit * few_threads > UINT32_MAX) || a.cache.kv_heads > 32767 ||
      (p.many && (int64_t)a.cache.kv_heads * p.chunk.nsplit * p.chunk.blocks > UINT32_MAX / 256) ||
      (p.many && p.chunk.ntiles > (int64_t)UINT32_MAX / 256) || (join && !kv_merge_fits(a))) {
    g_launch_refused_for_size = true;
    return (int)hipErrorInvalidConfiguration;
  }
  char* const ws = static_cast<char*>(a.workspace);
  const MergeArgs m = {{reinterpret_cast<float*>(ws + p.partial_at), reinterpret_cast<float*>(ws + p.chunk.partial_at)},
                       {p.few ? p.nsplit : 0, p.many ? p.chunk.nsplit : 0},
                       p.few && p.many,
                       p.many};
  int e = p.many ? launch_kv_chunk(a, dtype, p.chunk, da, stream) : 0;
  if (e == 0 && p.few) e = (int)launch_few(a, p, dtype, da, static_cast<hipStream_t>(stream));
  if (e != 0 || !join) return e;
  return launch_kv_merge(a, dtype, m, stream);
}

}  // namespace bq
