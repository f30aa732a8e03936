// k_tree_few.hip -- attention of a tree of drafted tokens over the cache: how a call is divided, and the launches for drafts with
// few rows to a key/value head (the kernel of bq_attend.h).
//
// That kernel's figures for trees, on MI355X: one draft of 26 tokens over 1026 keys, 32 heads over 8 of 128, 4-bit, B = 64, bf16:
// 12.4 us and join 3.9, the chain of loads from the arguments to the keys and two launches; 20 of up to 13 over a window of
// 4000, 20 over 5 of 64, 8-bit, B = 32, f16: 47 us and join 5.6, 1.0 TB/s: 16 rows are decoded for at a time, vector units;
// 5 of up to 21 over up to 6000, 8 over 1 of 256, 8-bit, B = 128, bf16: 28 us and join 5.6, 88 TFLOP/s: 11 row tiles decode the same keys.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bq_attend.h"
#include "bq_launch.h"

namespace bq {
namespace {

struct TreePlan {
  bool blocks;      // k_tree.hip
  int rt, tiles, nsplit;
  int64_t workgroups, grid;
  size_t bytes;
};

// Splits of the keys: those whose rounds of resident workgroups (`slots`; `base` without splits) take the least time, a
// workgroup costing its steps of 256 keys and about 3 more.  With several sequences, whose lengths may differ, a workgroup
// takes 8192 keys at most.
int64_t choose_splits(int64_t base, int64_t slots, int64_t keys, int num_seqs) {
  const int64_t steps = (keys + 255) / 256;
  const int64_t least = num_seqs > 1 ? std::max((steps + 31) / 32, (int64_t)1) : 1;
  int64_t best = INT64_MAX, n = 1;
  for (int64_t k = std::min(least, (int64_t)kMaxSplits); k <= kMaxSplits && (k <= steps || k <= 1); ++k) {
    const int64_t cost = (base * k + slots - 1) / slots * ((steps + k - 1) / k + 3);
    if (cost < best) {
      best = cost;
      n = k;
    }
  }
  return n;
}

// Splits for parts that are found on the device, of at least `least` units of keys: those of the longest sequence if all are as
// long and parts half as long as they can be, and room for as many more where the others are shorter.
int64_t most_splits(int64_t base, int64_t workgroups, int64_t units, int64_t least, int num_seqs) {
  const int64_t per = std::max((base * units + 2 * workgroups - 1) / (2 * workgroups), least);
  int64_t n = (units + per - 1) / per;
  if (num_seqs > 1) n = std::min(2 * n, (units + least - 1) / least);
  return std::max(std::min(n, (int64_t)kMaxSplits), (int64_t)1);
}

// Whether the kernel for many rows takes the call: it decodes a tile of keys once for 128 rows where the other does for 32, but
// begins more slowly and with longer pieces, and rounds more in binary16.  `keys`: the longest sequence's that a row can see; never true
// for fewer keys than it is false for (the workspace is asked for without a window).  It has to be a large call (`work`: tiles of 32 rows x
// keys).  Where its blocks of 128 rows leave compute units over, the keys of each are split further and its longer pieces show, all the
// more where the other kernel just fills the device; the other's lookups are dearer for 8-bit codes and for binary16, whose
// entries have two parts.  In us, the other kernel / that of k_tree.hip, 32 heads over 8, bfloat16 and 4-bit codes if not said otherwise, drafts of
// equal length on 256 compute units:
//   one sequence       64 tokens over 16384 keys 46 / 49, over 32768 77 / 70; 256 over 4096 42 / 50, over 16384 133 / 118
//   49 to 64 blocks    4 of 64 over 2048 28 / 39, over 4096 42 / 53, over 8192 73 / 76, over 16384 143 / 122; 8 of 32 over 2048 28 / 38;
//                      binary16 4 of 64 over 2048 37 / 43, over 4096 63 / 60; 8-bit over 2048 34 / 39, over 4096 55 / 57, over 8192 101 / 83
//   65 to 128          8 of 64 over 1024 37 / 40, over 2048 52 / 52, over 4096 82 / 76; 12 of 17 over 2048 58 / 43; 4 of 128 over 1024 36 / 40;
//                      binary16 8 of 64 over 1024 47 / 44
//   others             2 of 64 over 16384 80 / 75; 16 of 64 over 512 54 / 44; 24 of 32 over 2048 77 / 74
// Blocks that 96 rows or fewer leave a quarter empty, two or more to each compute unit (drafts and contexts of up to these, from a half and
// a quarter of them on): 65 of 17 tokens over 1024 73 / 101, 128 of 17 over 8192 478 / 767, binary16 and 8-bit 128 over 4096 464 / 563,
// but over 300 97 / 101 and, of equal lengths, over 256 126 / 70; with 26 tokens 232 / 188 and 807 / 745.
// With up to 64 rows (16 tokens) it is the other one up to 65536 keys (48.7 / 73.5), and with 16 sequences of 16384 too (124 /
// 158).  Below its least work k_tree.hip is often the faster one too, most for 8-bit codes and short contexts in many
// blocks (16 of 64 over 256 53 / 22), and past 256 sequences up to about 400 (300 of 64 over 4096 2063 / 1936; 1000 of 64 over 1024
// 4225 / 6065): left to the kernel that rounds less.
constexpr int64_t kFewRowsOfTree = 64;

bool blocks_take(const KvAttendArgs& a, int dtype, int64_t keys) {
  const int64_t rows = a.max_q_len * (int64_t)(a.heads / a.cache.kv_heads), cus = cu_count();
  if (a.cache.head_dim != 128 || rows <= kFewRowsOfTree || a.num_seqs > 256) return false;
  const int64_t heads = (int64_t)a.cache.kv_heads * a.num_seqs;
  const int64_t blocks = (rows + kTreeBlockRows - 1) / kTreeBlockRows * heads;
  if (rows <= kTreeBlockRows * 3 / 4 && blocks > 2 * cus && a.max_kv_len > 512) return false;
  const int64_t work = (rows + 31) / 32 * heads * keys;
  if (a.num_seqs > 1 ? work < 1 << 19 : work <= 1 << 20) return false;
  const int64_t dear = work * (dtype == F16 ? 2 : 1) * (a.bits == 8 ? 2 : 1);
  return blocks > cus / 2 || blocks <= cus * 3 / 16 || dear > (blocks > cus / 4 ? 1 << 19 : 1 << 20);
}

// The most keys that a row sees, where a window can leave some out.
int64_t keys_in_window(const KvAttendArgs& a) {
  return a.window > 0 ? std::min((int64_t)a.max_kv_len, (int64_t)a.window + a.max_q_len) : a.max_kv_len;
}

constexpr int kBlocks = 0;  // in place of a number of rows / 16: the kernel of k_tree.hip

// Rows / 16 of a workgroup of the kernel for few rows: as many as hold a short draft, where decoding the keys again for more
// of them costs more than the tiles' number gives, and 1 for small calls, whose time is the chain from arguments to result.
// With 16 rows, and with more, in us: 128 wide, 32 heads over 8, 4-bit codes, bfloat16: one draft of 26 tokens over 1000 keys 12.7 and
// 15.2, over 4000 19.4 and 18.3, 8 of 6 over 1000 14.0 and 16.7, 8 of 13 over 8000 36.9 and 34.6; 64 wide, 20 heads over 5, 8-bit
// codes, binary16: one of 13 over 1000 11.4 and 19.4, 20 of 13 over a window of 4000 56 and 61, 4 of 64 over 8000 60 and 52.  Held
// against 935 points of both types, 4 and 8 bits, 64 and 128 wide, 1 to 48 drafts of 5 to 64 tokens over 256 to 32768 keys, it loses 1.4 to 6.2% on
// the mean of a form to the best number of rows; most where the workgroups just miss a round: 48 of 8 over 2048, 64 wide, 32 over 8, 4-bit,
// bfloat16 64 where 32 rows take 31; 16 of 64 over 2048, 20 over 5, 8-bit, binary16 108 where 16 take 74.
int few_rows(const KvAttendArgs& a, int64_t keys) {
  const int64_t D = a.cache.head_dim, rows = a.max_q_len * (int64_t)(a.heads / a.cache.kv_heads);
  const int64_t work = (rows + 15) / 16 * a.cache.kv_heads * a.num_seqs * keys;
  if (D > 128 || rows <= 16 || work <= (D == 64 ? 1 << 21 : 1 << 17)) return 1;
  return rows <= 32 || D == 128 ? 2 : 4;
}

TreePlan make_plan(const KvAttendArgs& a, int rt) {
  TreePlan p = {};
  const int64_t group = a.heads / a.cache.kv_heads, D = a.cache.head_dim, cus = cu_count();
  const int64_t rows = a.max_q_len * group;
  p.blocks = rt == kBlocks;
  int64_t n;
  if (p.blocks) {
    p.tiles = (int)((rows + kTreeBlockRows - 1) / kTreeBlockRows);
    const int64_t tiles = ((int64_t)a.max_kv_len + 63) / 64;
    const int64_t base = a.cache.kv_heads * std::min((int64_t)p.tiles * a.num_seqs, a.tokens * group / kTreeBlockRows + a.num_seqs);
    // as many workgroups as the device holds at once, or a multiple
    const int64_t slots = tree_block_slots();
    p.workgroups = (base + slots - 1) / slots * slots;
    n = most_splits(base, p.workgroups, tiles, 4, a.num_seqs);
    // what is left over of each sequence is a part of its own
    p.grid = std::min(base * n, 2 * p.workgroups + base);
  } else {
    p.rt = rt;
    const int64_t per = 16 * p.rt, unit = D == 256 && a.cache.head_dim >> a.cache.log2b == 8 ? 128 : 256;
    const int nb = a.cache.head_dim >> a.cache.log2b;
    const int64_t slots = cus * (D == 256 || nb == 4 || p.rt * D > 128 || wide_form((int)D, nb, a.bits, p.rt) ? 1 : 2);
    p.tiles = (int)((rows + per - 1) / per);
    // tiles with rows in them: sequences may bring fewer tokens than the longest
    const int64_t base = a.cache.kv_heads * std::min((int64_t)p.tiles * a.num_seqs, a.tokens * group / per + a.num_seqs);
    // never more than without a window
    n = choose_splits(base, slots, a.max_kv_len, a.num_seqs);
    if (keys_in_window(a) < a.max_kv_len) n = std::min(n, choose_splits(base, slots, keys_in_window(a), a.num_seqs));
    if (n > 1 && a.num_seqs > 1 && a.num_seqs <= 64) {
      p.workgroups = (base + slots - 1) / slots * slots;
      auto most = [&](int64_t keys) { return most_splits(base, p.workgroups, (keys + unit - 1) / unit, 1, a.num_seqs); };
      n = std::min(most(a.max_kv_len), most(keys_in_window(a)));
      p.grid = std::min(base * n, 2 * p.workgroups + base);
    }
  }
  p.nsplit = (int)n;
  if (n > 1) p.bytes = (size_t)a.tokens * a.heads * n * (D + 3) * 4;
  return p;
}

template <int D, int NB, int KB, int RT>
hipError_t launch_rows(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  const dim3 grid = p.workgroups != 0 ? dim3((unsigned)p.grid)
                                      : dim3((unsigned)(p.tiles * p.nsplit), (unsigned)a.cache.kv_heads, (unsigned)a.num_seqs);
  const auto kernel = dtype == F16 ? attend_kernel<D, NB, KB, RT, true, true> : attend_kernel<D, NB, KB, RT, false, true>;
  return launch_kernel(kernel, grid, dim3(64 * Occupancy<D, NB, KB, RT>::kWaves), s, a, da, p.nsplit,
                       static_cast<float*>(a.workspace), (int)p.workgroups);
}

template <int D, int NB, int KB>
hipError_t launch_bits(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  if constexpr (D == 64) {
    if (p.rt == 4) return launch_rows<D, NB, KB, 4>(a, p, dtype, da, s);
  }
  if constexpr (D <= 128) {
    if (p.rt == 2) return launch_rows<D, NB, KB, 2>(a, p, dtype, da, s);
  }
  return launch_rows<D, NB, KB, 1>(a, p, dtype, da, s);
}

template <int D, int NB>
hipError_t launch_blocks(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  return da.K == 16 ? launch_bits<D, NB, 4>(a, p, dtype, da, s) : launch_bits<D, NB, 8>(a, p, dtype, da, s);
}

hipError_t launch_few(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
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

// The workspace is asked for without a window and holds for any, whichever form is the one with it.
size_t kv_tree_workspace(const KvAttendArgs& a, int dtype) {
  const size_t few = std::max(make_plan(a, 1).bytes, make_plan(a, few_rows(a, a.max_kv_len)).bytes);
  return blocks_take(a, dtype, a.max_kv_len) ? std::max(few, make_plan(a, kBlocks).bytes) : few;
}

int launch_kv_tree(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream) {
  const TreePlan p = make_plan(a, blocks_take(a, dtype, keys_in_window(a)) ? kBlocks : few_rows(a, keys_in_window(a)));
  if ((int64_t)p.tiles * p.nsplit > UINT32_MAX / 512 || a.cache.kv_heads > 32767 || (p.nsplit > 1 && !kv_merge_fits(a)) ||
      p.grid > UINT32_MAX / 512) {
    g_launch_refused_for_size = true;
    return (int)hipErrorInvalidConfiguration;
  }
  const int e = p.blocks ? launch_tree_blocks(a, dtype, (int)p.grid, p.nsplit, (int)p.workgroups, da, stream)
                         : (int)launch_few(a, p, dtype, da, static_cast<hipStream_t>(stream));
  if (e != 0 || p.nsplit <= 1) return e;
  const MergeArgs m = {{static_cast<float*>(a.workspace), nullptr}, {p.nsplit, 0}, 0, 0};
  return launch_kv_merge(a, dtype, m, stream);
}

}  // namespace bq
