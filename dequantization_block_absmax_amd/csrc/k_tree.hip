// k_tree.hip -- attention of a tree of drafted tokens over the cache.
//
//   o_i = sum_j p_ij v_j, p_ij = softmax over the keys j that token i sees: the context before the draft, the tokens on
//   its path from the tree's root, itself
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bq_attend.h"
#include "bq_launch.h"

namespace bq {
namespace {

struct TreePlan {
  int rt, tiles, nsplit;
  size_t bytes;
};

int64_t choose_splits(int64_t base, int64_t slots, int64_t keys, int num_seqs) {
  const int64_t steps = (keys + 255) / 256;
  const int64_t least = num_seqs > 1 ? std::max((steps + 31) / 32, (int64_t)1) : 1;
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

TreePlan make_plan(const KvAttendArgs& a) {
  TreePlan p = {};
  const int64_t group = a.heads / a.cache.kv_heads, D = a.cache.head_dim, cus = cu_count();
  const int64_t rows = a.max_q_len * group;
  p.rt = D > 128 || rows <= 16 ? 1 : 2;
  p.tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
  const int64_t rows_all = a.tokens * group / (16 * p.rt) + a.num_seqs;
  const int64_t base = a.cache.kv_heads * std::min((int64_t)p.tiles * a.num_seqs, rows_all);
  const int nb = a.cache.head_dim >> a.cache.log2b;
  const int64_t slots = cus * (D == 256 || nb == 4 || p.rt * D > 128 || wide_form((int)D, nb, a.bits, p.rt) ? 1 : 2);
  int64_t n = choose_splits(base, slots, a.max_kv_len, a.num_seqs);
  if (a.window > 0 && (int64_t)a.window + a.max_q_len < a.max_kv_len) {
    const int64_t k = choose_splits(base, slots, (int64_t)a.window + a.max_q_len, a.num_seqs);
    n = k < n ? k : n;
  }
  p.nsplit = (int)n;
  if (n > 1) p.bytes = (size_t)a.tokens * a.heads * n * (D + 3) * 4;
  return p;
}

template <int D, int NB, int KB, int RT, bool HL>
hipError_t launch_type(const KvAttendArgs& a, const TreePlan& p, const DequantArgs& da, hipStream_t s) {
  const dim3 grid((unsigned)(p.tiles * p.nsplit), (unsigned)a.cache.kv_heads, (unsigned)a.num_seqs);
  return launch_kernel(attend_kernel<D, NB, KB, RT, HL, true>, grid, dim3(64 * Occupancy<D, NB, KB, RT>::kWaves), s, a, da,
                       p.nsplit, static_cast<float*>(a.workspace), (int)kAllRows);
}

template <int D, int NB, int KB, int RT>
hipError_t launch_rows(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  return dtype == F16 ? launch_type<D, NB, KB, RT, true>(a, p, da, s) : launch_type<D, NB, KB, RT, false>(a, p, da, s);
}

template <int D, int NB, int KB>
hipError_t launch_bits(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  if constexpr (D <= 128) {
    if (p.rt == 2) return launch_rows<D, NB, KB, 2>(a, p, dtype, da, s);
  }
  return launch_rows<D, NB, KB, 1>(a, p, dtype, da, s);
}

template <int D, int NB>
hipError_t launch_blocks(const KvAttendArgs& a, const TreePlan& p, int dtype, const DequantArgs& da, hipStream_t s) {
  return da.K == 16 ? launch_bits<D, NB, 4>(a, p, dtype, da, s) : launch_bits<D, NB, 8>(a, p, dtype, da, s);
}

}  // namespace

size_t kv_tree_workspace(const KvAttendArgs& a, int dtype) { return make_plan(a).bytes; }

int launch_kv_tree(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream) {
  const TreePlan p = make_plan(a);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((int64_t)p.tiles * p.nsplit > UINT32_MAX / 512 || a.cache.kv_heads > 32767 || (p.nsplit > 1 && !kv_merge_fits(a))) {
    g_launch_refused_for_size = true;
    return (int)hipErrorInvalidConfiguration;
  }
  const int nb = a.cache.head_dim >> a.cache.log2b;
  hipError_t e;
  if (a.cache.head_dim == 64)
    e = nb == 1 ? launch_blocks<64, 1>(a, p, dtype, da, s) : launch_blocks<64, 2>(a, p, dtype, da, s);
  else if (a.cache.head_dim == 128)
    e = nb == 1   ? launch_blocks<128, 1>(a, p, dtype, da, s)
        : nb == 2 ? launch_blocks<128, 2>(a, p, dtype, da, s)
                  : launch_blocks<128, 4>(a, p, dtype, da, s);
  else
    e = nb == 1   ? launch_blocks<256, 1>(a, p, dtype, da, s)
        : nb == 2 ? launch_blocks<256, 2>(a, p, dtype, da, s)
        : nb == 4 ? launch_blocks<256, 4>(a, p, dtype, da, s)
                  : launch_blocks<256, 8>(a, p, dtype, da, s);
  if (e != hipSuccess || p.nsplit <= 1) return (int)e;
  const MergeArgs m = {{static_cast<float*>(a.workspace), nullptr}, {p.nsplit, 0}, 0, 0};
  return launch_kv_merge(a, dtype, m, stream);
}

}  // namespace bq
