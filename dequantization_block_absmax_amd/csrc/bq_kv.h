// bq_kv.h -- the paged key/value cache and the attention over it, as the boundary (bq_api.cpp) hands them to the
// kernels.  Apart from bq_internal.h, whose digest dates the traffic counted of the blockwise kernels: a change
// here is none to them.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "bq_internal.h"

namespace bq {

// A paged key/value cache as the kernels take it (k_kv.hip, bq_attend.h): index 0 the keys, 1 the
// values.
struct KvCacheArgs {
  uint8_t* packed[2];
  float* absmax[2];
  int32_t num_pages, log2_page, kv_heads, head_dim, log2b;
};
int launch_kv_write(const KvCacheArgs& c, int dtype, const void* k, const void* v, int64_t tokens, int64_t k_stride,
                    int64_t v_stride, const int64_t* slots, const PreparedTable& t, void* stream);
int launch_kv_read(const KvCacheArgs& c, int dtype, void* k, void* v, int64_t tokens, int64_t k_stride,
                   int64_t v_stride, const int64_t* slots, const DequantArgs& da, void* stream);


// Appending with the rotation by position (k_kv_append.hip).
struct KvAppendArgs {
  KvCacheArgs cache;
  const void *k, *v;
  int64_t tokens, k_stride, v_stride;  // strides in elements
  const int64_t *positions, *slots;
  const float *cos, *sin;
  int64_t angle_stride, max_positions;
  int32_t rotary_dim, interleaved;
  const void* q;  // or NULL
  int64_t q_stride;
  void* q_out;
  int64_t q_out_stride;
  int32_t heads;
};
int launch_kv_append(const KvAppendArgs& a, int dtype, const PreparedTable& t, void* stream);

// Moving the accepted path of a tree of drafted tokens to the front of its draft (k_kv_accept.hip).
struct KvAcceptArgs {
  KvCacheArgs cache;
  const int32_t *q_start, *kv_len, *page_table;
  int64_t table_stride, tokens;
  int32_t num_seqs, max_kv_len;
  const int32_t* path;
  int64_t path_stride;
  const int32_t* path_len;
  int32_t bits;
};
int launch_kv_accept(const KvAcceptArgs& a, void* stream);

// Attention over the cache (k_attn.hip, bq_attend.h).
struct KvAttendArgs {
  KvCacheArgs cache;
  const int32_t *q_start, *kv_len, *page_table;
  const int32_t* parents;  // of new tokens that are a tree, else NULL
  int64_t table_stride, tokens;
  int32_t num_seqs, max_q_len, max_kv_len;
  const void* q;
  int64_t q_stride;  // elements between tokens
  void* out;
  int64_t out_stride;
  float* lse;        // or NULL
  int32_t heads, causal, window;
  int32_t bits;      // of a code
  float scale;
  void* workspace;
};
// Bytes of workspace the launch needs (no device is touched beyond its CU count).
size_t kv_attend_workspace(const KvAttendArgs& a, int dtype);
int launch_kv_attend(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream);
// Attention of a tree of new tokens (k_tree_few.hip, k_tree.hip), at most kMostNodes to a sequence.
constexpr int kMostNodes = 256;
constexpr int kTreeBlockRows = 128;  // of a workgroup of k_tree.hip
int tree_block_slots();  // workgroups of that kernel the device holds at once
// The call spread over about `workgroups` workgroups, of `grid` at most; a block of rows takes up to nsplit.
int launch_tree_blocks(const KvAttendArgs& a, int dtype, int grid, int nsplit, int workgroups, const DequantArgs& da, void* stream);
size_t kv_tree_workspace(const KvAttendArgs& a, int dtype);
int launch_kv_tree(const KvAttendArgs& a, int dtype, const DequantArgs& da, void* stream);
// Joins the partial results of splits of the keys (k_attn_merge.hip): [0] those of sequences with few
// rows, [1] with many; nsplit <= 1: nothing to join.  Not both: every sequence is of `kind`.
struct MergeArgs {
  const float* partial[2];
  int nsplit[2];
  int both, kind;
};
int launch_kv_merge(const KvAttendArgs& a, int dtype, const MergeArgs& m, void* stream);
bool kv_merge_fits(const KvAttendArgs& a);  // the rows' launch counts its threads in 32 bits
// How k_attn_chunk.hip goes about a call: expanded tiles of keys, rows per workgroup, splits, and where
// its parts of the workspace begin (bytes).
struct ChunkPlan {
  int ntiles, blocks, nsplit;
  size_t rest_at, info_at, exponents_at, partial_at, end;
};
constexpr int kTileInfoBytes = 16;
constexpr int kChunkRows = 128;
int chunk_slots(int head_dim, int dtype);  // workgroups of that kernel the device holds at once
int64_t chunk_rest_bytes(int head_dim, int dtype);
int launch_kv_chunk(const KvAttendArgs& a, int dtype, const ChunkPlan& p, const DequantArgs& da, void* stream);

}  // namespace bq
