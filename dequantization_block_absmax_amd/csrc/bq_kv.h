// bq_kv.h -- the paged key/value cache and the attention over it, as the boundary (bq_api.cpp) hands them to the
// kernels.  Apart from bq_internal.h, whose digest dates the traffic counted of the blockwise kernels: a change
// here is none to them.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "bq_internal.h"

namespace bq {

// A paged key/value cache as the kernels take it (k_kv.hip, k_attn.hip): index 0 the keys, 1 the
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

// Attention over the cache (k_attn.hip).
struct KvAttendArgs {
  KvCacheArgs cache;
  const int32_t *q_start, *kv_len, *page_table;
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
