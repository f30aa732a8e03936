/*
 * bq.h -- blockwise absmax quantization and dequantization for AMD Instinct MI355X (gfx950).
 *
 * C ABI of libbq.so.  Every entry point validates its arguments on the host, then enqueues
 * its kernels on the caller's HIP stream and returns without waiting.  The library never
 * allocates or frees device memory, never copies between host and device, and never
 * synchronizes, so every call can be captured in a HIP graph.
 *
 * Conventions shared by all entry points
 *   - Device pointers (marked [device]) must be device memory of the current device, and
 *     data arrays must be 16-byte aligned (fp32 statistic arrays: 4-byte aligned).  The
 *     caller owns every buffer and keeps it alive until the enqueued work completes.
 *   - Host pointers (marked [host]) are read during the call only.
 *   - `stream` is the HIP stream to enqueue on; 0 is the legacy null stream.  This follows
 *     "Respect the current CUDA stream in blockwise quantization" (bitsandbytes PR 2052),
 *     Summary: quantization must run on the caller's current stream, not stream 0.
 *   - Errors: every check happens before any HIP call; on error nothing is enqueued and no
 *     output is written.  A failed launch returns BQ_ERR_HIP.  n == 0 is valid and enqueues
 *     nothing.  Element data is never inspected on the host (that would need a sync).
 *   - Determinism: outputs are bit-identical across runs, streams and devices of this kind.
 *
 * The arithmetic (each rule is also written where it is implemented):
 *   blocks      element i belongs to block i / B of the flattened 1-D array; the last
 *               block may be partial ("full blocks, and tails", PR 2052, "Correctness and
 *               safety"); B is a power of two from 32 to 4096 (PR 2052, Summary).
 *   absmax      a_b = max |x_i| over the finite elements of block b; +0 if there are none.
 *   normalize   y_i = fl32(fl32(x_i * s) * fl32(1 / fl32(a_b * s))), s = 2^64 if
 *               a_b < 2^-64, s = 2^-64 if a_b > 2^64, else 1 (|y_i| <= 1).
 *   nearest     q_i = the smallest index k minimizing |y_i - c_k| exactly (equal distances
 *               resolve to the lowest index, as in "[OMNIML-5899] Add CUDA kernels for IQ
 *               packing", review item "Search equivalence").  Non-finite x_i and every
 *               element of a block with a_b = 0 take z = the nearest code to 0.0.
 *   packing     16-entry table: two codes per byte, the first element of each pair in the
 *               high nibble, ceil(n/2) bytes, a zero pad nibble for odd n (33 values fill
 *               17 bytes, as in onnxruntime/mobius PR 794, finding F3).  256-entry table:
 *               one byte per element.
 *   dequantize  out_i = RN(fl32(c[q_i] * a_b)): one binary32 multiply, then one
 *               round-to-nearest-even to the output type (overflow to infinity, signed zeros
 *               and subnormals kept, NaN to a quiet NaN of the same sign).
 */
#ifndef BQ_H
#define BQ_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the unquantized side. */
typedef enum { BQ_F32 = 0, BQ_F16 = 1, BQ_BF16 = 2 } bq_dtype;

typedef enum {
  BQ_OK = 0,
  BQ_ERR_NULL = 1,      /* a required pointer is NULL */
  BQ_ERR_DTYPE = 2,     /* dtype is not a bq_dtype */
  BQ_ERR_SIZE = 3,      /* a count, length or stride out of its range: n < 0, more than INT32_MAX blocks, n not a whole number of rows, or a
                           launch of more than 2^32 - 1 threads, refused before any work is
                           enqueued (quantize and 4-bit dequantize from 2^37 elements, 8-bit
                           dequantize from 2^36) */
  BQ_ERR_BLOCKSIZE = 4, /* blocksize not a power of two in [32, 4096] */
  BQ_ERR_TABLE = 5,     /* code table: size, order, range or spacing (see bq_code_table) */
  BQ_ERR_ALIGNMENT = 6, /* a device pointer is not aligned as required */
  BQ_ERR_FORMAT = 7,    /* unknown bq_q32_format, row_len not a multiple of 32 (of 256 for
                           the IQ2_XS- and IQ1_S-style calls), page_size or head_dim of a cache, or rotary_dim */
  BQ_ERR_WORKSPACE = 8, /* workspace missing or smaller than bq_nested_workspace_bytes or
                           bq_kv_attention_workspace_bytes (bq_kv_tree_attention_workspace_bytes) */
  BQ_ERR_HIP = 9        /* the HIP runtime rejected a launch */
} bq_status;

/* A code table in host memory: `size` (16 or 256) binary32 entries, strictly ascending,
 * each finite and within [-1, 1], every nonzero entry of magnitude >= 2^-20 (so that sums
 * of two entries are exact in binary64); -0.0 is read as +0.0.  16 entries select 4-bit
 * codes (packed two per byte), 256 entries 8-bit codes.  The table is read during the call
 * and passed to the kernels by value; nothing is uploaded. */
typedef struct {
  const float* entries; /* [host] */
  int32_t size;
} bq_code_table;

/* Blockwise quantization (General8 / FP4 / NF4 family of "Respect the current CUDA stream
 * in blockwise quantization", bitsandbytes PR 2052, Summary and "Correctness and safety").
 *   in         [device] n elements of `dtype`, read only.
 *   absmax     [device] out: ceil(n / blocksize) binary32 block maxima.
 *   packed     [device] out: ceil(n / 2) bytes (16-entry table) or n bytes (256 entries). */
bq_status bq_quantize_blockwise(const void* in, bq_dtype dtype, int64_t n, int32_t blocksize,
                                const bq_code_table* code_table, float* absmax, uint8_t* packed,
                                hipStream_t stream);

/* Blockwise dequantization, the inverse of bq_quantize_blockwise: one binary32 multiply of
 * the code's table entry by the block absmax, rounded once to `dtype`.
 *   out        [device] out: n elements of `dtype`.
 *   absmax     [device] ceil(n / blocksize) binary32 values (any values; NaN propagates).
 *   packed     [device] codes laid out as bq_quantize_blockwise writes them. */
bq_status bq_dequantize_blockwise(void* out, bq_dtype dtype, int64_t n, int32_t blocksize,
                                  const bq_code_table* code_table, const float* absmax,
                                  const uint8_t* packed, hipStream_t stream);

/* Second-level statistics of nested quantization (nested General8 and compressed-statistics
 * NF4 of PR 2052, "Reproduced failure").  The block absmax values a_b are replaced by:
 *   mean     = RN32(S / nb), S the binary64 pairwise sum of a_0 .. a_{nb-1} zero-padded to a
 *              power-of-two length (sum of a range = sum of its left half + sum of its right);
 *   d_b      = fl32(a_b - mean), quantized with the 256-entry `table` in groups of
 *              `blocksize2` blocks by the same absmax / normalize / nearest rules;
 *   rebuilt  a'_b = fl32(fl32(c2[q2_b] * absmax2_g) + mean), used by the nested dequantize. */
typedef struct {
  uint8_t* qabsmax;            /* [device] nb codes q2_b (nb = ceil(n / blocksize)), 16-byte aligned */
  float* absmax2;              /* [device] ceil(nb / blocksize2) binary32 group maxima */
  float* mean;                 /* [device] 1 binary32 value */
  const bq_code_table* table;  /* [host] 256-entry statistics table */
  int32_t blocksize2;          /* blocks per statistics group: power of two in [32, 4096] */
  void* workspace;             /* [device] scratch, 256-byte aligned; quantize only */
  size_t workspace_bytes;
} bq_nested_stats;

/* Bytes of device workspace bq_quantize_nested needs (0 for n <= 0), for any dtype.  After the
 * call's stream work completes, the workspace starts with the nb = ceil(n / blocksize) block
 * maxima a_b: nb binary32 values for BQ_F32 input; for BQ_F16 / BQ_BF16 input, nb 16-bit
 * values of that type (the maximum of |x| over values of a format is itself a value of the
 * format, so they are exact). */
size_t bq_nested_workspace_bytes(int64_t n, int32_t blocksize, int32_t blocksize2);

/* Blockwise quantization with nested statistics: packed data codes as bq_quantize_blockwise,
 * and the statistics of bq_nested_stats written to stats->qabsmax, ->absmax2 and ->mean.
 * Enqueues up to four kernels on `stream`: the data pass, the partial-sum runs (inputs of more
 * than 2^20 elements), the mean (more than 2^31 elements), then the statistics. */
bq_status bq_quantize_nested(const void* in, bq_dtype dtype, int64_t n, int32_t blocksize,
                             const bq_code_table* code_table, bq_nested_stats* stats,
                             uint8_t* packed, hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc): bq_quantize_nested with the library's own scratch
 * memory in place of the caller's workspace.  stats->workspace and stats->workspace_bytes are
 * ignored; everything else, the outputs and the errors are those of bq_quantize_nested.
 * The scratch is a fixed 36 MiB array per GPU (37,748,736 bytes, held by every GPU the library
 * runs on until the process ends), enough for any input whose bq_nested_workspace_bytes is at
 * most that size, e.g. 2^29 elements at block size 64; a larger input returns
 * BQ_ERR_WORKSPACE before anything is enqueued.  The call allocates nothing.  All calls on one
 * GPU share its scratch, which keeps the last call's contents: calls that overlap on one GPU
 * (two streams or host threads without ordering between them) race and give wrong results. */
bq_status bq_quantize_nested_noalloc(const void* in, bq_dtype dtype, int64_t n, int32_t blocksize,
                                     const bq_code_table* code_table, bq_nested_stats* stats,
                                     uint8_t* packed, hipStream_t stream);

/* Dequantization from nested statistics: rebuilds each a'_b from (q2_b, absmax2_g, mean) and
 * dequantizes with it, in one kernel.  stats->workspace is not used. */
bq_status bq_dequantize_nested(void* out, bq_dtype dtype, int64_t n, int32_t blocksize,
                               const bq_code_table* code_table, const bq_nested_stats* stats,
                               const uint8_t* packed, hipStream_t stream);

/* GGUF-style 32-element blocks (the Q4_0 / Q8_0 shapes of "Cache device-side constants in
 * dequant kernels", ComfyUI-GGUF PR 472, "Verification" table):
 *   BQ_Q32_Q4: 18 bytes = binary16 scale d (little-endian) + 16 bytes; element j < 16 is the
 *              low nibble of byte j, element 16 + j its high nibble (the low-before-high
 *              nibble order of that page's "Problem" section); value (q - 8) * d.
 *   BQ_Q32_Q8: 34 bytes = binary16 d + 32 int8; value q * d.
 * The binary32 product is exact; it is rounded once to `dtype`. */
typedef enum { BQ_Q32_Q4 = 0, BQ_Q32_Q8 = 1 } bq_q32_format;

/* Dequantizes n / 32 consecutive blocks (row-major rows of row_len elements; row_len a
 * multiple of 32 dividing n, so no block straddles a row: the per-row alignment check of
 * "[OMNIML-5899] Add CUDA kernels for IQ packing").
 *   blocks  [device] (n / 32) * 18 or * 34 bytes, 2-byte aligned (the records themselves are;
 *           a slice starting at any block is accepted; 16-byte aligned arrays are read faster).
 *   out     [device] out: n elements of `dtype`. */
bq_status bq_dequant_q32(const void* blocks, bq_dtype dtype, int64_t n, int32_t row_len,
                         bq_q32_format format, void* out, hipStream_t stream);

/* Fused dequantize + linear for small batches (decoding): y = x . deq(W)^T, with the
 * dequantized weights formed in registers and never written out (weights used without
 * expanding the full tensor, as in the mixed-input GEMMs of "stable-diffusion.cpp PR 2278",
 * Summary; here for the blockwise codes of bq_quantize_blockwise).
 *   x          [device] M x K row-major activations of `dtype`, 16-byte aligned.
 *   M, K, N    1 <= M <= 4; K > 0 and a multiple of 16; 0 <= N <= 67,108,860 (a launch holds
 *              at most 2^32 - 1 threads; N = 0: nothing enqueued).
 *   blocksize, code_table
 *              the block size and table W was quantized with.
 *   absmax     [device] ceil(N*K / blocksize) binary32 block maxima of W.
 *   packed     [device] W's codes, 16-byte aligned, as bq_quantize_blockwise writes them for
 *              the N*K-element weight tensor stored row-major (element (n, k) of W is flat
 *              element n*K + k; blocks run over the flat index).
 *   y          [device] out: M x N row-major binary32.
 * y[m][n] approximates sum_k x[m][k] * w[n][k], w = fl32(c[q] * a) the binary32 dequantized
 * weight (never rounded to 16 bits), accumulated in binary32 in an unspecified order: its
 * error is at most (K/1024 + 64) * 2^-24 * sum_k |x[m][k] w[n][k]|.
 * Errors: BQ_ERR_SIZE for M outside [1, 4], K not a positive multiple of 16, N outside
 * [0, 67108860], or more than INT32_MAX blocks; otherwise as bq_dequantize_blockwise. */
bq_status bq_linear_blockwise(const void* x, bq_dtype dtype, int64_t M, int64_t K, int64_t N, int32_t blocksize,
                              const bq_code_table* code_table, const float* absmax, const uint8_t* packed,
                              float* y, hipStream_t stream);

/* Fused dequantize + GEMM on the matrix cores, for batches of rows (the 16-bit-activation,
 * 4-bit-weight GEMM named in "stable-diffusion.cpp PR 2278", Summary, here for the blockwise
 * codes of bq_quantize_blockwise): y = x . W16^T, where W16 is exactly the 16-bit tensor
 * bq_dequantize_blockwise writes for W with this `dtype`, w16 = RN16(fl32(c[q] * a)), formed
 * in registers and never written out.
 *   x          [device] M x K row-major activations, BQ_BF16 or BQ_F16, 16-byte aligned.
 *   M, K, N    M >= 1 (at most 4,194,240); K > 0 and a multiple of 64; 0 <= N <= 536,870,848
 *              (a launch holds at most 2^32 - 1 threads; N = 0: nothing enqueued).
 *   blocksize, code_table, absmax, packed
 *              W, as for bq_linear_blockwise (packed 16-byte aligned).
 *   y          [device] out: M x N row-major binary32.
 * Each product x[m][k] * w16[n][k] is exact in binary32; the products are accumulated in
 * binary32 in an unspecified order, so y[m][n] lies within (K + 64) * 2^-24 * sum_k
 * |x[m][k] w16[n][k]| of the exact sum (products below the binary32 normal range may be
 * flushed to zero by the matrix cores).  The result is the same on every call on one device.
 * Errors: BQ_ERR_DTYPE for BQ_F32; BQ_ERR_SIZE for M outside [1, 4194240], K not a positive
 * multiple of 64, N outside [0, 536870848], or more than INT32_MAX blocks; otherwise as
 * bq_dequantize_blockwise. */
bq_status bq_gemm_blockwise(const void* x, bq_dtype dtype, int64_t M, int64_t K, int64_t N, int32_t blocksize,
                            const bq_code_table* code_table, const float* absmax, const uint8_t* packed,
                            float* y, hipStream_t stream);

/* IQ2_XS-style search encoding ("[OMNIML-5899] Add CUDA kernels for IQ packing", Model-
 * Optimizer PR 2448: the Summary's caller-computed fp16 superblock scales, the review items
 * "Wire format", "Scale anchors", "Even-parity sign field" and "Search equivalence", and the
 * round-3 "IQ2_XS grouping" item).  A superblock is 256 consecutive elements, stored in 74
 * bytes:
 *   bytes 0-1   the caller's binary16 scale d (little-endian);
 *   bytes 2-65  32 little-endian 16-bit words, one per 8-element vector v: bits 0-8 the grid
 *               entry e, bits 9-15 the signs of the vector's elements 0-6 (bit set =
 *               negative); element 7's sign is the parity of those seven bits, so every
 *               vector holds an even number of negative elements;
 *   bytes 66-73 byte i = ls[2i] | ls[2i+1] << 4, the 4-bit local scale of each 16-element
 *               group g (vectors 2g and 2g+1).
 * Element j of vector v decodes to d * (2 * ls + 1) / 8 * grid[e][j], negated if its sign is
 * set (exact in binary32, then rounded once to the output type).
 * The grid is the caller's: 512 entries of 8 magnitude bytes (entry e, element j at byte
 * 8e + j), for the IQ2_XS format those of the GGML grid (bytes 0x08, 0x19, 0x2b).
 *
 * The search, per superblock with a valid d (binary32 throughout, fused multiply-adds where
 * written fma, every other operation rounded once):
 *   a_j = |x_j| (a NaN or infinite element reads as +0; -0 is not negative);
 *   xn = fma-chain sum of a_j^2 and dot_e = fma-chain sum of a_j * q_j (j = 0..7, from +0);
 *   with an odd count of negative elements, dot_e = fma(-2, w_e, dot_e), w_e the least
 *   fl(a_j * q_j), and the first element reaching w_e has its sign flipped;
 *   s = d * (2 * ls + 1) / 8; error(e, s) = max(fma(s*s, qn_e, fma(-2s, dot_e, xn)), 0),
 *   qn_e = sum of q_j^2;
 *   each group takes the ls whose fl(E(v0) + E(v1)) is least (E(v) = least error of vector v
 *   over the grid; equal sums: the lower ls), then each vector the entry of least error at
 *   that ls (equal errors: the lower entry).
 * Scales: d = +0 or -0 gives an all-zero superblock.  A NaN, infinite or negative d is
 * rejected: the superblock is written as zeros and *rejected is incremented (atomically, on
 * the device: the caller sets it beforehand and reads it after the stream work completes).
 *   in        [device] n elements of `dtype`, 16-byte aligned.
 *   n, row_len  row_len a positive multiple of 256 dividing n (n = 0: nothing enqueued), so no
 *             superblock straddles a row (the per-row check of that page's round-3 review).
 *   grid      [device] 4096 bytes, 16-byte aligned.
 *   scales    [device] n / 256 binary16 bit patterns, 2-byte aligned.
 *   blocks    [device] out: (n / 256) * 74 bytes, 2-byte aligned.
 *   rejected  [device] one uint32 counter, 4-byte aligned.
 * Errors: BQ_ERR_DTYPE, BQ_ERR_FORMAT (row_len), BQ_ERR_SIZE (n negative or not a multiple of
 * row_len, more than INT32_MAX superblocks), BQ_ERR_NULL, BQ_ERR_ALIGNMENT, BQ_ERR_HIP. */
bq_status bq_iq2xs_quantize(const void* in, bq_dtype dtype, int64_t n, int64_t row_len, const uint8_t* grid,
                            const uint16_t* scales, uint8_t* blocks, uint32_t* rejected, hipStream_t stream);

/* Decodes n / 256 superblocks laid out as bq_iq2xs_quantize writes them (any bytes: d is read
 * as binary16 whatever it holds) to n elements of `dtype`.
 *   blocks    [device] (n / 256) * 74 bytes, 2-byte aligned.
 *   grid      [device] 4096 bytes, 8-byte aligned.
 *   out       [device] out: n elements of `dtype`, 16-byte aligned.
 * Errors: as bq_iq2xs_quantize. */
bq_status bq_iq2xs_dequantize(const uint8_t* blocks, const uint8_t* grid, int64_t n, int64_t row_len,
                              bq_dtype dtype, void* out, hipStream_t stream);

/* IQ1_S-style encoding ("[OMNIML-5899] Add CUDA kernels for IQ packing", Model-Optimizer PR
 * 2448: "Provenance" (16.875 = 15 x (1 + 1/8), the 0.61 scale predictor, the 0.125 delta), the
 * review items "Wire format", "Scale anchors" and "Search equivalence", the round-3 item on
 * the shifted objective).  A superblock is 256 consecutive elements, stored in 50 bytes:
 *   bytes 0-1   binary16 scale d (little-endian);
 *   bytes 2-33  byte v = the low 8 bits of vector v's 11-bit grid entry (vector v = elements
 *               8v .. 8v+7);
 *   bytes 34-49 8 little-endian 16-bit words, one per 32-element sub-block b (vectors
 *               4b .. 4b+3): bits 3l..3l+2 the high 3 bits of vector 4b+l's entry, bits 12-14
 *               the local scale ls, bit 15 the delta sign (set: delta = -1/8, else +1/8).
 * Element j of vector v decodes to fl32(d * (2 ls + 1) * (g_j + delta)), g the grid's signed
 * byte (exact for the ternary IQ1_S grid), rounded once to the output type.
 * The grid is the caller's: 2048 entries of 8 signed bytes (entry e, element j at byte 8e + j),
 * for the IQ1_S format those of the GGML ternary grid (-1, 0, +1).
 *
 * The encoder, per superblock (binary32 throughout, fused multiply-adds where written fma):
 *   x_j = the element, a NaN or infinite element read as +0;
 *   d = RN16(fl32(fl32(amax / 16.875) * 0.61)), amax = max |x_j| over the superblock,
 *   saturated to the largest finite binary16; d = 0 gives an all-zero superblock;
 *   per vector: xn, dot_e and xsum are fma chains of x_j^2, x_j * g_j and x_j * 1 (j = 0..7,
 *   from +0); for a choice c = ls + 8 * sign, dl = d * (2 ls + 1), delta = +-1/8:
 *   error(e, c) = max(fma(dl*dl, sn, fma(-2 dl, fma(delta, xsum, dot_e), xn)), 0),
 *   sn = qn_e + 2 delta qs_e + 8 delta^2 (qn, qs = sum of g^2 and of g);
 *   each sub-block takes the choice whose summed error over its four vectors (in vector
 *   order) is least (equal sums: the lower c), then each vector the entry of least error at
 *   that choice (equal errors: the lower entry).
 *   in        [device] n elements of `dtype`, 16-byte aligned.
 *   n, row_len  row_len a positive multiple of 256 dividing n (n = 0: nothing enqueued).
 *   grid      [device] 16384 bytes, 16-byte aligned.
 *   blocks    [device] out: (n / 256) * 50 bytes, 2-byte aligned.
 * Errors: BQ_ERR_DTYPE, BQ_ERR_FORMAT (row_len), BQ_ERR_SIZE (n negative or not a multiple of
 * row_len, more than INT32_MAX superblocks), BQ_ERR_NULL, BQ_ERR_ALIGNMENT, BQ_ERR_HIP. */
bq_status bq_iq1s_quantize(const void* in, bq_dtype dtype, int64_t n, int64_t row_len, const int8_t* grid,
                           uint8_t* blocks, hipStream_t stream);

/* Decodes n / 256 superblocks laid out as bq_iq1s_quantize writes them (any bytes) to n
 * elements of `dtype`.
 *   blocks    [device] (n / 256) * 50 bytes, 2-byte aligned.
 *   grid      [device] 16384 bytes, 8-byte aligned.
 *   out       [device] out: n elements of `dtype`, 16-byte aligned.
 * Errors: as bq_iq1s_quantize. */
bq_status bq_iq1s_dequantize(const uint8_t* blocks, const int8_t* grid, int64_t n, int64_t row_len,
                             bq_dtype dtype, void* out, hipStream_t stream);

/* ---- A paged key/value cache in blockwise codes --------------------------------------------
 *
 * The cache of a served transformer: a pool of pages of `page_size` tokens each, for keys and for
 * values.  Element (page, head, slot, d) of a pool is flat element
 *     ((page * kv_heads + head) * page_size + slot) * head_dim + d
 * of an array held exactly as bq_quantize_blockwise holds it (packed codes and block maxima; B
 * divides head_dim, so a block holds elements of one token's head): bq_dequantize_blockwise
 * expands a whole pool.  Token slot s of the cache is slot s % page_size of page s / page_size.
 * Which pages belong to which sequence is the caller's affair (see bq_kv_batch). */
typedef struct {
  uint8_t* k_packed;  /* [device] codes of num_pages * kv_heads * page_size * head_dim keys, 16-byte aligned */
  float* k_absmax;    /* [device] their block maxima, 16-byte aligned */
  uint8_t* v_packed;  /* [device] the values' codes, 16-byte aligned */
  float* v_absmax;    /* [device] the values' block maxima, 16-byte aligned */
  const bq_code_table* table; /* [host] 16 or 256 entries, for keys and values */
  int32_t num_pages;
  int32_t page_size;  /* tokens per page: a power of two from 16 to 4096 */
  int32_t kv_heads;
  int32_t head_dim;   /* a multiple of 32 from 32 to 256 (bq_kv_attention: 64, 128 or 256) */
  int32_t blocksize;  /* a power of two from 32 that divides head_dim */
} bq_kv_cache;

/* Quantizes the keys and values of `tokens` new tokens into the cache, by the absmax, normalize and
 * nearest rules above (the codes and maxima are those of bq_quantize_blockwise, bit for bit).
 *   k, v       [device] tokens rows of kv_heads * head_dim elements of `dtype`, 16-byte aligned.
 *   k_stride, v_stride
 *              elements from one token's row to the next, at least kv_heads * head_dim, a multiple of
 *              16 bytes (the rows may be parts of a fused projection's output).
 *   slots      [device] one cache slot per token, 8-byte aligned.  A token whose slot is outside
 *              [0, num_pages * page_size) is not written.  Slots must differ: of two tokens with one
 *              slot, either may be kept, in parts.
 * Errors: BQ_ERR_DTYPE; BQ_ERR_SIZE (tokens negative or tokens * kv_heads * head_dim >= 2^34, a pool of
 * more than INT32_MAX blocks, num_pages or kv_heads below 1, a stride too short); BQ_ERR_FORMAT
 * (page_size or head_dim); BQ_ERR_BLOCKSIZE; BQ_ERR_TABLE; BQ_ERR_NULL; BQ_ERR_ALIGNMENT; BQ_ERR_HIP.
 * tokens == 0 enqueues nothing. */
bq_status bq_kv_write(const bq_kv_cache* cache, bq_dtype dtype, const void* k, const void* v, int64_t tokens,
                      int64_t k_stride, int64_t v_stride, const int64_t* slots, hipStream_t stream);

/* Reads the keys and values of `tokens` cache slots back, each element RN(fl32(c[q] * a)) as
 * bq_dequantize_blockwise gives it; a token whose slot is outside the pool reads as zeros.
 *   k, v       [device] out: tokens rows of kv_heads * head_dim elements of `dtype`, 16-byte aligned, with
 *              strides as in bq_kv_write.
 *   slots      [device] one cache slot per token, 8-byte aligned, in any order, repeats allowed.
 * Errors: as bq_kv_write. */
bq_status bq_kv_read(const bq_kv_cache* cache, bq_dtype dtype, void* k, void* v, int64_t tokens, int64_t k_stride,
                     int64_t v_stride, const int64_t* slots, hipStream_t stream);

/* The sequences of one attention call.  Sequence s brings the new tokens q_start[s] ..
 * q_start[s + 1] - 1 (rows of q and out) and has kv_len[s] tokens in the cache, its new ones included:
 * key j is in slot j % page_size of page page_table[s * table_stride + j / page_size].  New token i of
 * n stands at position kv_len[s] - n + i. */
typedef struct {
  const int32_t* q_start;    /* [device] num_seqs + 1 ascending row numbers */
  const int32_t* kv_len;     /* [device] num_seqs; read as at most max_kv_len and table_stride * page_size */
  const int32_t* page_table; /* [device] num_seqs rows; a page outside the pool hides its keys */
  int64_t table_stride;      /* entries from one row to the next */
  int64_t tokens;            /* rows of q and out; rows outside every sequence are left as they are */
  int32_t num_seqs;          /* at most 65535 */
  int32_t max_q_len;         /* no sequence brings more new tokens (later ones are left out) */
  int32_t max_kv_len;        /* no sequence has more keys (later ones are left out) */
} bq_kv_batch;

/* Bytes of workspace bq_kv_attention needs for this call's shape (the batch's pointers are not
 * read); 0 if an argument is not valid.  It depends on the device's number of compute units.  A call whose
 * max_q_len is long (above 384 rows, new tokens x query heads of a key/value head; 256 for binary16, 128 for
 * 256-wide heads) asks for num_seqs x max_kv_len keys and values expanded to 16 bits, 4 GiB (4.75 for binary16) at
 * most: a call that would need more does without, and is several times slower.  Give max_kv_len as it is. */
size_t bq_kv_attention_workspace_bytes(const bq_kv_cache* cache, const bq_kv_batch* batch, bq_dtype dtype,
                                       int32_t heads);

/* Attention of new tokens over the cache, for single tokens (decoding), a few (drafts) and long
 * pieces of a prompt alike:
 *     out[i] = sum_j p_ij v_j,   p_ij = softmax over j of scale * (q_i . k_j),
 * query head h over key/value head h / (heads / kv_heads), keys and values being the cached
 * fl32(c[q] * a).  Row i at position t sees the keys j <= t if `causal` is nonzero, else all kv_len;
 * of these, if window > 0, those with j > t - window.  What is cached for keys that no row of a
 * sequence sees does not matter (it may be NaN).  A row that sees no key gives zeros, and -infinity in lse.
 *   dtype      BQ_F16 or BQ_BF16: the type of q and out.
 *   q          [device] tokens rows of heads * head_dim elements, 16-byte aligned; q_stride elements
 *              from row to row (at least heads * head_dim, a multiple of 8).
 *   heads      a positive multiple of kv_heads.
 *   out        [device] out: rows as in q, with out_stride.
 *   lse        [device] out, or NULL: tokens x heads binary32, the natural logarithm of
 *              sum_j exp(scale * (q_i . k_j)).
 *   workspace  [device] bq_kv_attention_workspace_bytes bytes, 256-byte aligned (NULL if that is 0).
 * Products, maxima and sums are held in binary32; bq_attend.h (few rows) and k_attn_chunk.hip (many) say what is
 * rounded to 16 bits on the way.  Over many keys the 2-norm of the error is up to 1.2 times that of rounding the
 * exact result to bfloat16, 1.5 times for binary16; where one key carries a row of binary16, a part in 2^11 more.
 * Results are the same on every call on one device.  Block maxima of keys that are seen must be
 * finite and at most 2^100; from token to token they may differ by any factor (values below 2^-80 lose bits).
 * Errors: BQ_ERR_DTYPE; BQ_ERR_SIZE (a negative count or length, num_seqs > 65535, heads, tokens * heads
 * above INT32_MAX, more than 2^30 keys, a stride, window < 0, a scale that is not finite, kv_heads above
 * 32767, or a launch of more than 2^32 - 1 threads); BQ_ERR_WORKSPACE;
 * otherwise as bq_kv_write.  tokens, num_seqs or max_q_len of 0 enqueue nothing. */
bq_status bq_kv_attention(const bq_kv_cache* cache, const bq_kv_batch* batch, bq_dtype dtype, const void* q,
                          int64_t q_stride, int32_t heads, float scale, int32_t causal, int32_t window, void* out,
                          int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* ---- Drafted tokens over the cache -----------------------------------------------------------
 *
 * A server that drafts several continuations of a sequence at once, as a tree, and verifies them in one
 * step: bq_kv_append puts the draft's keys and values into the cache, keys (and queries) rotated to their
 * positions; bq_kv_tree_attention attends over context and draft; bq_kv_tree_accept moves the accepted
 * path to the front of the draft, where the next one follows it. */

/* Rotation by position.  Pair i of a head, i < rotary_dim / 2, of a token at position t is turned by the
 * angle whose cosine and sine are cos[t * stride + i] and sin[t * stride + i]:
 *     (x, y) -> (fl32(fl32(x cos) - fl32(y sin)), fl32(fl32(y cos) + fl32(x sin)))
 * in binary32, every operation rounded once.  Pair i is elements i and i + rotary_dim / 2, or, if
 * `interleaved` is nonzero, elements 2 i and 2 i + 1; elements from rotary_dim on stay as they are. */
typedef struct {
  const float* cos;      /* [device] max_positions rows, 16-byte aligned */
  const float* sin;      /* [device] likewise */
  int64_t stride;        /* elements from one position's row to the next: at least rotary_dim / 2, a multiple of 4 */
  int64_t max_positions;
  int32_t rotary_dim;    /* a multiple of 16 from 16 to head_dim */
  int32_t interleaved;
} bq_rotation;

/* bq_kv_write with the rotation on the way: the codes and maxima of the keys are those of the rotated
 * binary32 values (not rounded to `dtype` in between), bit for bit; values are written as by bq_kv_write.
 * In the same launch the tokens' queries are rotated, each element rounded once to `dtype`.
 *   k, v, k_stride, v_stride, slots
 *              as in bq_kv_write.
 *   positions  [device] one position per token, 8-byte aligned, in any order, repeats allowed (tokens of one
 *              depth of a tree).  A token whose position is outside [0, max_positions) is left out: nothing
 *              of it is written, to the cache or to q_out.
 *   q          [device] tokens rows of heads * head_dim elements of `dtype`, 16-byte aligned, or NULL: no
 *              queries (heads, the strides and q_out are not looked at then).
 *   heads      at least 1; tokens * heads * head_dim < 2^34.
 *   q_out      [device] out: rows as in q, with q_out_stride; q itself (with its stride) rotates in place.  A
 *              token whose slot is outside the pool has its queries rotated all the same.
 * q_out overlaps none of the inputs but q, and that not in part.
 * Errors: as bq_kv_write, and BQ_ERR_FORMAT (rotary_dim), BQ_ERR_SIZE (max_positions below 1, a stride too
 * short, heads, q_out == q with another stride, or a launch of more than 2^32 - 1 threads, each with
 * 8 elements of the keys or values, or 8 to 64 of the queries). */
bq_status bq_kv_append(const bq_kv_cache* cache, const bq_rotation* rotation, bq_dtype dtype, const void* k,
                       const void* v, int64_t tokens, int64_t k_stride, int64_t v_stride, const int64_t* positions,
                       const int64_t* slots, const void* q, int64_t q_stride, int32_t heads, void* q_out,
                       int64_t q_out_stride, hipStream_t stream);

/* Bytes of workspace bq_kv_tree_attention needs for this call's shape (the batch's pointers are not read); 0
 * if an argument is not valid.  It depends on the device's number of compute units. */
size_t bq_kv_tree_attention_workspace_bytes(const bq_kv_cache* cache, const bq_kv_batch* batch, bq_dtype dtype,
                                            int32_t heads);

/* bq_kv_attention for new tokens that are a tree.  New token i of a sequence's n (its key in place
 * kv_len - n + i, like theirs in bq_kv_attention) has a parent among those before it, or follows the context, the
 * kv_len - n keys before the draft.  It stands at position kv_len - n + depth, its depth the number of its
 * ancestors in the draft, and sees the context, its ancestors and itself; of these, if window > 0, those
 * at positions above its own minus window.
 *   parents    [device] one per row of q, 4-byte aligned: the number (0 .. i - 1) of the parent among the
 *              sequence's new tokens, or -1: it follows the context.  Any other number marks an unused place:
 *              that token and all that descend from it see no key and give zeros, and -infinity in lse.  What
 *              is cached in an unused place does not matter (it may be NaN).
 *   batch      max_q_len at most 256.
 * Everything else, the rounding and the errors are as in bq_kv_attention; the workspace is that of
 * bq_kv_tree_attention_workspace_bytes. */
bq_status bq_kv_tree_attention(const bq_kv_cache* cache, const bq_kv_batch* batch, const int32_t* parents,
                               bq_dtype dtype, const void* q, int64_t q_stride, int32_t heads, float scale,
                               int32_t window, void* out, int64_t out_stride, float* lse, void* workspace,
                               size_t workspace_bytes, hipStream_t stream);

/* Keeps the accepted path of each sequence's draft: the cached keys and values of its new token path[i] move to the
 * place of new token i, codes and maxima as they are (along a path, position and depth agree, so rotated keys stay
 * right).  With m accepted tokens the sequence's length is then kv_len - n + m: the caller's to set.  Places of
 * the draft from m on keep what they held.
 *   batch      as of the tree attention (q_start, kv_len, page_table; any max_q_len).
 *   path       [device] num_seqs rows of numbers of new tokens, 4-byte aligned, strictly ascending (0 <= path[i] < n);
 *              at an entry that is not, the row ends.
 *   path_stride  entries from one row to the next, at least 0 (0: one row for all).
 *   path_len   [device] num_seqs, 4-byte aligned: entries of each row, read as at most the sequence's new tokens.
 * A token whose place, old or new, is on a page outside the pool is not moved.  No two sequences share a page of
 * their drafts.
 * Errors: as bq_kv_write (of the batch: a negative count or length, num_seqs > 65535, kv_heads above 2^20).  tokens or
 * num_seqs of 0 enqueue nothing. */
bq_status bq_kv_tree_accept(const bq_kv_cache* cache, const bq_kv_batch* batch, const int32_t* path,
                            int64_t path_stride, const int32_t* path_len, hipStream_t stream);

/* The hipError_t (as int) of the most recent launch that failed on the calling thread with
 * BQ_ERR_HIP, or 0 if none has. */
int bq_last_hip_error(void);

/* Static description of a status code (never NULL). */
const char* bq_status_string(bq_status status);

#ifdef __cplusplus
}
#endif

#endif /* BQ_H */
