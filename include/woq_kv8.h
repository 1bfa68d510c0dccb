/*
 * woq_kv8.h - C ABI of the 8-bit key/value cache between the qkv linear and the o linear of a
 * decode step on NVIDIA GB300 (sm_103a): rotary positions and append, attention, and the page
 * operations.  "Doubling LLM token rates in ComfyUI" (blog.comfy.org): section "Paying
 * attention to the attention!" (a split key/value decode attention for one or a few query rows
 * whose draft rows are masked causally, and a cache held in 8 bits) and section "Adaptive tree
 * MTP" (eight rows per verify pass); the arithmetic is this library's own, stated below.
 *
 * The conventions of woq.h hold (statuses, host validation before any launch, caller-owned
 * buffers, no allocation, asynchronous on the given stream).  In addition:
 *   - A cache is ONE device buffer of woq_kv8_bytes(cfg) bytes, initialised by woq_kv8_init and
 *     passed to every call with the same woq_kv8_config.  Its lengths and page tables live in
 *     it and are changed on the device only, so every call can be captured in a CUDA graph.
 *   - What only the device can see (sequence numbers, kept rows, positions, free pages) is
 *     checked by the kernels.  A call that fails such a check sets a bit of the cache's status
 *     word (its first word: woq_read_status(cache, ...) reads and clears it) and changes
 *     nothing else, unless its description says otherwise.  A buffer that is not an initialised
 *     cache is left alone; one initialised for another config gets WOQ_DEVERR_HEADER.
 *   - Calls on one cache must not overlap on the GPU (one stream, or ordered by events).
 *     Calls that only read it (woq_kv8_attention with workspaces of their own, woq_kv8_read,
 *     woq_kv8_state, the source of woq_kv8_copy) may overlap each other.
 *
 * What a cache holds.  A sequence's tokens are grouped in blocks of 64.  A full block lies in a
 * page (one page: the block's keys and values of every layer and kv head); for each layer, head
 * and of keys and values separately it has one fp32 scale s and 8-bit codes:
 *   WOQ_KV8_INT8: s = RN(amax / 127), code = rne(RN(x / s)), an int8;
 *   WOQ_KV8_E4M3: s = the least power of two with amax / s <= 448 (at least 2^-126), code =
 *                 rne(x / s), an e4m3 float;
 *   amax = the largest magnitude among the 64 x head_dim bf16 values; amax = 0: s = 0, codes 0.
 * Tokens behind the last full block (at most 63), and the draft rows behind them (at most 8),
 * are held in bf16 in the sequence's tail.  So codes do not depend on how tokens arrived, draft
 * rows that are not accepted leave no trace, and a full page never changes: sequences share it.
 * A token with a key or value that is not finite makes NaN of the attention of every row that
 * sees it and, once its block is full, of every row that sees a token of that block (head by
 * head); rows that do not see it are not affected.
 */
#ifndef WOQ_KV8_H
#define WOQ_KV8_H

#include <stddef.h>
#include <stdint.h>

#include "woq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WOQ_KV8_BLOCK 64 /* tokens of a block */
#define WOQ_KV8_ROWS 8   /* most draft rows behind a sequence */

enum { WOQ_KV8_INT8 = 0, WOQ_KV8_E4M3 = 1 };
enum { WOQ_KV8_BF16 = 0, WOQ_KV8_F32 = 1 }; /* element types of qkv */

/* More bits of the status word (a cache's first word). */
#define WOQ_DEVERR_PAGES 0x4u     /* not enough free pages */
#define WOQ_DEVERR_STATE 0x8u     /* a sequence number, length or list that the call does not allow */
#define WOQ_DEVERR_POSITION 0x10u /* a position outside the rotary table */

typedef struct {
  int format;     /* WOQ_KV8_INT8 or WOQ_KV8_E4M3 */
  int layers;     /* 1 .. 1024 */
  int kv_heads;   /* 1 .. 256 */
  int head_dim;   /* 64, 128 or 256 */
  int seqs;       /* 1 .. 1024 sequences, numbered from 0 */
  int max_tokens; /* 1 .. 2^24: longest sequence */
  int pages;      /* 1 .. 2^24: pages of 64 tokens in the pool, shared by all sequences */
} woq_kv8_config;

/* Bytes of a cache; 0 if the config is invalid. */
WOQ_API size_t woq_kv8_bytes(const woq_kv8_config* cfg);

/* Make an empty cache of a buffer (16-byte aligned, at least woq_kv8_bytes(cfg) bytes).
 * Errors of this and every call below: WOQ_ERR_NULL, WOQ_ERR_ALIGN, WOQ_ERR_SHAPE (the config or
 * an argument out of range), WOQ_ERR_LAYOUT (cache_bytes too small), WOQ_ERR_CUDA. */
WOQ_API int woq_kv8_init(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, woq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Rotary positions.  Frequency i < rot_dim / 2 turns one pair of a head's elements by the angle
 * p theta^(-2 i / rot_dim), p being the row's position on axis axis_of[i] (one axis for text;
 * time, height and width for images and video, in any arrangement over the frequencies):
 *   a' = RN(RN(a c) - RN(b s)),   b' = RN(RN(b c) + RN(a s))   (fp32), then rounded to bf16.
 * Pairs: elements (i, i + rot_dim / 2), or (2 i, 2 i + 1) if interleaved.  Elements from
 * rot_dim on are only rounded to bf16.
 * --------------------------------------------------------------------------- */

/* Fill table (device fp32 [positions][rot_dim / 2][2]: cos, sin), from angles worked out in 64
 * bits; once per model.  rot_dim a multiple of 4 in [4, 256], positions >= 0, theta > 0. */
WOQ_API int woq_rope_table(double theta, int rot_dim, int positions, float* table, woq_stream_t stream);

typedef struct {
  const float* table;     /* device, 16-byte aligned, from woq_rope_table; NULL: no rotation */
  int positions;          /* rows of the table */
  int rot_dim;            /* as the table was made; at most head_dim */
  int interleaved;        /* 0 or 1 */
  int axes;               /* 1 .. 4 */
  const int32_t* pos;     /* device int32 [axes][rows of the call]: 0 <= pos < positions */
  const uint8_t* axis_of; /* HOST [rot_dim / 2], each < axes; read during the call; NULL: all 0 */
} woq_rope;

/* ---------------------------------------------------------------------------
 * Append.  qkv: device [rows][row_stride] of bf16 or fp32 (a qkv linear's y), each row q_heads
 * query heads, then kv_heads keys, then kv_heads values, head_dim elements each; 16-byte
 * aligned, row_stride (elements) a multiple of 8 and at least (q_heads + 2 kv_heads) head_dim.
 * Queries and keys are rotated (rope NULL: not), everything is rounded to bf16; queries go to
 * q_out (device bf16 [rows][q_heads][head_dim]; q_heads = 0 and q_out NULL: none), keys and
 * values into layer `layer` of the cache.  A row whose position is outside the table sets
 * WOQ_DEVERR_POSITION and is rotated as by position 0.  seqs (device int32 [n], n <= 1024; NULL: 0 .. n-1)
 * names the sequences; the lists' entries must differ.
 * --------------------------------------------------------------------------- */

/* `rows` (1 .. 8) draft rows behind each of n sequences (a plain decode step: 1 row, accepted
 * after it); rows of qkv and q_out are entry-major [n][rows].  They replace the draft rows
 * there were, and the lengths do not change.  An entry that is out of range or repeats an
 * earlier one is left out (WOQ_DEVERR_STATE; its q_out rows are not written).
 * Launched with programmatic dependent launch, like the linears. */
WOQ_API int woq_kv8_append_rows(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer,
                                const int32_t* seqs, int n, int rows, const void* qkv, int dtype, int row_stride,
                                int q_heads, const woq_rope* rope, void* q_out, woq_stream_t stream);

/* Take the draft rows whose bits are set in keep[e] (device uint32 [n]; bit j: row j; in order;
 * what the accepted row sees) into sequence e, in every layer; a block that becomes full is
 * quantised into the free page of lowest number.  Bits above 7 are not allowed
 * (WOQ_DEVERR_STATE); as is a sequence that would exceed max_tokens.  All entries or none. */
WOQ_API int woq_kv8_accept(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, const int32_t* seqs, int n,
                           const uint32_t* keep, woq_stream_t stream);

/* Make room for `tokens` more tokens of sequence seq (the prompt), in every layer: pages are
 * taken (lowest numbers first) and the length grows.  Then woq_kv8_append_prompt must fill each
 * layer once, before the sequence is used otherwise.  A refused one (WOQ_DEVERR_STATE: longer than
 * max_tokens; WOQ_DEVERR_PAGES) changes nothing, but that a prompt before it of as many tokens
 * is over: what is then filled could not be told from the refused one's, and is refused too. */
WOQ_API int woq_kv8_extend(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int seq, int tokens,
                           woq_stream_t stream);

/* Fill the `tokens` last tokens of sequence seq, in one layer.  tokens must be what the
 * sequence's last woq_kv8_extend (refused ones aside) was given, with no accept, fork or free of it since
 * (WOQ_DEVERR_STATE otherwise, and then nothing is written but q_out). */
WOQ_API int woq_kv8_append_prompt(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer, int seq,
                                  int tokens, const void* qkv, int dtype, int row_stride, int q_heads,
                                  const woq_rope* rope, void* q_out, woq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of `rows` rows of each of n sequences (the draft rows' queries).
 *   q, out: device bf16 [n][rows][q_heads][head_dim]; q_heads a multiple of kv_heads, query head
 *   i reads kv head i / (q_heads / kv_heads); rows * q_heads / kv_heads <= 128;
 *   n * kv_heads * c * (ceil(max_tokens / 64) + 8) < 2^31 - 2^16, where c is the number of
 *   parts that rows * q_heads / kv_heads queries are worked on in (1 up to 40, else up to 4;
 *   head_dim 256: one for each 16).
 *   vis: device uint32 [n][rows], bit j: draft row j is seen (bits 0 .. 7); NULL: row m sees
 *   draft rows 0 .. m.  Only rows that were appended may be seen.
 *   A row sees, in this order, the sequence's tokens and the draft rows of its vis; with
 *   window > 0 only the first `sinks` and the last `window` of them (window 0: all, sinks not
 *   used; window, sinks <= 2^30).  out = sum_j softmax_j(scale q . k_j) v_j over what it sees, rounded to bf16; a row
 *   that sees nothing gives 0.  Scores, maxima and sums are fp32 and 8-bit codes exact; fewer bits are held of
 *   queries against 8-bit keys (f16 under the row's power of two: exact but for elements below 2^-17 of the row's
 *   largest, rounded to multiples of 2^-24 of it), and of the weights in the product with the
 *   values (f16, 11 significant bits; 16 for tokens and draft rows that are held in bf16).
 *   scale finite; q finite; sums of |q_i k_i| and scale times them below 2^100, sums of |v| over
 *   the tokens seen below 2^127.
 *   seqs: as above, but entries may repeat; one out of range gives 0 and WOQ_DEVERR_STATE.
 *   ws: device, 16-byte aligned, woq_kv8_attention_workspace(...) bytes, zero-filled once before
 *   first use (woq_workspace_init); each launch leaves zero what has to be, so launches of
 *   different shapes may use one that is large enough.  Not shared by launches that can overlap.
 *   A wait that runs out sets WOQ_DEVERR_TIMEOUT: rows of out whose result is not complete keep what they held, and ws
 *   has to be zero-filled before it is used again.
 * The result does not depend on the run (fixed order of summation).  Launched with
 * programmatic dependent launch.
 * --------------------------------------------------------------------------- */
WOQ_API size_t woq_kv8_attention_workspace(const woq_kv8_config* cfg, int n, int rows, int q_heads);
WOQ_API int woq_kv8_attention(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer,
                              const int32_t* seqs, int n, int rows, const void* q, int q_heads, const uint32_t* vis,
                              float scale, int window, int sinks, void* out, void* ws, size_t ws_bytes,
                              woq_stream_t stream);

/* The attention's launch shape for n sequences of `rows` rows, worked out on the host without launching
 * anything; sms, smem_max: the device to plan for (0 for either = the current device's value).
 * WOQ_ERR_NULL, WOQ_ERR_SHAPE (arguments that woq_kv8_attention refuses, or nothing fits smem_max),
 * WOQ_ERR_CUDA. */
typedef struct {
  int ctas;         /* grid: one CTA per SM; those beyond the work end at once */
  int warps;        /* consumer warps of a CTA (one more copies) */
  int query_groups; /* warps that read the same block: 1, or a team of 4 that shares it out */
  int stages;       /* ring stages of one block each: a multiple of warps / query_groups */
  int least_units;  /* blocks (and tails) a CTA takes at least */
  int smem_bytes;   /* dynamic shared memory of a CTA */
} woq_kv8_plan;
WOQ_API int woq_kv8_plan_attention(const woq_kv8_config* cfg, int n, int rows, int q_heads, int sms, int smem_max,
                                   woq_kv8_plan* out);

/* ---------------------------------------------------------------------------
 * Pages
 * --------------------------------------------------------------------------- */

/* Sequence dst[e] becomes a copy of src[e] (device int32 [n], n <= 1024), draft rows included:
 * full blocks are shared, the tail is copied, in every layer.  Each dst must be empty, named
 * once and no src; a src may repeat.  All entries or none. */
WOQ_API int woq_kv8_fork(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, const int32_t* src,
                         const int32_t* dst, int n, woq_stream_t stream);

/* Empty the sequences (device int32 [n], n <= 1024, each named once); pages that no sequence
 * holds any more become free.  All entries or none. */
WOQ_API int woq_kv8_free(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, const int32_t* seqs, int n,
                         woq_stream_t stream);

/* Sequence dst_seqs[e] of cache dst becomes a copy of src_seqs[e] of cache src with pages of its
 * own (lowest free numbers first, in the order of the list).  The caches may be one and the
 * same, or must not overlap; their configs may differ in seqs, max_tokens and pages only
 * (WOQ_ERR_SHAPE).  Conditions on dst as for woq_kv8_fork; a pair that does not fit sets
 * WOQ_DEVERR_PAGES or WOQ_DEVERR_STATE in dst, a source that is no cache of src_cfg WOQ_DEVERR_HEADER
 * in dst.  All entries or none. */
WOQ_API int woq_kv8_copy(const woq_kv8_config* src_cfg, const void* src, size_t src_bytes,
                         const woq_kv8_config* dst_cfg, void* dst, size_t dst_bytes, const int32_t* src_seqs,
                         const int32_t* dst_seqs, int n, woq_stream_t stream);

/* Move every page in use at or above `limit` (1 .. cfg->pages) into free pages below it (the
 * k-th such page into the k-th free one) and use only pages below `limit` from here on, so that
 * the memory of the pool's end is the caller's until a later call raises the limit again
 * (woq_kv8_page_offset says where it starts).  WOQ_DEVERR_PAGES, and no change, if they do not fit. */
WOQ_API int woq_kv8_compact(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int limit,
                            woq_stream_t stream);

/* Byte offset of page `page` (0 .. cfg->pages) in the cache buffer; pages lie one behind the
 * other up to woq_kv8_bytes(cfg).  0 for invalid arguments. */
WOQ_API size_t woq_kv8_page_offset(const woq_kv8_config* cfg, int page);

/* Tokens first .. first + count - 1 of a sequence, back in bf16 (code * s rounded to fp32 and then
 * to bf16, or as held in the tail; of a token that was not finite the value is 0 and the key NaN,
 * and so are the other keys of its block and head once the block is full): k, v device bf16
 * [layers read][count][kv_heads][head_dim], 16-byte aligned.  layer -1: all layers.  Places up to 7 behind the sequence's end are its draft rows; if
 * first + count goes beyond them nothing is written (WOQ_DEVERR_STATE). */
WOQ_API int woq_kv8_read(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer, int seq, int first,
                         int count, void* k, void* v, woq_stream_t stream);

/* Copies of the cache's bookkeeping into device buffers (each may be NULL): lens int32 [seqs];
 * refs int32 [pages], how many sequences hold each page; table int32 [seqs][ceil(max_tokens /
 * 64)], the pages of each sequence's full blocks (entries behind them: unspecified). */
WOQ_API int woq_kv8_state(const woq_kv8_config* cfg, const void* cache, size_t cache_bytes, int32_t* lens,
                          int32_t* refs, int32_t* table, woq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WOQ_KV8_H */
