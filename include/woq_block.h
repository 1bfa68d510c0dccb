/*
 * woq_block.h - C ABI of the parts of a decoder block around its linears on NVIDIA GB300
 * (sm_103a): the norms before and after a block with its gate and residual scale, the routing of
 * rows to experts, and the experts' products over int4 or int6 weights.  They stand beside the
 * linears of woq.h (the same packed weights; "Doubling LLM token rates in ComfyUI",
 * blog.comfy.org, section "Optimizing the Linear Kernel") and take a block whose feed-forward part is a mixture
 * of experts; the arithmetic is this library's own, stated below.
 *
 * The conventions of woq.h hold (statuses, host validation before any launch, caller-owned
 * buffers, no allocation, asynchronous on the given stream, programmatic dependent launch).
 * T = 0 launches nothing.
 */
#ifndef WOQ_BLOCK_H
#define WOQ_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "woq.h"
#include "woq_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Norms before and after a block.  For each of T rows of D elements:
 *   n  = u / sqrt(mean(u^2) + eps) * (post + offset)      (post NULL: n = u)
 *   r' = alpha * r + beta * gate * n                      (gate NULL: 1)
 *   h  = r' / sqrt(mean(r'^2) + eps) * (pre + offset)     (out NULL: not formed)
 * u is a block's output (a linear's fp32 y, or bf16), r the residual stream; r' is rounded to r's
 * type into r_out (which may be r itself), h to bf16 into out.  Everything between is fp32, and
 * h is formed from r' before that rounding; mean squares have to be finite in fp32, and with eps 0 not below 2^-126 (a row of
 * zeros is).
 *   u: device bf16 or fp32 [T][D]; r, r_out: device bf16 or fp32 [T][D]; out: device bf16 [T][D];
 *   post, pre: device bf16 [D]; gate: device bf16 [gate_rows][D], row t uses gate row
 *   t / (T / gate_rows) (1: one scale per channel; T: a gate per row); T % gate_rows == 0.
 *   D % 8 == 0, 8 <= D <= 16384; T >= 0; eps >= 0.  All pointers 16-byte aligned; the buffers must not
 *   overlap, but r and r_out may be one and the same.
 * Errors: WOQ_ERR_NULL (pre missing where out is given among them), WOQ_ERR_ALIGN, WOQ_ERR_SHAPE, WOQ_ERR_CUDA.
 * --------------------------------------------------------------------------- */
WOQ_API int woq_block_norm(const void* u, int u_dtype, const void* r, void* r_out, int r_dtype, void* out, int T, int D,
                           const void* post, const void* gate, int gate_rows, const void* pre, float alpha, float beta,
                           float offset, float eps, woq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Routing of T rows to k of E experts each.  logits: device bf16 or fp32 [T][row_stride] (the
 * router linear's y), E of them a row.  For each row:
 *   s_i = e^l_i / sum_j e^l_j (WOQ_ROUTE_SOFTMAX) or 1 / (1 + e^-l_i) (WOQ_ROUTE_SIGMOID);
 *   c_i = s_i + bias_i (bias NULL: 0); an expert with l_i = -inf is never chosen.
 *   groups > 1: the experts stand in `groups` equal runs; a run's score is its largest c
 *   (group_best 1) or the sum of its two largest (2; less than two that may be chosen: -inf), and only the top_groups runs
 *   of highest score keep their experts.
 *   The k largest c are chosen, in descending order; ties (of groups too) go to the lower number.
 *   Their weights are s_i, divided by their sum if renormalise, times scale.
 * ids: device int32 [T][k]; weights: device fp32 [T][k].  Places left over (fewer than k experts may be
 * chosen) get id -1 and weight 0, as do all places of rows from *live on (device int32; NULL: T).
 * A NaN logit counts as the largest, and makes the weights of its row's chosen NaN; so does +inf under softmax.
 * The choice is that of scores formed in fp64: they are compared in fp32 where they are further apart than its error, else in
 * fp64 (where sigmoids of logits above 36 can tie under a bias).  bias finite.
 *   1 <= E <= 1024; 1 <= k <= 32, k <= E; groups 1 .. 32 divides E; 1 <= top_groups <= groups, k <= top_groups * E / groups;
 *   group_best 1 or 2 (2: E / groups >= 2); scale finite; row_stride >= E.  logits 16-byte aligned, the others 4.
 * Errors: WOQ_ERR_NULL, WOQ_ERR_ALIGN, WOQ_ERR_SHAPE, WOQ_ERR_CUDA.
 * --------------------------------------------------------------------------- */
enum { WOQ_ROUTE_SOFTMAX = 0, WOQ_ROUTE_SIGMOID = 1 };

typedef struct {
  int score;       /* WOQ_ROUTE_SOFTMAX or WOQ_ROUTE_SIGMOID */
  int experts;     /* E */
  int k;           /* experts of a row */
  int groups;      /* 1: none */
  int top_groups;  /* groups kept (1 with groups = 1) */
  int group_best;  /* members of a group that make its score: 1 or 2 */
  int renormalise; /* 0 or 1 */
  float scale;
} woq_router;

WOQ_API int woq_route(const woq_router* cfg, const void* logits, int dtype, int row_stride, int T, const float* bias,
                      const int32_t* live, int32_t* ids, float* weights, woq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Experts: y_t = sum_j w_tj D_e (silu(G_e x_t) * U_e x_t), e = ids_tj, for T rows of k places.
 *   gate_up: device, E packed matrices of (bits, 2 I, H), rows 0 .. I-1 the gate G, I .. 2 I-1 the up projection U, as
 *   for woq_w4a8_linear_swiglu_f32; down: device, E packed matrices of (bits, H, I).  The matrices lie one
 *   behind the other, each as its packer wrote it (woq_packed_bytes, a multiple of 256).
 *   x: device bf16 [T][H]; ids: device int32 [T][k]; weights: device fp32 [T][k] (woq_route's, or any: an expert may
 *   stand in a row twice); y: device bf16 [T][H].  A place with id -1 has no part in y (a row without any gives 0);
 *   so has one with an id outside [-1, E), which sets WOQ_DEVERR_STATE in the workspace.
 *   Activations are not quantised to 8 bits as the linears': an x is taken as the sum of two 8-bit floats (e4m3) under a power of two
 *   for each row and group of 128 elements, exactly but for elements below 2^-13 of the group's largest, which are off by at most 2^-17 of that; h = silu(g) * u
 *   is taken so too, rounded to at most 2^-8 of itself.  Products are exact, sums fp32, a group of 128 times its scale in
 *   fp32, y rounded once.  |x| below 2^100; a row whose gate or up, or their
 *   product, passes fp32's range gets NaN.  What a row gives does not depend on the run, nor on the other rows' x and weights; the
 *   order of its sums goes by the ids of all rows of the call (how many places each expert has), so its last bits can go by those.
 *   bits 4 or 6; 1 <= E <= 1024; 1 <= k <= 32; H, I multiples of 128 in [128, 32768]; 0 <= T, T k <= 32768 (a longer
 *   prompt is cut by rows into several calls).
 *   ws: device, 16-byte aligned, woq_experts_workspace(...) bytes, zero-filled once before first use
 *   (woq_workspace_init); launches of different shapes may use one that is large enough, launches that can overlap must not.
 *   A wait that runs out sets WOQ_DEVERR_TIMEOUT: then y is left as it was, by this call and by the next ones (which set it again,
 *   whether or not it has been cleared) until ws has been zero-filled.
 *   A chosen expert with a packed matrix whose header does not match sets WOQ_DEVERR_HEADER (woq_read_status(ws, ...)), and
 *   the rows of y that chose it are left as they were.
 * Errors: WOQ_ERR_NULL, WOQ_ERR_ALIGN, WOQ_ERR_SHAPE, WOQ_ERR_LAYOUT (gate_up_bytes or down_bytes too
 * small), WOQ_ERR_WORKSPACE, WOQ_ERR_CUDA.
 * --------------------------------------------------------------------------- */

/* Bytes of E packed matrices of (bits, N, K) one behind the other; 0 if the shape is invalid. */
WOQ_API size_t woq_experts_bytes(int bits, int E, int N, int K);

/* Bytes of workspace of woq_experts_swiglu; 0 if the shape is invalid. */
WOQ_API size_t woq_experts_workspace(int E, int T, int k, int H, int I);

WOQ_API int woq_experts_swiglu(int bits, int E, const void* gate_up, size_t gate_up_bytes, const void* down,
                               size_t down_bytes, const void* x_bf16, const int32_t* ids, const float* weights, int T,
                               int k, int H, int I, void* y_bf16, void* ws, size_t ws_bytes, woq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WOQ_BLOCK_H */
