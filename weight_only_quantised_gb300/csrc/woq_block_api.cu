// C ABI of the parts of a block around its linears (include/woq_block.h): argument checks and layout.
#include <math.h>

#include "woq_block.h"
#include "woq_block_internal.h"
#include "woq_internal.h"
#include "woq_layout.h"

namespace woq {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool known_type(int t) { return t == WOQ_KV8_BF16 || t == WOQ_KV8_F32; }

// Where the parts of the experts' workspace lie.  What has to be zero between launches comes first and lies in the same place for every shape, so launches of different shapes may share a workspace.
struct ExpertsLayout {
  size_t split_counts, split_sums, item, order, x_halves, x_meta, h_halves, h_meta, parts, total;
  int item_rows;
};

// Rows of an item: the fewest columns of B that hold what an expert has where every one is as likely (16 at most with int6: its two
// sums a column fill tensor memory).  A wider item costs more for few rows, a second item of an expert its weights once more.  int4, 128 experts
// of 2048 x 768, k 8, in us with items of 8 / 16 / 32 rows: 4.1 rows an expert 77 / 79 / 98, 6.0 83 / 88 / 107, 8.0 101 / 92 / 111,
// 12 126 / 100 / 118, 16 155 / 125 / 126 (so the crossings lie nearer to 7 and 16 than the rule has them).
int choose_item_rows(int E, size_t n) {
  const double rows = n / (E * (1.0 - pow(1.0 - 1.0 / E, (double)n)));
  return rows <= 6.0 ? 8 : rows <= 12.0 ? 16 : 32;
}

bool experts_layout(int E, int T, int k, int H, int I, ExpertsLayout* l) {
  if (E < 1 || E > 1024 || k < 1 || k > 32 || T < 0 || (long long)T * k > kMostEntries) return false;
  for (const int d : {H, I})
    if (d < kGroup || d > 32768 || d % kGroup) return false;
  const size_t n = (size_t)T * k;
  l->item_rows = choose_item_rows(E, n);
  // an item holds kLeastItemRows places of one expert at least, an expert's last one fewer
  const size_t most = n / kLeastItemRows + (size_t)E;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  l->split_counts = take((size_t)kMostCtas * 4);
  l->split_sums = take((size_t)kMostCtas * 2 * l->item_rows * 256 * 4);
  l->item = take((n < most ? n : most) * sizeof(ExpertItem));
  l->order = take(n * 4);
  l->x_halves = take((size_t)T * H * 2);
  l->x_meta = take((size_t)T * (H / kGroup) * 8);
  l->h_halves = take(n * I * 2);
  l->h_meta = take(n * (I / kGroup) * 8);
  l->parts = take(n * H * 4);
  l->total = at;
  return true;
}

}  // namespace
}  // namespace woq

using namespace woq;

extern "C" {

int woq_block_norm(const void* u, int u_dtype, const void* r, void* r_out, int r_dtype, void* out, int T, int D,
                   const void* post, const void* gate, int gate_rows, const void* pre, float alpha, float beta,
                   float offset, float eps, woq_stream_t stream) {
  if (!known_type(u_dtype) || !known_type(r_dtype) || T < 0 || D < 8 || D > 16384 || D % 8) return WOQ_ERR_SHAPE;
  if (!isfinite(alpha) || !isfinite(beta) || !isfinite(offset) || !isfinite(eps) || eps < 0.0f) return WOQ_ERR_SHAPE;
  if (gate && (gate_rows < 1 || T % gate_rows)) return WOQ_ERR_SHAPE;
  if (T == 0) return WOQ_OK;
  if (!u || !r || !r_out || (out && !pre)) return WOQ_ERR_NULL;
  for (const void* p : {u, r, (const void*)r_out, (const void*)out, post, gate, pre})
    if (!aligned(p, 16)) return WOQ_ERR_ALIGN;
  BlockNorm a = {};
  a.u = u;
  a.r = r;
  a.r_out = r_out;
  a.out = static_cast<uint16_t*>(out);
  a.post = static_cast<const uint16_t*>(post);
  a.gate = static_cast<const uint16_t*>(gate);
  a.pre = static_cast<const uint16_t*>(pre);
  a.u_f32 = u_dtype == WOQ_KV8_F32;
  a.r_f32 = r_dtype == WOQ_KV8_F32;
  a.rows = T;
  a.dim = D;
  a.rows_per_gate = gate ? T / gate_rows : 1;
  a.alpha = alpha;
  a.beta = beta;
  a.offset = offset;
  a.eps = eps;
  a.inv_dim = 1.0f / (float)D;
  return cuda_result(launch_block_norm(a, (cudaStream_t)stream));
}

int woq_route(const woq_router* cfg, const void* logits, int dtype, int row_stride, int T, const float* bias,
              const int32_t* live, int32_t* ids, float* weights, woq_stream_t stream) {
  if (!cfg) return WOQ_ERR_NULL;
  const woq_router& c = *cfg;
  if (c.score != WOQ_ROUTE_SOFTMAX && c.score != WOQ_ROUTE_SIGMOID) return WOQ_ERR_SHAPE;
  if (!known_type(dtype) || T < 0 || c.experts < 1 || c.experts > 1024 || row_stride < c.experts) return WOQ_ERR_SHAPE;
  if (c.groups < 1 || c.groups > 32 || c.experts % c.groups || c.top_groups < 1 || c.top_groups > c.groups) return WOQ_ERR_SHAPE;
  const int size = c.experts / c.groups;
  if ((c.group_best != 1 && c.group_best != 2) || c.group_best > size) return WOQ_ERR_SHAPE;
  if (c.k < 1 || c.k > 32 || c.k > c.top_groups * size) return WOQ_ERR_SHAPE;
  if ((c.renormalise != 0 && c.renormalise != 1) || !isfinite(c.scale)) return WOQ_ERR_SHAPE;
  if (T == 0) return WOQ_OK;
  if (!logits || !ids || !weights) return WOQ_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(live, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return WOQ_ERR_ALIGN;
  Route a = {};
  a.logits = logits;
  a.bias = bias;
  a.live = live;
  a.ids = ids;
  a.weights = weights;
  a.stride = row_stride;
  a.f32 = dtype == WOQ_KV8_F32;
  a.softmax = c.score == WOQ_ROUTE_SOFTMAX;
  a.rows = T;
  a.experts = c.experts;
  a.k = c.k;
  a.groups = c.groups;
  a.group_size = size;
  a.top_groups = c.top_groups;
  a.group_best = c.group_best;
  a.renormalise = c.renormalise;
  a.scale = c.scale;
  return cuda_result(launch_route(a, (cudaStream_t)stream));
}

size_t woq_experts_bytes(int bits, int E, int N, int K) {
  if (E < 1 || E > 1024) return 0;
  return packed_bytes(bits, N, K) * (size_t)E;
}

size_t woq_experts_workspace(int E, int T, int k, int H, int I) {
  ExpertsLayout l;
  return experts_layout(E, T, k, H, I, &l) ? l.total : 0;
}

int woq_experts_swiglu(int bits, int E, const void* gate_up, size_t gate_up_bytes, const void* down, size_t down_bytes,
                       const void* x_bf16, const int32_t* ids, const float* weights, int T, int k, int H, int I,
                       void* y_bf16, void* ws, size_t ws_bytes, woq_stream_t stream) {
  ExpertsLayout l;
  if ((bits != 4 && bits != 6) || !experts_layout(E, T, k, H, I, &l)) return WOQ_ERR_SHAPE;
  if (T == 0) return WOQ_OK;
  if (!gate_up || !down || !x_bf16 || !ids || !weights || !y_bf16 || !ws) return WOQ_ERR_NULL;
  for (const void* p : {gate_up, down, x_bf16, (const void*)y_bf16, (const void*)ws})
    if (!aligned(p, 16)) return WOQ_ERR_ALIGN;
  if (!aligned(ids, 4) || !aligned(weights, 4)) return WOQ_ERR_ALIGN;
  Experts a = {};
  a.gate_up_stride = packed_bytes(bits, 2 * I, H);
  a.down_stride = packed_bytes(bits, H, I);
  if (gate_up_bytes < a.gate_up_stride * E || down_bytes < a.down_stride * E) return WOQ_ERR_LAYOUT;
  if (ws_bytes < l.total) return WOQ_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.gate_up = static_cast<const uint8_t*>(gate_up);
  a.down = static_cast<const uint8_t*>(down);
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.ids = ids;
  a.weights = weights;
  a.y = static_cast<uint16_t*>(y_bf16);
  a.bits = bits;
  a.experts = E;
  a.rows = T;
  a.k = k;
  a.hidden = H;
  a.inner = I;
  a.entries = T * k;
  a.item_rows = bits == 6 && l.item_rows > 16 ? 16 : l.item_rows;
  a.wait_ns = wait_bound_ns();
  a.fault_cta = fault_cta(1);
  a.status = reinterpret_cast<uint32_t*>(w);
  a.split_counts = reinterpret_cast<uint32_t*>(w + l.split_counts);
  a.split_sums = reinterpret_cast<float*>(w + l.split_sums);
  a.item = reinterpret_cast<ExpertItem*>(w + l.item);
  a.order = reinterpret_cast<int32_t*>(w + l.order);
  a.x_halves = w + l.x_halves;
  a.x_meta = reinterpret_cast<float2*>(w + l.x_meta);
  a.h_halves = w + l.h_halves;
  a.h_meta = reinterpret_cast<float2*>(w + l.h_meta);
  a.parts = reinterpret_cast<float*>(w + l.parts);
  return cuda_result(launch_experts(a, (cudaStream_t)stream));
}

}  // extern "C"
