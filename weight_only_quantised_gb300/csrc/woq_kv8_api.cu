// C ABI of the 8-bit cache (include/woq_kv8.h): argument checks, layout and launch shapes.
#include <math.h>

#include <algorithm>

#include "woq_internal.h"
#include "woq_kv8_attn.cuh"

namespace woq {

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Fills v (base excepted); false if the config is out of range.
bool make_view(const woq_kv8_config& c, Kv8View* v) {
  if (c.format != WOQ_KV8_INT8 && c.format != WOQ_KV8_E4M3) return false;
  if (c.layers < 1 || c.layers > 1024 || c.kv_heads < 1 || c.kv_heads > 256) return false;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return false;
  if (c.seqs < 1 || c.seqs > kKv8MaxSeqs || c.max_tokens < 1 || c.max_tokens > 1 << 24) return false;
  if (c.pages < 1 || c.pages > 1 << 24) return false;
  v->base = nullptr;
  v->fmt = c.format;
  v->layers = c.layers;
  v->heads = c.kv_heads;
  v->dim = c.head_dim;
  v->seqs = c.seqs;
  v->max_tokens = c.max_tokens;
  v->pages = c.pages;
  v->blocks = (c.max_tokens + kKv8Block - 1) / kKv8Block;
  uint32_t h = 2166136261u;  // FNV-1a over the config's words
  for (int x : {c.format, c.layers, c.kv_heads, c.head_dim, c.seqs, c.max_tokens, c.pages}) h = (h ^ (uint32_t)x) * 16777619u;
  v->hash = h;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  v->lens = take((size_t)c.seqs * 4);
  v->reserved = take((size_t)c.seqs * 4);
  v->refs = take((size_t)c.pages * 4);
  v->map = take((size_t)c.pages * 4);
  v->moves = take((size_t)kKv8MaxSeqs * 16);
  v->pairs = take((size_t)(c.pages + 1) * 8);
  v->table = take((size_t)c.seqs * v->blocks * 4);
  v->tails = take((size_t)c.layers * c.seqs * c.kv_heads * v->tail_elems() * 2);
  v->pool = at;
  v->total = at + (size_t)c.pages * v->page_bytes();
  return true;
}

// The checks that every call on a cache makes.
int open_cache(const woq_kv8_config* cfg, const void* cache, size_t cache_bytes, Kv8View* v) {
  if (!cfg) return WOQ_ERR_NULL;
  if (!make_view(*cfg, v)) return WOQ_ERR_SHAPE;
  if (!cache) return WOQ_ERR_NULL;
  if (!aligned(cache, 16)) return WOQ_ERR_ALIGN;
  if (cache_bytes < v->total) return WOQ_ERR_LAYOUT;
  v->base = static_cast<uint8_t*>(const_cast<void*>(cache));
  return WOQ_OK;
}

int check_list(const void* list, int n, bool required) {
  if (n < 0 || n > kKv8MaxSeqs) return WOQ_ERR_SHAPE;
  if (n > 0 && required && !list) return WOQ_ERR_NULL;
  return aligned(list, 4) ? WOQ_OK : WOQ_ERR_ALIGN;
}

int fill_append(const Kv8View& v, int layer, const void* qkv, int dtype, int row_stride, int q_heads,
                const woq_rope* rope, void* q_out, Kv8Append* p) {
  if (layer < 0 || layer >= v.layers || (dtype != WOQ_KV8_BF16 && dtype != WOQ_KV8_F32)) return WOQ_ERR_SHAPE;
  if (q_heads < 0 || q_heads > 4096 || row_stride % 8 ||
      (long long)row_stride < (long long)(q_heads + 2 * v.heads) * v.dim)
    return WOQ_ERR_SHAPE;
  if (!qkv || (q_heads > 0 && !q_out)) return WOQ_ERR_NULL;
  if (!aligned(qkv, 16) || !aligned(q_out, 16)) return WOQ_ERR_ALIGN;
  *p = Kv8Append{};
  p->v = v;
  p->qkv = qkv;
  p->q_out = static_cast<uint16_t*>(q_out);
  p->row_stride = row_stride;
  p->layer = layer;
  p->q_heads = q_heads;
  p->f32 = dtype == WOQ_KV8_F32;
  if (rope && rope->table) {
    if (rope->rot_dim < 4 || rope->rot_dim > v.dim || rope->rot_dim % 4 || rope->positions < 1 || rope->axes < 1 ||
        rope->axes > 4 || (rope->interleaved != 0 && rope->interleaved != 1))
      return WOQ_ERR_SHAPE;
    if (!rope->pos) return WOQ_ERR_NULL;
    if (!aligned(rope->table, 16) || !aligned(rope->pos, 4)) return WOQ_ERR_ALIGN;
    p->rope.table = rope->table;
    p->rope.pos = rope->pos;
    p->rope.positions = rope->positions;
    p->rope.half = rope->rot_dim / 2;
    p->rope.interleaved = rope->interleaved;
    p->rope.axes = rope->axes;
    for (int i = 0; i < p->rope.half; ++i) {
      p->rope.axis_of[i] = rope->axis_of ? rope->axis_of[i] : 0;
      if (p->rope.axis_of[i] >= rope->axes) return WOQ_ERR_SHAPE;
    }
  }
  return WOQ_OK;
}

constexpr int kMostQueries = 128;  // of one kv head

// Parts that rows * group queries are worked on in.
int attn_chunks(int dim, int queries) {
  const int most = kv8::team_tiles(dim);
  return ((queries + 7) / 8 + most - 1) / most;
}

// What the attention takes of sequences, rows and heads (its unit counts fit 32 bits).
bool attn_shape_ok(const Kv8View& v, int n, int rows, int q_heads) {
  return n >= 0 && n <= kKv8MaxSeqs && rows >= 1 && rows <= WOQ_KV8_ROWS && q_heads >= 1 && q_heads <= 4096 &&
         q_heads % v.heads == 0 && rows * (q_heads / v.heads) <= kMostQueries &&
         (long long)n * v.heads * attn_chunks(v.dim, rows * (q_heads / v.heads)) * (v.blocks + kv8::kTailUnits) <= 0x7FFF0000ll;
}

// Workspace of the attention: [256 B: word 1 says that a wait ran out][tickets][where parts are][parts].  What has to be zero at the
// beginning of a launch, that word and the tickets, lies in the same place for every shape, so launches of different shapes may share a workspace.
size_t attn_joins_offset(int sms) { return 256 + ((size_t)sms * 4 + 255) / 256 * 256; }
size_t attn_parts_offset(const Kv8View& v, int n, int chunks, int sms) {
  return attn_joins_offset(sms) + ((size_t)n * v.heads * chunks * 8 + 255) / 256 * 256;
}

}  // namespace

// A team per block for more than 8 queries, in chunks of at most 40 (head_dim 256: 16), and for head_dim 256; else a warp per
// block, and as many warps as leave each two stages of the ring at least.
// 8 heads x 32,768 tokens, head_dim 128: 12 queries 24 us (a warp per block: 48), 24 29 (61), 40 36 (86); and in two
// chunks of 24 or 32 queries, four of 32: 48 queries 45 us (89), 64 53 (116), 128 103 (220).  head_dim 256: 32 queries
// 67 us (130), 4 35 (45).  Up to 8 queries of head_dim 128 the other way round: 131,072 tokens x 5 queries 57 us in
// teams, 50 in warps, 1,000 tokens 11.5 and 10.4; head_dim 64, 65,536 x 7 29 and 26.
//
// The stages are a multiple of the warps (the teams).  Block b goes to warp (team) b % per and to stage
// b % stages, so then a stage always serves the same.  Otherwise a warp could wait for
// block b while the copy of block b - stages, another warp's, is still under way (copies end in
// any order): a wait on a barrier's parity two phases ahead returns at once.
int kv8_attn_plan(Kv8Attn* p, int smem_max) {
  const int queries = p->rows * p->group, dim = p->v.dim;
  const int tiles = (queries + 7) / 8;
  p->team = tiles > 1 || dim == 256;
  p->chunks = attn_chunks(dim, queries);
  p->heads = p->v.heads * p->chunks;
  p->tiles = (tiles + p->chunks - 1) / p->chunks;
  p->queries = p->chunks > 1 ? 8 * p->tiles : queries;
  p->least_units = 8;
  const int record = 128 * dim + 16;
  if (p->team) {
    p->query_groups = 4;  // the team's warps all read its blocks
    const int teams = kv8::teams_of(dim);
    p->warps = 4 * teams;
    const int fixed = kv8::misc_bytes(p->n) + kv8::team_fixed_bytes(p->tiles, dim);
    int stages = (smem_max - fixed) / record;
    stages = (stages < kv8::kMaxStages ? stages : kv8::kMaxStages) / teams * teams;
    if (stages < 2 * teams) return 0;
    p->stages = stages;
    return fixed + stages * record;
  }
  p->query_groups = 1;
  for (int warps = kv8::kMaxWarps; warps >= 1; --warps) {
    const int fixed = kv8::misc_bytes(p->n) + kv8::merge_bytes(warps, 1, dim);
    int stages = (smem_max - fixed) / record;
    stages = (stages < kv8::kMaxStages ? stages : kv8::kMaxStages) / warps * warps;
    if (stages < 2 * warps) continue;
    p->warps = warps;
    p->stages = stages;
    return fixed + stages * record;
  }
  return 0;
}

}  // namespace woq

using namespace woq;

extern "C" {

size_t woq_kv8_bytes(const woq_kv8_config* cfg) {
  Kv8View v;
  return cfg && make_view(*cfg, &v) ? v.total : 0;
}

size_t woq_kv8_page_offset(const woq_kv8_config* cfg, int page) {
  Kv8View v;
  if (!cfg || !make_view(*cfg, &v) || page < 0 || page > cfg->pages) return 0;
  return v.pool + (size_t)page * v.page_bytes();
}

int woq_kv8_init(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  return cuda_result(launch_kv8_init(v, (cudaStream_t)stream));
}

int woq_rope_table(double theta, int rot_dim, int positions, float* table, woq_stream_t stream) {
  if (!(theta > 0.0) || !isfinite(theta) || rot_dim < 4 || rot_dim > 256 || rot_dim % 4 || positions < 0)
    return WOQ_ERR_SHAPE;
  if (positions == 0) return WOQ_OK;
  if (!table) return WOQ_ERR_NULL;
  if (!aligned(table, 16)) return WOQ_ERR_ALIGN;
  return cuda_result(launch_rope_table(theta, rot_dim / 2, positions, table, (cudaStream_t)stream));
}

int woq_kv8_append_rows(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer, const int32_t* seqs,
                        int n, int rows, const void* qkv, int dtype, int row_stride, int q_heads, const woq_rope* rope,
                        void* q_out, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (const int e = check_list(seqs, n, false)) return e;
  if (rows < 1 || rows > WOQ_KV8_ROWS || layer < 0 || layer >= v.layers) return WOQ_ERR_SHAPE;
  if (n == 0) return WOQ_OK;
  Kv8Append p;
  if (const int e = fill_append(v, layer, qkv, dtype, row_stride, q_heads, rope, q_out, &p)) return e;
  p.seqs = seqs;
  p.n = n;
  p.rows = rows;
  return cuda_result(launch_kv8_append_rows(p, (cudaStream_t)stream));
}

int woq_kv8_append_prompt(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer, int seq, int tokens,
                          const void* qkv, int dtype, int row_stride, int q_heads, const woq_rope* rope, void* q_out,
                          woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (layer < 0 || layer >= v.layers || seq < 0 || seq >= v.seqs || tokens < 0 || tokens > v.max_tokens)
    return WOQ_ERR_SHAPE;
  if (tokens == 0) return WOQ_OK;
  Kv8Append p;
  if (const int e = fill_append(v, layer, qkv, dtype, row_stride, q_heads, rope, q_out, &p)) return e;
  p.n = seq;
  p.rows = tokens;
  return cuda_result(launch_kv8_prompt(p, (cudaStream_t)stream));
}

int woq_kv8_accept(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, const int32_t* seqs, int n,
                   const uint32_t* keep, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (const int e = check_list(seqs, n, false)) return e;
  if (const int e = check_list(keep, n, true)) return e;
  if (n == 0) return WOQ_OK;
  cudaError_t e = launch_kv8_accept_meta(v, seqs, n, keep, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_kv8_accept_rows(v, n, (cudaStream_t)stream);
  return cuda_result(e);
}

int woq_kv8_extend(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int seq, int tokens,
                   woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (seq < 0 || seq >= v.seqs || tokens < 0 || tokens > v.max_tokens) return WOQ_ERR_SHAPE;
  return cuda_result(launch_kv8_extend(v, seq, tokens, (cudaStream_t)stream));
}

size_t woq_kv8_attention_workspace(const woq_kv8_config* cfg, int n, int rows, int q_heads) {
  Kv8View v;
  if (!cfg || !make_view(*cfg, &v) || !attn_shape_ok(v, n, rows, q_heads)) return 0;
  const int sms = sm_count();
  if (sms <= 0) return 0;
  const int all = rows * (q_heads / v.heads), chunks = attn_chunks(v.dim, all);
  const int queries = chunks > 1 ? ((all + 7) / 8 + chunks - 1) / chunks * 8 : all;
  return attn_parts_offset(v, n, chunks, sms) + (size_t)2 * sms * queries * (v.dim + 4) * 4;
}

int woq_kv8_plan_attention(const woq_kv8_config* cfg, int n, int rows, int q_heads, int sms, int smem_max,
                           woq_kv8_plan* out) {
  if (!cfg || !out) return WOQ_ERR_NULL;
  Kv8View v;
  if (!make_view(*cfg, &v) || !attn_shape_ok(v, n, rows, q_heads) || sms < 0 || smem_max < 0) return WOQ_ERR_SHAPE;
  if (sms == 0) sms = sm_count();
  if (smem_max == 0) smem_max = max_dynamic_smem();
  if (sms <= 0 || smem_max <= 0) return WOQ_ERR_CUDA;
  Kv8Attn p = {};
  p.v = v;
  p.n = n;
  p.rows = rows;
  p.group = q_heads / v.heads;
  const int smem = kv8_attn_plan(&p, smem_max);
  if (smem == 0) return WOQ_ERR_SHAPE;
  *out = woq_kv8_plan{sms, p.warps, p.query_groups, p.stages, p.least_units, smem};
  return WOQ_OK;
}

int woq_kv8_attention(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer, const int32_t* seqs, int n,
                      int rows, const void* q, int q_heads, const uint32_t* vis, float scale, int window, int sinks,
                      void* out, void* ws, size_t ws_bytes, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (const int e = check_list(seqs, n, false)) return e;
  if (layer < 0 || layer >= v.layers || !attn_shape_ok(v, n, rows, q_heads) || !isfinite(scale) || window < 0 ||
      window > 1 << 30 || sinks < 0 || sinks > 1 << 30)
    return WOQ_ERR_SHAPE;
  if (n == 0) return WOQ_OK;
  if (!q || !out || !ws) return WOQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(vis, 4)) return WOQ_ERR_ALIGN;
  const int sms = sm_count(), smem_max = max_dynamic_smem();
  if (sms <= 0 || smem_max <= 0) return WOQ_ERR_CUDA;
  if (ws_bytes < woq_kv8_attention_workspace(cfg, n, rows, q_heads)) return WOQ_ERR_WORKSPACE;
  Kv8Attn p = {};
  p.v = v;
  p.seqs = seqs;
  p.q = static_cast<const uint16_t*>(q);
  p.vis = vis;
  p.out = static_cast<uint16_t*>(out);
  p.failed = reinterpret_cast<uint32_t*>(ws) + 1;
  p.tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + 256);
  p.joins = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + attn_joins_offset(sms));
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.layer = layer;
  p.n = n;
  p.rows = rows;
  p.q_heads = q_heads;
  p.group = q_heads / v.heads;
  p.window = window;
  p.sinks = sinks;
  p.ctas = sms;
  p.fault_cta = fault_cta(1);
  p.wait_ns = (uint32_t)wait_bound_ns();  // at most 2 s
  const int smem = kv8_attn_plan(&p, smem_max);
  if (smem == 0) return WOQ_ERR_SHAPE;
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + attn_parts_offset(v, n, p.chunks, sms));
  // whether an item can lie in several CTAs: there are more items than CTAs, or one has more units than stay whole
  // (as far as max_tokens and the window tell)
  long long most = v.max_tokens / kKv8Block;
  if (window > 0) most = std::min(most, ((long long)window + kKv8Block - 1) / kKv8Block + 1 + ((long long)sinks + kKv8Block - 1) / kKv8Block);
  p.joined = (long long)n * p.heads > sms || most + kv8::kTailUnits > kv8::kWhole;
  const bool int8 = v.fmt == WOQ_KV8_INT8;
  const auto launch = p.team ? (int8 ? launch_kv8_team_int8 : launch_kv8_team_e4m3)
                             : (int8 ? launch_kv8_attn_int8 : launch_kv8_attn_e4m3);
  return cuda_result(launch(p, sms, smem, (cudaStream_t)stream));
}

int woq_kv8_fork(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, const int32_t* src, const int32_t* dst,
                 int n, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (const int e = check_list(src, n, true)) return e;
  if (const int e = check_list(dst, n, true)) return e;
  if (n == 0) return WOQ_OK;
  return cuda_result(launch_kv8_fork(v, src, dst, n, (cudaStream_t)stream));
}

int woq_kv8_free(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, const int32_t* seqs, int n,
                 woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (const int e = check_list(seqs, n, true)) return e;
  if (n == 0) return WOQ_OK;
  return cuda_result(launch_kv8_free(v, seqs, n, (cudaStream_t)stream));
}

int woq_kv8_copy(const woq_kv8_config* src_cfg, const void* src, size_t src_bytes, const woq_kv8_config* dst_cfg,
                 void* dst, size_t dst_bytes, const int32_t* src_seqs, const int32_t* dst_seqs, int n,
                 woq_stream_t stream) {
  Kv8View sv, dv;
  if (const int e = open_cache(src_cfg, src, src_bytes, &sv)) return e;
  if (const int e = open_cache(dst_cfg, dst, dst_bytes, &dv)) return e;
  if (const int e = check_list(src_seqs, n, true)) return e;
  if (const int e = check_list(dst_seqs, n, true)) return e;
  if (sv.fmt != dv.fmt || sv.layers != dv.layers || sv.heads != dv.heads || sv.dim != dv.dim) return WOQ_ERR_SHAPE;
  if (sv.base == dv.base ? sv.hash != dv.hash : (sv.base < dv.base + dv.total && dv.base < sv.base + sv.total))
    return WOQ_ERR_LAYOUT;
  if (n == 0) return WOQ_OK;
  return cuda_result(launch_kv8_copy(sv, dv, src_seqs, dst_seqs, n, (cudaStream_t)stream));
}

int woq_kv8_compact(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int limit, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (limit < 1 || limit > v.pages) return WOQ_ERR_SHAPE;
  return cuda_result(launch_kv8_compact(v, limit, (cudaStream_t)stream));
}

int woq_kv8_read(const woq_kv8_config* cfg, void* cache, size_t cache_bytes, int layer, int seq, int first, int count,
                 void* k, void* v_out, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (layer < -1 || layer >= v.layers || seq < 0 || seq >= v.seqs || first < 0 || count < 0 ||
      (long long)first + count > (long long)v.max_tokens + WOQ_KV8_ROWS)
    return WOQ_ERR_SHAPE;
  if (count == 0) return WOQ_OK;
  if (!k || !v_out) return WOQ_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v_out, 16)) return WOQ_ERR_ALIGN;
  return cuda_result(launch_kv8_read(v, layer < 0 ? 0 : layer, layer < 0 ? v.layers : 1, seq, first, count,
                                     static_cast<uint16_t*>(k), static_cast<uint16_t*>(v_out), (cudaStream_t)stream));
}

int woq_kv8_state(const woq_kv8_config* cfg, const void* cache, size_t cache_bytes, int32_t* lens, int32_t* refs,
                  int32_t* table, woq_stream_t stream) {
  Kv8View v;
  if (const int e = open_cache(cfg, cache, cache_bytes, &v)) return e;
  if (!aligned(lens, 4) || !aligned(refs, 4) || !aligned(table, 4)) return WOQ_ERR_ALIGN;
  if (!lens && !refs && !table) return WOQ_OK;
  return cuda_result(launch_kv8_state(v, lens, refs, table, (cudaStream_t)stream));
}

}  // extern "C"
