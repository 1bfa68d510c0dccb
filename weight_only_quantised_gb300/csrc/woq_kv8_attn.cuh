// Attention of a few rows over the 8-bit cache.
//
//   out = sum_j softmax_j(scale q . k_j) v_j      q: rows * group queries of one kv head
//
// The keys and values of a long context are read once and used by few queries, so the bound is HBM:
// 2 D bytes per (token, head) plus 16 per block, while the operations stay below what the
// tensor cores do in that time for up to 16 queries (mma.sync m16n8k16 f16 with fp32 sums runs at
// about 512 multiply-adds a clock and SM here; 16 queries need 440 at the copy peak).
//
// Split: an item (entry, kv head) is its blocks and kTailUnits units for its tail.  With at most as many items
// as CTAs (one CTA per SM) every item is cut into equal pieces, one piece per CTA, the longer items
// into more; a CTA that held the end of one item and the beginning of another would wait twice for
// the tail, the joining of its warps and the counting in (131,071 tokens, 8 heads: 62 us against 54).
// Items of up to kWhole units stay whole: joining partials costs as much as those blocks.  With more items the
// units are laid end to end and every CTA takes an equal share.  Lengths are read on the device, so
// this plan is made there.  An item in several CTAs leaves fp32 partials (maximum, sum, weighted
// values); the CTA that counts in last joins them in CTA order, so the result does not depend on the run.
//
// CTA: one producer warp copies whole records (16 KB at D = 128, one bulk copy each) into a ring; with up to 8
// queries each consumer warp takes whole blocks by itself (always from the same stages, in order), with its own
// running maximum and sums in registers, so the main loop has no barrier but the ring's.
//
// Block: scores transposed, S^T = K Q^T (tokens x queries), so that both codes operands are the
// 16-row one and the 8-wide one is the queries: nothing is padded beyond 8 queries.  Codes
// become f16 in registers, exactly (int8: a byte permute into 1024 + 128 + c and a subtraction; e4m3: one
// conversion); queries are bf16 scaled into f16 by the power of two that brings the row's largest to [1, 2):
// exactly, but for elements below 2^-17 of it, which f16 holds to multiples of 2^-24.  Weights are 2^(s - m) in
// fp32 (ex2.approx, good to 2^-22) for the sum, rounded to f16 for the product: half a step is 2^-11, an eighth of the
// result's own in bf16, and a second product for their low parts would double the work on values.
// m is raised only when a score passes it by 7, and weights carry a factor 2^7, so
// f16 holds them to 2^-31 of the largest; the value scale takes their greatest factor off again (kUnit).  movmatrix turns the score fragments into the other
// product's operand: O^T = V^T P^T, from the transposed value codes.  Each block's product is
// scaled by its value scale in fp32.
//
// Measured (8 heads, D = 128, launches back to back): 131,071 tokens x 5 queries 50 us (5.4 TB/s of codes and scales; the
// copy rate alone would be 39.5), x 1 head's 4 of 8 sequences up to 20,000 42.  Of these about 4.5 us pass before the
// first block (plan, queries, code that is not in the instruction cache) and 4 in the joins.
//
// Tail: at most 63 tokens and the draft rows, bf16, straight from global memory; same fragments with
// bf16 products, 16 tokens per warp, queries as they are, weights as two bf16 parts (16 bits, half a step 2^-17: values may
// be any bf16, so the product is one of bf16).
#pragma once

#include <atomic>

#include "woq_internal.h"
#include "woq_kv8_device.cuh"

namespace woq {
namespace kv8 {

constexpr float kRaise = 7.0f;    // a score may pass the running maximum by this (log2) before it is raised
constexpr float kOffset = 7.0f;   // weights carry 2^kOffset
static_assert(kRaise + kOffset == 14.0f && kUnit == 0x1p-14f, "weights are at most 1 / kUnit");
constexpr int kMergePad = 4;      // floats behind each row of the merge buffer (bank spread)

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What an entry's rows see of its blocks: [0, head_blocks) and [from, full).
struct Span {
  int len, full, head_blocks, from, units;  // units: blocks seen, and kTailUnits for the tail
};

// Units that the tail counts for: it takes a CTA as long as so many blocks (3 to 4 us).  They lie behind the
// item's blocks; whoever has the last of them does the tail.
constexpr int kTailUnits = 8;

__device__ __forceinline__ Span span_of(int len, int window, int sinks) {
  Span s;
  s.len = len;
  s.full = len / kKv8Block;
  s.head_blocks = 0;
  s.from = 0;
  if (window > 0 && len > window) {  // no row sees tokens in [sinks, len - window)
    s.from = (len - window) / kKv8Block;
    s.head_blocks = (sinks + kKv8Block - 1) / kKv8Block;
    if (s.head_blocks >= s.from) s.head_blocks = s.from;
  }
  s.units = s.head_blocks + (s.full - s.from) + kTailUnits;
  return s;
}

// Running state of a warp's queries: columns 2t, 2t + 1 of each tile of 8.
template <int D>
struct State {
  float m[2], l[2];
  float o[D / 16][4];  // rows g, g + 8 of each 16 elements
};

template <int D>
__device__ __forceinline__ void clear(State<D>& st) {
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) st.o[j][i] = 0.0f;
}

// Raise the maxima to cover mx (per column, the same in the lanes of a column) where it passes them
// by more than kRaise, and scale what was summed.
template <int D>
__device__ __forceinline__ void raise(State<D>& st, const float (&mx)[2]) {
  if (!__any_sync(~0u, mx[0] > st.m[0] + kRaise || mx[1] > st.m[1] + kRaise)) return;
  float a[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float n = fmaxf(st.m[c], mx[c]);
    a[c] = n == -INFINITY ? 1.0f : exp2_approx(st.m[c] - n);
    st.m[c] = n;
    st.l[c] *= a[c];
  }
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    st.o[j][0] *= a[0];
    st.o[j][1] *= a[1];
    st.o[j][2] *= a[0];
    st.o[j][3] *= a[1];
  }
}

__device__ __forceinline__ float column_max(float x) {  // over the lanes that share t
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
  return fmaxf(x, __shfl_xor_sync(~0u, x, 16));
}

// What the lane knows about its columns' rows for the masks: first place seen by the window, draft mask.
struct Columns {
  int low[2];       // places >= low are in the window
  uint32_t vis[2];  // draft rows seen
};

// One block of codes at `rec` (shared memory), first token `token0`.
template <int FMT, int D>
__device__ __forceinline__ void block_step(State<D>& st, const uint8_t* rec, const uint32_t (&qf)[D / 16][2],
                                           const float (&coef)[2], const Columns& col, int token0, bool masked, int sinks,
                                           int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float ks = *reinterpret_cast<const float*>(rec + 128 * D);
  const float vs = *reinterpret_cast<const float*>(rec + 128 * D + 8);  // times kUnit
  const uint8_t* kc = rec + t * 128 + g * 16;
  float s[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[i][c] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(kc + (2 * i * (D / 16) + 4 * c) * 128);
      const uint4 y = *reinterpret_cast<const uint4*>(kc + ((2 * i + 1) * (D / 16) + 4 * c) * 128);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[4];
        f16x4_of_codes<FMT>(xs[k], a[0], a[2]);
        f16x4_of_codes<FMT>(ys[k], a[1], a[3]);
        mma_f16(s[i], a, qf[4 * c + k][0], qf[4 * c + k][1]);
      }
    }
  }
  float mx[2];
  const float f0 = coef[0] * ks, f1 = coef[1] * ks;
  mx[0] = mx[1] = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[i][0] *= f0;
    s[i][1] *= f1;
    s[i][2] *= f0;
    s[i][3] *= f1;
    if (masked) {
      const int tok = token0 + 16 * (g >> 1) + 4 * i + (g & 1);
      if (tok >= sinks) {
        if (tok < col.low[0]) s[i][0] = -INFINITY;
        if (tok < col.low[1]) s[i][1] = -INFINITY;
      }
      if (tok + 2 >= sinks) {
        if (tok + 2 < col.low[0]) s[i][2] = -INFINITY;
        if (tok + 2 < col.low[1]) s[i][3] = -INFINITY;
      }
    }
    mx[0] = fmaxf(mx[0], fmaxf(s[i][0], s[i][2]));
    mx[1] = fmaxf(mx[1], fmaxf(s[i][1], s[i][3]));
  }
  mx[0] = column_max(mx[0]);
  mx[1] = column_max(mx[1]);
  raise(st, mx);
  uint32_t pb[4][2];
  const float r0 = (st.m[0] == -INFINITY ? 0.0f : st.m[0]) - kOffset;
  const float r1 = (st.m[1] == -INFINITY ? 0.0f : st.m[1]) - kOffset;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p0 = exp2_approx(s[i][0] - r0), p1 = exp2_approx(s[i][1] - r1);
    const float p2 = exp2_approx(s[i][2] - r0), p3 = exp2_approx(s[i][3] - r1);
    st.l[0] += p0 + p2;
    st.l[1] += p1 + p3;
    pb[i][0] = transpose8x8(pack_f16(p0, p1));
    pb[i][1] = transpose8x8(pack_f16(p2, p3));
  }
  const uint8_t* vc = rec + 64 * D + t * 128 + g * 16;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const uint4 x = *reinterpret_cast<const uint4*>(vc + 2 * j * 512);
    const uint4 y = *reinterpret_cast<const uint4*>(vc + (2 * j + 1) * 512);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    float acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4];
      f16x4_of_codes<FMT>(xs[i], a[0], a[2]);
      f16x4_of_codes<FMT>(ys[i], a[1], a[3]);
      mma_f16(acc, a, pb[i][0], pb[i][1]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) st.o[j][c] = fmaf(vs, acc[c], st.o[j][c]);
  }
}

// Whether a row with draft mask vis and window from place `low` sees row r of the tail (in_tail tokens, then drafts).
__device__ __forceinline__ bool tail_sees(int r, uint32_t vis, int low, int in_tail, int there, int len, int sinks) {
  if (r >= there) return false;
  const int draft = r - in_tail;
  int place = len + draft;
  if (draft >= 0) {
    if (!((vis >> draft) & 1u)) return false;
    place = len + __popc(vis & ((1u << draft) - 1u));
  }
  return place < sinks || place >= low;
}

// Tail tile i: i < 4: tokens 16 t' + 4 i + {0 .. 3} of the tail (t' = 0 .. 3), in the order of the
// key rows of a block; i = 4: tail rows 64 .. 71.  there: rows of the tail that anything may be seen of.
template <int D>
__device__ __forceinline__ void tail_step(State<D>& st, const uint16_t* tail, int i, int in_tail, int len, int there,
                                          const uint16_t* qrow, float scale_log2, const Columns& col, int sinks,
                                          int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int r0 = i < 4 ? 16 * (g >> 1) + 4 * i + (g & 1) : 64 + g;
  const int r1 = i < 4 ? r0 + 2 : kKv8Tail;
  // values first: their loads are under way while the scores are worked out
  const uint16_t* tv = tail + kKv8Tail * D;
  uint32_t va[D / 16][4];
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const uint16_t* v0 = tv + (16 * j + g) * kKv8Tail;
    const uint16_t* v1 = v0 + 8 * kKv8Tail;
    if (i < 4) {
      const uint2 x = *reinterpret_cast<const uint2*>(v0 + 16 * t + 4 * i);
      const uint2 y = *reinterpret_cast<const uint2*>(v1 + 16 * t + 4 * i);
      va[j][0] = x.x, va[j][1] = y.x, va[j][2] = x.y, va[j][3] = y.y;
    } else {
      va[j][0] = *reinterpret_cast<const uint32_t*>(v0 + 64 + 2 * t);
      va[j][1] = *reinterpret_cast<const uint32_t*>(v1 + 64 + 2 * t);
      va[j][2] = va[j][3] = 0u;
    }
  }
  float s[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) s[c] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint32_t x[8], y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (r0 < there) a = *reinterpret_cast<const uint4*>(tail + r0 * D + 16 * (4 * c + t) + 8 * h);
      if (r1 < there) b = *reinterpret_cast<const uint4*>(tail + r1 * D + 16 * (4 * c + t) + 8 * h);
      x[4 * h] = a.x, x[4 * h + 1] = a.y, x[4 * h + 2] = a.z, x[4 * h + 3] = a.w;
      y[4 * h] = b.x, y[4 * h + 1] = b.y, y[4 * h + 2] = b.z, y[4 * h + 3] = b.w;
    }
    uint32_t w[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 a = {0, 0, 0, 0};
      if (qrow) a = *reinterpret_cast<const uint4*>(qrow + 16 * (4 * c + t) + 8 * h);
      w[4 * h] = a.x, w[4 * h + 1] = a.y, w[4 * h + 2] = a.z, w[4 * h + 3] = a.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a[4] = {x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1]};
      mma_bf16(s, a, w[2 * k], w[2 * k + 1]);
    }
  }
  float mx[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    s[c] = tail_sees(r0, col.vis[c], col.low[c], in_tail, there, len, sinks) ? s[c] * scale_log2 : -INFINITY;
    s[2 + c] = tail_sees(r1, col.vis[c], col.low[c], in_tail, there, len, sinks) ? s[2 + c] * scale_log2 : -INFINITY;
    mx[c] = column_max(fmaxf(s[c], s[2 + c]));
  }
  raise(st, mx);
  uint32_t hi[2], lo[2];
  float p[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float r = (st.m[c & 1] == -INFINITY ? 0.0f : st.m[c & 1]) - kOffset;
    p[c] = exp2_approx(s[c] - r);
    st.l[c & 1] += p[c];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float w0 = p[2 * h] * kUnit, w1 = p[2 * h + 1] * kUnit;
    const uint32_t u = pack_bf16(w0, w1);
    const float f0 = __uint_as_float(u << 16), f1 = __uint_as_float(u & 0xFFFF0000u);
    hi[h] = transpose8x8(u);
    lo[h] = transpose8x8(pack_bf16(w0 - f0, w1 - f1));
  }
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    mma_bf16(st.o[j], va[j], hi[0], hi[1]);
    mma_bf16(st.o[j], va[j], lo[0], lo[1]);
  }
}

// Query row of the lane's column (nullptr: zeros) as operands, scaled by 2^-e to below 2; returns 2^e.
template <int D>
__device__ __forceinline__ float load_query(uint32_t (&qf)[D / 16][2], const uint16_t* qrow, int lane) {
  const int t = lane & 3;
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 a = {0, 0, 0, 0};
      if (qrow) a = *reinterpret_cast<const uint4*>(qrow + 16 * (4 * c + t) + 8 * h);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        qf[4 * c + 2 * h + (k >> 1)][k & 1] = w[k];
        top = dev::bf16x2_absmax(top, w[k]);
      }
    }
  }
  float m = dev::bf16x2_absmax_to_float(top);
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
  int e = (int)(__float_as_uint(m) >> 23) - 127;  // m = 0 or subnormal: -127
  e = e < -126 ? -126 : e > 126 ? 126 : e;
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = qf[k][h];
      qf[k][h] = pack_f16(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xFFFF0000u) * down);
    }
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

constexpr int kMaxStages = 32;
// Most warps that each take a block: two per sub-partition with the producer, so 255 registers each.
constexpr int kMaxWarps = 7;
// Shared memory: barriers, flags, units and lengths of the entries; the merge buffer; the ring.
struct Misc {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int fail, last;
  uint32_t wait_ns;  // bound of the teams' waits
  int share;      // units of a piece, 0: more items than CTAs
  int redo;       // the plan made before the wait does not hold
  // [n + 1] units of one head of the entries before, [n] lengths (-1: out of range), [n + 1] pieces (CTAs) of
  // the entries before, [n] sequence numbers (if they are given)
  int entries[];
};
__host__ __device__ inline int misc_bytes(int n) { return (int)((sizeof(Misc) + (size_t)(4 * n + 2) * 4 + 127) / 128 * 128); }
constexpr int kWhole = 32;  // units of an item that is not cut

__device__ __forceinline__ int pieces_of(int units, int share) { return units <= kWhole ? 1 : (units + share - 1) / share; }
__host__ __device__ inline int merge_bytes(int warps, int qt, int dim) {
  return (warps * 8 * qt * (dim + kMergePad + 2) * 4 + 127) / 128 * 128;
}

// What the joining of partials does with one: its weight against the common maximum m.  A part whose
// maximum is -inf has seen nothing (sum 0) or only scores that are not numbers (sum NaN: kept).
__device__ __forceinline__ float part_factor(float pm, float pl, float m) {
  return pm == -INFINITY ? (pl == 0.0f ? 0.0f : 1.0f) : exp2_approx(pm - m);
}

__device__ __forceinline__ int* lens_of(const Kv8Attn& p, Misc& misc) { return misc.entries + p.n + 1; }
__device__ __forceinline__ int* seqs_of(const Kv8Attn& p, Misc& misc) { return misc.entries + 3 * p.n + 2; }

// Where query n of a kv head is in p.q and p.out.
template <int D>
__device__ __forceinline__ size_t query_at(const Kv8Attn& p, int e, int kv_head, int n) {
  return (((size_t)e * p.rows + n / p.group) * p.q_heads + (size_t)kv_head * p.group + n % p.group) * D;
}

// This CTA's units [begin, end), of all items laid end to end.  All counts fit 32 bits (checked on the host).
struct Plan {
  int begin, end;
  bool cut;            // pieces of items, one per CTA
  int piece0, pieces;  // cut: the item's first CTA and their number
  int share;           // else: units of a CTA
};

// Number of entry e's sequence; its length, -1 if the number is out of range.
__device__ __forceinline__ int number_of(const Kv8Attn& p, int e) { return p.seqs ? (int)dev::ld_relaxed_u32(p.seqs + e) : e; }
__device__ __forceinline__ int length_of(const Kv8Attn& p, int seq) {
  return seq >= 0 && seq < p.v.seqs ? (int)dev::ld_relaxed_u32(p.v.lens_p() + seq) : -1;
}
__device__ __forceinline__ bool is_ours(const Kv8View& v, uint32_t* magic) {
  *magic = dev::ld_relaxed_u32(v.status() + 1);
  return dev::ld_relaxed_u32(v.status() + 2) == v.hash && *magic == kKv8Magic;
}

// Reads the lengths and lays out the units and pieces of the entries.  Warp 0; lengths out of range (a cache
// that is being changed, before the wait for who changes it) count as 0.
__device__ __forceinline__ void lay_out(const Kv8Attn& p, Misc& misc, int lane) {
  const Kv8View& v = p.v;
  int* lens = lens_of(p, misc);
  int* cuts = lens + p.n;
  const int ctas = (int)gridDim.x;
  int run = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < p.n; e0 += 32) {
    const int e = e0 + lane;
    int units = 0;
    if (e < p.n) {
      const int seq = number_of(p, e);
      int len = length_of(p, seq);
      if (len > v.max_tokens) len = 0;
      if (len < -1) len = -1;
      lens[e] = len;
      if (p.seqs) seqs_of(p, misc)[e] = seq;
      units = len >= 0 ? span_of(len, p.window, p.sinks).units : kTailUnits;
    }
    int y = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(~0u, y, d);
      if (lane >= d) y += z;
    }
    if (e < p.n) misc.entries[e] = run + y - units;
    run += __shfl_sync(~0u, y, 31);
  }
  if (lane == 0) misc.entries[p.n] = run;
  // The least share with which all pieces have a CTA, to 1/32: the lanes try 32 of them at once.
  int share = 0;
  if (p.n * p.heads <= ctas) {
    __syncwarp();
    const int room = ctas / p.heads;  // pieces of one head
    share = max(p.least_units, (run + room - 1) / room);
#pragma unroll 1
    while (p.n > 1) {  // ends: with a share beyond the longest item there are n <= room pieces
      const int mine = share + (int)((long long)share * lane / 32);
      int total = 0;
#pragma unroll 1
      for (int e = 0; e < p.n; ++e) total += pieces_of(misc.entries[e + 1] - misc.entries[e], mine);
      const uint32_t fits = __ballot_sync(~0u, total <= room);
      share = __shfl_sync(~0u, mine, fits ? __ffs((int)fits) - 1 : 31);
      if (fits) break;
      ++share;
    }
    int total = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.n; e0 += 32) {
      const int e = e0 + lane;
      int y = e < p.n ? pieces_of(misc.entries[e + 1] - misc.entries[e], share) : 0;
      const int own = y;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int z = __shfl_up_sync(~0u, y, d);
        if (lane >= d) y += z;
      }
      if (e < p.n) cuts[e] = (total + y - own) * p.heads;
      total += __shfl_sync(~0u, y, 31);
    }
    if (lane == 0) cuts[p.n] = total * p.heads;
  }
  if (lane == 0) misc.share = share;
}

// This CTA's share of what lay_out left; false: none.
__device__ __forceinline__ bool take_share(const Kv8Attn& p, Misc& misc, Plan& pl) {
  const int heads = p.heads, block = (int)blockIdx.x;
  const int* cuts = lens_of(p, misc) + p.n;
  if (misc.share > 0) {
    if (block >= cuts[p.n]) return false;
    int lo = 0, hi = p.n - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cuts[mid] <= block) lo = mid; else hi = mid - 1;
    }
    const int per = misc.entries[lo + 1] - misc.entries[lo], pieces = (cuts[lo + 1] - cuts[lo]) / heads;
    const int head = (block - cuts[lo]) / pieces, j = block - cuts[lo] - head * pieces;
    const int first = misc.entries[lo] * heads + head * per;
    const int some = per / pieces, rest = per - some * pieces;  // per * j / pieces, in 32 bits
    pl = Plan{first + some * j + rest * j / pieces, first + some * (j + 1) + rest * (j + 1) / pieces, true, block - j, pieces, 0};
    return true;
  }
  const int units = misc.entries[p.n] * heads;
  const int share = max(p.least_units, (units + (int)gridDim.x - 1) / (int)gridDim.x), begin = block * share;
  if (begin >= units) return false;
  pl = Plan{begin, min(begin + share, units), false, 0, 0, share};
  return true;
}

// The item that holds unit u: entry, head, first unit.
__device__ __forceinline__ void locate(const Kv8Attn& p, const Misc& misc, int u, int* entry, int* head, int* item_begin) {
  const int* prefix = misc.entries;
  int lo = 0, hi = p.n - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] * p.heads <= u) lo = mid; else hi = mid - 1;
  }
  const int per = prefix[lo + 1] - prefix[lo], first = prefix[lo] * p.heads;
  *entry = lo;
  *head = (u - first) / per;
  *item_begin = first + *head * per;
}

// The records that fill the ring first, the queries and the tail, into L2.  One warp; nothing read here is relied on, so
// numbers are only used if they are in range.
__device__ __forceinline__ void prefetch_first(const Kv8Attn& p, Misc& misc, const Plan& pl, int lane) {
  const Kv8View& v = p.v;
  int e, head, ib;
  locate(p, misc, pl.begin, &e, &head, &ib);
  const int per = misc.entries[e + 1] - misc.entries[e], len = lens_of(p, misc)[e];
  const int seq = p.seqs ? (int)dev::ld_relaxed_u32(p.seqs + e) : e;
  if (len < 0 || seq < 0 || seq >= v.seqs) return;
  const Span sp = span_of(len, p.window, p.sinks);
  const int k = pl.begin - ib + lane, stop = min(pl.end - ib, per - kTailUnits);
  if (lane < p.stages && k < stop) {
    const int page = (int)dev::ld_relaxed_u32(v.table_row(seq) + (k < sp.head_blocks ? k : sp.from + (k - sp.head_blocks)));
    if (page >= 0 && page < v.pages) dev::bulk_prefetch_l2(v.record(page, p.layer, head / p.chunks), (uint32_t)v.record_bytes());
  }
  const int kv_head = head / p.chunks, q_elems = p.group * v.dim;  // of one row
#pragma unroll 1
  for (int x = lane * 64; x < q_elems * p.rows; x += 32 * 64) {
    const int row = x / q_elems;
    dev::prefetch_l2(p.q + (((size_t)e * p.rows + row) * p.q_heads + (size_t)kv_head * p.group) * v.dim + (x - row * q_elems));
  }
  if (lane == 31 && pl.end >= ib + per)
    dev::bulk_prefetch_l2(v.tail(p.layer, seq, kv_head), (uint32_t)v.tail_elems() * 2u);
}

// This CTA's plan; false: nothing to do.  All threads.
//
// The chain sequence number, length, page number, record is four dependent reads, most of them from
// HBM.  So before the wait for the prior grid the plan is made from what the cache holds then, and the first
// records are brought into L2; after the wait the lengths are read again and, if one has changed,
// the plan is made anew.  (In a step the CTA gets its SM while the grid before it ends; nothing but the
// plan is kept from before the wait, and that is checked.)
__device__ __forceinline__ bool make_plan(const Kv8Attn& p, Misc& misc, int tid, Plan& pl) {
  const Kv8View& v = p.v;
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t magic;
  bool known = __syncthreads_and(is_ours(v, &magic)), active = false;
  const bool guessed = known;
#pragma unroll 1
  for (int pass = 0;; ++pass) {  // (once more, if the first plan does not hold)
    if (known) {
      if (warp == 0) lay_out(p, misc, lane);
      __syncthreads();
      active = take_share(p, misc, pl);
    }
    if (pass > 0) return active;
    if (active && warp == p.warps) prefetch_first(p, misc, pl, lane);
    begin_after_prior();
    known = is_ours(v, &magic);
    if (warp == 0) {
      bool same = guessed;
#pragma unroll 1
      for (int e = lane; e < p.n; e += 32) {
        const int seq = number_of(p, e), before = guessed ? (p.seqs ? seqs_of(p, misc)[e] : e) : seq;
        const int len = length_of(p, before);  // beside the number's read, not behind it
        if (guessed) same &= seq == before && len == lens_of(p, misc)[e];
        if (known && (seq < 0 || seq >= v.seqs) && blockIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
      }
      same = __all_sync(~0u, same);
      if (lane == 0) misc.redo = !same;
    }
    if (!known) {
      if (magic == kKv8Magic && tid == 0) flag(v, WOQ_DEVERR_HEADER);
      return false;
    }
    __syncthreads();
    if (!misc.redo) return active;
  }
}

// The producer warp: the records of this CTA's blocks, in order, into the ring's stages.
template <int D>
__device__ __forceinline__ void produce(const Kv8Attn& p, Misc& misc, const Plan& pl, uint8_t* ring, int lane) {
  constexpr int kRecord = 128 * D + 16;
  const Kv8View& v = p.v;
  const int S = p.stages;
  int issued = 0;
  if ((int)blockIdx.x == p.fault_cta) return;  // injected fault: the consumers' waits run out
#pragma unroll 1
  for (int u = pl.begin; u < pl.end;) {
    int e, head, ib;
    locate(p, misc, u, &e, &head, &ib);
    const int per = misc.entries[e + 1] - misc.entries[e];
    const int stop = min(ib + per, pl.end);
    const int b0 = u - ib, b1 = min(stop - ib, per - kTailUnits);
    if (b0 < b1) {
      const Span sp = span_of(lens_of(p, misc)[e], p.window, p.sinks);
      const int32_t* table = v.table_row(p.seqs ? p.seqs[e] : e);
      const int kv_head = head / p.chunks;
#pragma unroll 1
      for (int c0 = b0; c0 < b1; c0 += 32) {
        const int k = c0 + lane;
        int page = 0;
        if (k < b1) page = table[k < sp.head_blocks ? k : sp.from + (k - sp.head_blocks)];
        const int some = b1 - c0 < 32 ? b1 - c0 : 32;
#pragma unroll 1
        for (int i = 0; i < some; ++i) {
          const int pg = __shfl_sync(~0u, page, i);
          const int stage = issued % S;
          bool ok = true;
          if (issued >= S) ok = dev::mbar_wait_bounded(&misc.empty[stage], (uint32_t)((issued / S - 1) & 1), p.wait_ns);
          if (!__all_sync(~0u, ok)) {
            // the consumers stopped (they report it): nothing more is issued; copies in flight are waited for below
              u = pl.end;
            break;
          }
          if (lane == 0) {
            dev::mbar_arrive_expect_tx(&misc.full[stage], kRecord);
            dev::bulk_copy_g2s(ring + (size_t)stage * kRecord, v.record(pg, p.layer, kv_head), kRecord, &misc.full[stage]);
          }
          ++issued;
        }
        if (u >= pl.end) break;
      }
    }
    if (u >= pl.end) break;
    u = stop;
  }
  // copies in flight end before this CTA's shared memory is given up
#pragma unroll 1
  for (int i = issued > S ? issued - S : 0; i < issued; ++i)
    dev::mbar_wait_bounded(&misc.full[i % S], (uint32_t)((i / S) & 1));
}

// The item's result, or this CTA's part of it, from `sets` sets of partials (at most 8) that the consumers left in
// shared memory: set w, query n at row n + w * stride of merge ([D] floats) and of ml_of (maximum, sum).
// merge holds `room` floats and is scratch afterwards.  All consumers; the caller has synchronised them.
//
// Joining parts is one CTA's work while the others have ended, so what counts is how many loads are under way.
// A part in p.parts: [R][D] values, [R][2] maxima and sums, in steps of R (D + 4) floats; two slots a CTA.
//
// LATER: parts are left for join_kernel, and the CTA that has the item's first unit says where they are.
template <int D, bool LATER>
__device__ __forceinline__ void finish(const Kv8Attn& p, Misc& misc, const Plan& plan, float* merge, int room,
                                       const float* ml_of, int sets, int stride, int e, int head, int ib, int per, int tid,
                                       int consumers) {
  constexpr int kRow = D + kMergePad;
  // this item's queries: [base, base + R) of the kv head
  const int kv_head = LATER ? head / p.chunks : head, base = LATER ? head % p.chunks * p.queries : 0;
  const int Q = p.queries, R = LATER ? min(Q, p.rows * p.group - base) : Q, lane = tid & 31;
  const bool whole = plan.cut ? plan.pieces == 1 : ib >= plan.begin && ib + per <= plan.end;
  const int mine = plan.cut || ib <= plan.begin ? 0 : 1;  // the item that holds the share's first unit, and the other
  const size_t slot = (size_t)Q * (D + 4);
  float* part = p.parts + ((size_t)blockIdx.x * 2 + mine) * slot;
#pragma unroll 1
  for (int x = tid; x < R * (D / 4); x += consumers) {
    const int n = x / (D / 4), d = (x % (D / 4)) * 4;
    float pm[8], ps[8], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float2 ml = w < sets ? *reinterpret_cast<const float2*>(ml_of + 2 * (n + w * stride)) : make_float2(-INFINITY, 0.0f);
      pm[w] = ml.x;
      ps[w] = ml.y;
      m = fmaxf(m, ml.x);
    }
    float4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w >= sets) break;
      const float f = part_factor(pm[w], ps[w], m);
      const float4 y = *reinterpret_cast<const float4*>(merge + (size_t)(n + w * stride) * kRow + d);
      o.x += f * y.x;
      o.y += f * y.y;
      o.z += f * y.z;
      o.w += f * y.w;
      l += f * ps[w];
    }
    if (whole) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      *reinterpret_cast<uint2*>(p.out + query_at<D>(p, e, kv_head, base + n) + d) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    } else {
      *reinterpret_cast<float4*>(part + (size_t)n * D + d) = o;
      if (d == 0) *reinterpret_cast<float2*>(part + (size_t)Q * D + 2 * n) = make_float2(m, l);
    }
  }
  if (LATER && tid == 0 && ib >= plan.begin) {
    const int c0 = (int)blockIdx.x;
    const int pieces = whole ? 1 : plan.cut ? plan.pieces : (ib + per - 1) / plan.share - c0 + 1;
    p.joins[(size_t)e * p.heads + head] = make_int2(2 * c0 + mine, pieces);
  }
  if (whole || LATER) return;
  // CTAs c0 .. c1 share the item; the one that counts in last joins their parts in CTA order
  const int c0 = plan.cut ? plan.piece0 : ib / plan.share;
  const int c1 = plan.cut ? plan.piece0 + plan.pieces - 1 : (ib + per - 1) / plan.share;
  dev::named_barrier_sync(1, consumers);
  uint32_t* ticket = p.tickets + c0;
  if (tid == 0) misc.last = dev::atomic_add_acq_rel_gpu(ticket, 1u) == (uint32_t)(c1 - c0);
  dev::named_barrier_sync(1, consumers);
  if (!misc.last) return;
  if (tid == 0) *ticket = 0u;
  // The item is the first of each CTA's slots but perhaps of c0's, where it may be the second.
  const size_t step = 2 * slot;
  const float* parts = p.parts + (size_t)c0 * step;
  const size_t first = !plan.cut && ib > c0 * plan.share ? slot : 0;
  const int np = c1 - c0 + 1, warps = consumers >> 5;
  const int some = min(R, room / (np + 1));  // queries at a time: np factors and a sum each in the scratch
  constexpr int kAhead = 20;  // loads under way per thread, the first unit's before the maxima and sums are read
  float4 ahead[kAhead];
#pragma unroll 1
  for (int n0 = 0; n0 < R; n0 += some) {
    const int n1 = min(R, n0 + some);
    float* sums = merge + some * np;
    const float* values = parts + (size_t)n0 * D;
    if (tid < (n1 - n0) * (D / 4)) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < np) ahead[i] = __ldcg(reinterpret_cast<const float4*>(values + 4 * tid + i * step + (i == 0 ? first : 0)));
    }
#pragma unroll 1
    for (int nb = n0 + (tid >> 5); nb < n1; nb += 4 * warps) {  // a warp per query, four of them under way
      float2 ml[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nb + j * warps;
        ml[j] = n < n1 && lane < np
                    ? __ldcg(reinterpret_cast<const float2*>(parts + lane * step + (lane == 0 ? first : 0) + (size_t)R * D + 2 * n))
                    : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nb + j * warps;
        if (n >= n1) break;
        const float* at = parts + (size_t)R * D + 2 * n;
        float m = ml[j].x;
#pragma unroll 1
        for (int c = lane + 32; c < np; c += 32) m = fmaxf(m, __ldcg(at + c * step));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        float f = part_factor(ml[j].x, ml[j].y, m), l = f * ml[j].y;
        if (lane < np) merge[(n - n0) * np + lane] = f;
#pragma unroll 1
        for (int c = lane + 32; c < np; c += 32) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(at + c * step));
          f = part_factor(x.x, x.y, m);
          l += f * x.y;
          merge[(n - n0) * np + c] = f;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
        if (lane == 0) sums[n - n0] = l;
      }
    }
    dev::named_barrier_sync(1, consumers);
#pragma unroll 1
    for (int x = tid; x < (n1 - n0) * (D / 4); x += consumers) {
      const int n = n0 + x / (D / 4), d = (x % (D / 4)) * 4;
      const float* fs = merge + (n - n0) * np;
      float4 o = {0, 0, 0, 0};
      auto add = [&](float f, const float4& y) {
        o.x += f * y.x;
        o.y += f * y.y;
        o.z += f * y.z;
        o.w += f * y.w;
      };
      const float* from = values + 4 * x;
      int c = 0;
      if (x == tid) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i < np) add(fs[i], ahead[i]);
        c = min(kAhead, np);
      }
#pragma unroll 8
      for (; c < np; ++c) add(fs[c], __ldcg(reinterpret_cast<const float4*>(from + c * step + (c == 0 ? first : 0))));
      const float l = sums[n - n0], inv = l == 0.0f ? 0.0f : 1.0f / l;
      *reinterpret_cast<uint2*>(p.out + query_at<D>(p, e, kv_head, base + n) + d) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    }
    if (n1 < R) dev::named_barrier_sync(1, consumers);
  }
}

// A wait of this CTA ran out: its item, and those behind it, are not written.  One thread.
__device__ __forceinline__ void report_wait(const Kv8Attn& p) {
  flag(p.v, WOQ_DEVERR_TIMEOUT);
  atomicOr(p.failed, 1u);
}

template <int FMT, int D>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1), 1) attn_kernel(const __grid_constant__ Kv8Attn p) {
  extern __shared__ __align__(128) uint8_t smem[];
  Misc& misc = *reinterpret_cast<Misc*>(smem);
  const Kv8View& v = p.v;
  const int W = p.warps, S = p.stages, R = p.rows * p.group;
  constexpr int kRecord = 128 * D + 16;
  constexpr int kRow = D + kMergePad;
  float* merge = reinterpret_cast<float*>(smem + misc_bytes(p.n));  // [W][8][D + pad]
  float* warp_ml = merge + (size_t)W * 8 * kRow;                    // [W][8][2]
  uint8_t* ring = smem + misc_bytes(p.n) + merge_bytes(W, 1, D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      dev::mbar_init(&misc.full[i], 1);
      dev::mbar_init(&misc.empty[i], 1);
    }
    misc.fail = 0;
    dev::fence_mbar_init();
  }
  Plan pl;
  if (!make_plan(p, misc, tid, pl)) return;
  if (warp == W) {
    produce<D>(p, misc, pl, ring, lane);
    return;
  }

  const int g = lane >> 2, t = lane & 3, consumers = W * 32;
  int taken = 0;  // blocks of this CTA that earlier items had
#pragma unroll 1
  for (int u = pl.begin; u < pl.end;) {
    int e, head, ib;
    locate(p, misc, u, &e, &head, &ib);
    const int per = misc.entries[e + 1] - misc.entries[e];
    const int stop = min(ib + per, pl.end);
    const int len = lens_of(p, misc)[e];
    const bool there = len >= 0;
    const Span sp = span_of(there ? len : 0, p.window, p.sinks);
    const bool has_tail = stop == ib + per && there;
    const int b0 = u - ib, b1 = min(stop - ib, per - kTailUnits);
    const int seq = p.seqs ? p.seqs[e] : e;

    // queries and what their rows see
    Columns col;
    int low_max = 0;
    uint32_t any_vis = 0;
    const uint16_t* qrow = g < R ? p.q + query_at<D>(p, e, head, g) : nullptr;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = 2 * t + c, m = k < R ? k / p.group : 0;
      const uint32_t vis = (p.vis ? p.vis[(size_t)e * p.rows + m] : (2u << m) - 1u) & 0xFFu;
      col.vis[c] = vis;
      any_vis |= vis;
      col.low[c] = p.window > 0 ? len + __popc(vis) - p.window : 0;
      low_max = max(low_max, col.low[c]);
    }
    low_max = __reduce_max_sync(~0u, low_max);
    State<D> st;
    clear(st);
    uint32_t qf[D / 16][2];
    const float unit = load_query<D>(qf, qrow, lane);
    float coef[2];
    coef[0] = __shfl_sync(~0u, unit, 8 * t) * p.scale_log2;  // lane 4 g' holds column g'
    coef[1] = __shfl_sync(~0u, unit, 8 * t + 4) * p.scale_log2;
    if (has_tail) {
      const uint16_t* tail = v.tail(p.layer, seq, head);
      const int in_tail = len - sp.full * kKv8Block;
      const int there = in_tail + 32 - __clz((int)__reduce_or_sync(~0u, any_vis));  // at most 63 + 8
#pragma unroll 1
      for (int i = warp; i < 5; i += W)
        if (there > (i < 4 ? 4 * i : 64))
          tail_step<D>(st, tail, i, in_tail, len, there, qrow, p.scale_log2, col, p.sinks, lane);
    }
    bool ok = true;
    int k = b0 + ((warp - taken) % W + W) % W;  // ring positions taken + (k - b0) = warp mod W (S a multiple of W)
#pragma unroll 1
    for (; k < b1 && ok; k += W) {
      const int at = taken + (k - b0), stage = at % S;
      ok = dev::mbar_wait_bounded(&misc.full[stage], (uint32_t)((at / S) & 1), p.wait_ns);
      if (!__all_sync(~0u, ok)) {
        ok = false;
        break;
      }
      const int blk = k < sp.head_blocks ? k : sp.from + (k - sp.head_blocks);
      const int token0 = blk * kKv8Block;
      block_step<FMT, D>(st, ring + (size_t)stage * kRecord, qf, coef, col, token0,
                         token0 < low_max && token0 + kKv8Block > p.sinks, p.sinks, lane);
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&misc.empty[stage]);
    }
    if (!ok && lane == 0) misc.fail = 1;
    taken += b1 > b0 ? b1 - b0 : 0;

    // join the warps: sums over the lanes of a column, then over the warps
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = st.l[c];
      l += __shfl_xor_sync(~0u, l, 4);
      l += __shfl_xor_sync(~0u, l, 8);
      l += __shfl_xor_sync(~0u, l, 16);
      if (g == 0) {
        const int row = warp * 8 + 2 * t + c;
        warp_ml[2 * row] = st.m[c];
        warp_ml[2 * row + 1] = l * kUnit;  // as the weighted values
      }
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        merge[(size_t)(warp * 8 + 2 * t + (c & 1)) * kRow + 16 * j + g + 8 * (c >> 1)] = st.o[j][c];
    dev::named_barrier_sync(1, consumers);
    if (misc.fail) {
      if (tid == 0) report_wait(p);
      return;
    }
    finish<D, false>(p, misc, pl, merge, W * 8 * kRow, warp_ml, W, 8, e, head, ib, per, tid, consumers);
    dev::named_barrier_sync(1, consumers);  // the merge buffer is free again
    u = stop;
  }
}

// ---------------------------------------------------------------------------------------------------
// More than 8 queries, or head_dim 256: teams of four warps per block.
//
// With more tiles of queries, warps that each take a whole block would have to share out the
// queries and every one of them would turn the block's codes into f16 again, and few warps of many
// registers leave the tensor pipe waiting (40 queries: 25 % busy, 107 us at 65,531 tokens).  Here the four
// warps of a team share out the block instead: each works out the scores of 16 of its tokens (a
// quarter of the keys) for all NT tiles of queries, leaves the weights in shared memory, and
// after one barrier sums its quarter of the elements over all 64 tokens (a quarter of the values).  Codes are
// converted once, and a thread holds the weighted values of 2 NT fragments only.
//
// The running maxima belong to the team: weights are formed against them at once, and a score
// that passes its maximum by more than kRaise raises a flag that all four warps see behind that
// barrier; then (rarely) they agree on new maxima and form the weights again.
//
// Measured: issue 0.32 to 0.38 per cycle, tensor pipe 17 % (12 queries) to 32 % (40); what limits it is the chain
// products, exponentials, exchange, products of a block, which three teams in different blocks cover in part.
// Three teams: at 65,531 tokens x 40 queries 57 us (61 when two took 64), 32,785 x 12 24 (two: 26, four: 25 to
// 27).  With head_dim 256 two, of two tiles: shared memory holds four records beside what they exchange.
//
// Registers: the warps have 128 (168) a thread at launch.  The last four, of which one copies records and the others
// end, give up most of theirs to the teams (128 for all spill: two teams at 168 took 73 us, with 232 64).  With 152 the
// instances of head_dim 128 still spill, 36 to 68 bytes a thread with two to four tiles and 288 with five (455 thousand requests in 57 us).
__host__ __device__ constexpr int teams_of(int dim) { return dim == 256 ? 2 : 3; }
__host__ __device__ constexpr int team_tiles(int dim) { return dim == 256 ? 2 : 5; }  // most tiles of 8 queries
template <int D>
struct TeamShape {
  static constexpr int kTeams = teams_of(D), kThreads = 32 * (4 * kTeams + 4);
  static constexpr int kLaunch = kTeams == 2 ? 168 : 128, kCopying = 40, kTeam = kTeams == 2 ? 232 : 152;
  static_assert(kThreads * kLaunch <= 65536 && 128 * kCopying + 128 * kTeams * kTeam <= kThreads * kLaunch,
                "more registers than the launch has: the teams would wait for them for ever");
};

// Shared memory of one team: weights, twice (for two blocks in turn), column maxima of its warps, flags.
template <int NT>
struct TeamShared {
  uint4 weights[2][NT][2][32];  // [buffer][tile][pair of 16-token steps][lane]: operands of both steps
  float top[4][8 * NT];
  int raise[2];
};

__host__ __device__ constexpr int team_bytes(int nt) { return (2 * nt * 2 * 32 * 16 + 4 * 8 * nt * 4 + 8 + 127) / 128 * 128; }
// Queries as operands in shared memory: [tile][16 elements each][lane][2], kept there from three tiles on (24 queries,
// 32,768 tokens: 29 us, in registers, which then spill, 33; with two tiles 24 in registers, 25 in shared memory).
__host__ __device__ constexpr bool shared_queries(int nt, int dim) { return nt >= 3 || dim == 256; }
__host__ __device__ constexpr int query_bytes(int nt, int dim) { return shared_queries(nt, dim) ? nt * (dim / 16) * 32 * 8 : 0; }
// All that is not the ring: the join's buffer, the teams', the queries, and what their rows see.
__host__ __device__ constexpr int sight_bytes(int nt) { return (2 * 8 * nt * 4 + 127) / 128 * 128; }
__host__ __device__ inline int team_fixed_bytes(int nt, int dim) {
  return merge_bytes(teams_of(dim), nt, dim) + teams_of(dim) * team_bytes(nt) + query_bytes(nt, dim) + sight_bytes(nt);
}

template <int D, int NT>
struct TeamState {
  float m[NT][2], l[NT][2];  // maxima (the same in the team's warps), sums over this lane's tokens
  float o[D / 64][NT][4];
};

__device__ __forceinline__ void team_sync(int team) { dev::named_barrier_sync(2 + team, 128); }

// Weights against the maxima, rounded; their sums into l.
template <int D, int NT>
__device__ __forceinline__ void weigh(TeamState<D, NT>& st, const float (&s)[NT][4], float (&w)[NT][4], float (&l)[NT][2]) {
#pragma unroll
  for (int q = 0; q < NT; ++q) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float r = (st.m[q][c] == -INFINITY ? 0.0f : st.m[q][c]) - kOffset;
      w[q][c] = exp2_approx(s[q][c] - r);
      w[q][2 + c] = exp2_approx(s[q][2 + c] - r);
      l[q][c] = w[q][c] + w[q][2 + c];
    }
  }
}

// Agree on maxima that cover s, and scale what was summed.  The team's warps, between two barriers.
template <int D, int NT>
__device__ __forceinline__ void raise_team(TeamState<D, NT>& st, TeamShared<NT>& ts, const float (&s)[NT][4], int wi, int team,
                                           int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float x = column_max(fmaxf(s[q][c], s[q][2 + c]));
      if (g == 0) ts.top[wi][8 * q + 2 * t + c] = x;
    }
  team_sync(team);
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    float a[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float n = st.m[q][c];
#pragma unroll
      for (int w = 0; w < 4; ++w) n = fmaxf(n, ts.top[w][8 * q + 2 * t + c]);
      a[c] = n == -INFINITY ? 1.0f : exp2_approx(st.m[q][c] - n);
      st.m[q][c] = n;
      st.l[q][c] *= a[c];
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      st.o[j][q][0] *= a[0];
      st.o[j][q][1] *= a[1];
      st.o[j][q][2] *= a[0];
      st.o[j][q][3] *= a[1];
    }
  }
}

template <int D, int NT>
__device__ __forceinline__ bool passes(const TeamState<D, NT>& st, const float (&s)[NT][4]) {
  bool up = false;
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int c = 0; c < 2; ++c) up |= fmaxf(s[q][c], s[q][2 + c]) > st.m[q][c] + kRaise;
  return __any_sync(~0u, up);
}

// This warp's 16 tokens' weights (f16) into buffer `buf`.
template <int NT>
__device__ __forceinline__ void put_weights(TeamShared<NT>& ts, int buf, const float (&w)[NT][4], int wi, int lane) {
#pragma unroll
  for (int q = 0; q < NT; ++q)
    reinterpret_cast<uint2*>(&ts.weights[buf][q][wi >> 1][lane])[wi & 1] =
        make_uint2(transpose8x8(pack_f16(w[q][0], w[q][1])), transpose8x8(pack_f16(w[q][2], w[q][3])));
}

template <int FMT, int D, int NT, class Queries>
__device__ __forceinline__ void team_block(TeamState<D, NT>& st, TeamShared<NT>& ts, const uint8_t* rec, const Queries& queries,
                                           const float (&coef)[NT][2], const int* low, int token0, bool masked, int sinks,
                                           int buf, int wi, int team, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float ks = *reinterpret_cast<const float*>(rec + 128 * D);
  const float vs = *reinterpret_cast<const float*>(rec + 128 * D + 8);  // times kUnit
  const uint8_t* kc = rec + (2 * wi * (D / 16) + t) * 128 + g * 16;
  float s[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[q][c] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(kc + 4 * c * 128);
    const uint4 y = *reinterpret_cast<const uint4*>(kc + (D / 16 + 4 * c) * 128);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a[4];
      f16x4_of_codes<FMT>(xs[k], a[0], a[2]);
      f16x4_of_codes<FMT>(ys[k], a[1], a[3]);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const uint2 b = queries(q, 4 * c + k);
        mma_f16(s[q], a, b.x, b.y);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const float f0 = coef[q][0] * ks, f1 = coef[q][1] * ks;
    s[q][0] *= f0;
    s[q][1] *= f1;
    s[q][2] *= f0;
    s[q][3] *= f1;
  }
  if (masked) {
    const int tok = token0 + 16 * (g >> 1) + 4 * wi + (g & 1);
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int lo = low[8 * q + 2 * t + c];
        if (tok >= sinks && tok < lo) s[q][c] = -INFINITY;
        if (tok + 2 >= sinks && tok + 2 < lo) s[q][2 + c] = -INFINITY;
      }
  }
  float w[NT][4], l[NT][2];
  if (passes(st, s) && lane == 0) ts.raise[buf] = 1;
  weigh(st, s, w, l);
  put_weights<NT>(ts, buf, w, wi, lane);
  team_sync(team);
  if (ts.raise[buf]) {
    raise_team(st, ts, s, wi, team, lane);  // its barrier: every warp has read the flag
    if (wi == 0 && lane == 0) ts.raise[buf] = 0;
    weigh(st, s, w, l);
    put_weights<NT>(ts, buf, w, wi, lane);
    team_sync(team);
  }
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    st.l[q][0] += l[q][0];
    st.l[q][1] += l[q][1];
  }
  const uint8_t* vc = rec + 64 * D + t * 128 + g * 16 + wi * (D / 64) * 1024;
  // one strip of 16 elements after the other: the weights are read once for each, but the sums of one are all that is held
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const uint4 x = *reinterpret_cast<const uint4*>(vc + 2 * j * 512), y = *reinterpret_cast<const uint4*>(vc + (2 * j + 1) * 512);
    float acc[NT][4];
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[q][c] = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a0[4], a1[4];
      f16x4_of_codes<FMT>(h ? x.z : x.x, a0[0], a0[2]);
      f16x4_of_codes<FMT>(h ? y.z : y.x, a0[1], a0[3]);
      f16x4_of_codes<FMT>(h ? x.w : x.y, a1[0], a1[2]);
      f16x4_of_codes<FMT>(h ? y.w : y.y, a1[1], a1[3]);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const uint4 pb = ts.weights[buf][q][h][lane];
        mma_f16(acc[q], a0, pb.x, pb.y);
        mma_f16(acc[q], a1, pb.z, pb.w);
      }
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int c = 0; c < 4; ++c) st.o[j][q][c] = fmaf(vs, acc[q][c], st.o[j][q][c]);
  }
}

// The tail, or (over = true) its rows 64 .. 71: as team_block, from bf16 in global memory; weights as two
// bf16 parts, the high ones in buffer 0 and the low ones in buffer 1.
template <int D, int NT>
__device__ void team_tail(TeamState<D, NT>& st, TeamShared<NT>& ts, const uint16_t* tail, bool over, int in_tail, int len,
                          int there, const Kv8Attn& p, int e, int kv_head, int base, int R, const int* low, const uint32_t* vis, int wi, int team,
                          int lane) {
  const int g = lane >> 2, t = lane & 3;
  const bool mine = !over || wi == 0;  // this warp has tokens
  const int r0 = over ? 64 + g : 16 * (g >> 1) + 4 * wi + (g & 1), r1 = over ? kKv8Tail : r0 + 2;
  // every load is issued before the first product: they go to L2 or HBM, one round trip instead of one each
  const uint16_t* tv = tail + kKv8Tail * D + wi * (D / 4) * kKv8Tail;
  uint4 vx[D / 64][2], vy[D / 64][2];
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const uint16_t* v0 = tv + (16 * j + g) * kKv8Tail;
    const uint16_t* v1 = v0 + 8 * kKv8Tail;
    vx[j][0] = vx[j][1] = vy[j][0] = vy[j][1] = make_uint4(0, 0, 0, 0);
    if (over) {
      vx[j][0].x = *reinterpret_cast<const uint32_t*>(v0 + 64 + 2 * t);
      vy[j][0].x = *reinterpret_cast<const uint32_t*>(v1 + 64 + 2 * t);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        vx[j][h] = *reinterpret_cast<const uint4*>(v0 + 16 * t + 8 * h);
        vy[j][h] = *reinterpret_cast<const uint4*>(v1 + 16 * t + 8 * h);
      }
    }
  }
  float s[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[q][c] = mine ? 0.0f : -INFINITY;
  if (mine) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4 x[2], y[2], w[NT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = 16 * (4 * c + t) + 8 * h;
        x[h] = y[h] = make_uint4(0, 0, 0, 0);
        if (r0 < there) x[h] = *reinterpret_cast<const uint4*>(tail + r0 * D + d);
        if (r1 < there) y[h] = *reinterpret_cast<const uint4*>(tail + r1 * D + d);
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int n = min(8 * q + g, R - 1);  // columns from R on repeat the last query (their results are not used)
          w[q][h] = *reinterpret_cast<const uint4*>(p.q + query_at<D>(p, e, kv_head, base + n) + d);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a0[4] = {x[h].x, y[h].x, x[h].y, y[h].y}, a1[4] = {x[h].z, y[h].z, x[h].w, y[h].w};
#pragma unroll
        for (int q = 0; q < NT; ++q) mma_bf16(s[q], a0, w[q][h].x, w[q][h].y);
#pragma unroll
        for (int q = 0; q < NT; ++q) mma_bf16(s[q], a1, w[q][h].z, w[q][h].w);
      }
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = 8 * q + 2 * t + c;
        s[q][c] = tail_sees(r0, vis[k], low[k], in_tail, there, len, p.sinks) ? s[q][c] * p.scale_log2 : -INFINITY;
        s[q][2 + c] = tail_sees(r1, vis[k], low[k], in_tail, there, len, p.sinks) ? s[q][2 + c] * p.scale_log2 : -INFINITY;
      }
  }
  raise_team(st, ts, s, wi, team, lane);
  float w[NT][4], l[NT][2];
  weigh(st, s, w, l);
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    st.l[q][0] += l[q][0];
    st.l[q][1] += l[q][1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w0 = w[q][2 * h] * kUnit, w1 = w[q][2 * h + 1] * kUnit;
      const uint32_t u = pack_bf16(w0, w1);
      const float f0 = __uint_as_float(u << 16), f1 = __uint_as_float(u & 0xFFFF0000u);
      reinterpret_cast<uint32_t*>(&ts.weights[0][q][wi >> 1][lane])[2 * (wi & 1) + h] = transpose8x8(u);
      reinterpret_cast<uint32_t*>(&ts.weights[1][q][wi >> 1][lane])[2 * (wi & 1) + h] =
          transpose8x8(pack_bf16(w0 - f0, w1 - f1));
    }
  }
  team_sync(team);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const uint4 b = ts.weights[part][q][h][lane];
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint32_t a0[4] = {vx[j][h].x, vy[j][h].x, vx[j][h].y, vy[j][h].y};
          const uint32_t a1[4] = {vx[j][h].z, vy[j][h].z, vx[j][h].w, vy[j][h].w};
          mma_bf16(st.o[j][q], a0, b.x, b.y);
          mma_bf16(st.o[j][q], a1, b.z, b.w);
        }
      }
  team_sync(team);  // the buffers are free again
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(TeamShape<D>::kThreads, 1) attn_team_kernel(const __grid_constant__ Kv8Attn p) {
  extern __shared__ __align__(128) uint8_t smem[];
  using Shape = TeamShape<D>;
  constexpr bool kShared = shared_queries(NT, D);
  constexpr int kTeams = Shape::kTeams, kRecord = 128 * D + 16, kRow = D + kMergePad, W = 4 * kTeams, kQueries = 8 * NT;
  Misc& misc = *reinterpret_cast<Misc*>(smem);
  float* merge = reinterpret_cast<float*>(smem + misc_bytes(p.n));  // [teams][8 NT][D + pad]
  float* team_ml = merge + kTeams * kQueries * kRow;                // [teams][8 NT][2]
  uint8_t* at_teams = smem + misc_bytes(p.n) + merge_bytes(kTeams, NT, D);
  uint2* shared_q = reinterpret_cast<uint2*>(at_teams + kTeams * team_bytes(NT));
  int* low = reinterpret_cast<int*>(at_teams + kTeams * team_bytes(NT) + query_bytes(NT, D));  // [8 NT]
  uint32_t* vis = reinterpret_cast<uint32_t*>(low + kQueries);                                                 // [8 NT]
  uint8_t* ring = smem + misc_bytes(p.n) + team_fixed_bytes(NT, D);
  const Kv8View& v = p.v;
  const int S = p.stages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      dev::mbar_init(&misc.full[i], 1);
      dev::mbar_init(&misc.empty[i], 4);
    }
    misc.fail = 0;
    misc.wait_ns = p.wait_ns;
    dev::fence_mbar_init();
  }
  const int team = (warp >> 2) % kTeams, wi = warp & 3;
  TeamShared<NT>& ts = *reinterpret_cast<TeamShared<NT>*>(at_teams + team * team_bytes(NT));
  if (warp < W && wi == 0 && lane < 2) ts.raise[lane] = 0;
  Plan pl;
  if (!make_plan(p, misc, tid, pl)) return;
  if (warp >= W) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shape::kCopying));
    if (warp == W) produce<D>(p, misc, pl, ring, lane);
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shape::kTeam));

  int taken = 0;
#pragma unroll 1
  for (int u = pl.begin; u < pl.end;) {
    int e, head, ib;
    locate(p, misc, u, &e, &head, &ib);
    const int per = misc.entries[e + 1] - misc.entries[e];
    const int stop = min(ib + per, pl.end);
    const int len = lens_of(p, misc)[e];
    const bool there = len >= 0;
    const Span sp = span_of(there ? len : 0, p.window, p.sinks);
    const bool has_tail = stop == ib + per && there;
    const int b0 = u - ib, b1 = min(stop - ib, per - kTailUnits), blocks = max(0, b1 - b0);
    // this item's queries: [base, base + R) of the kv head
    const int kv_head = head / p.chunks, base = head % p.chunks * kQueries, R = min(kQueries, p.rows * p.group - base);

    // what the rows see
    int low_max = 0;
    uint32_t any_vis = 0;
#pragma unroll 1
    for (int k = lane; k < kQueries; k += 32) {
      const int m = (base + min(k, R - 1)) / p.group;
      const uint32_t x = (p.vis ? p.vis[(size_t)e * p.rows + m] : (2u << m) - 1u) & 0xFFu;
      const int lo = p.window > 0 ? len + __popc(x) - p.window : 0;
      any_vis |= x;
      low_max = max(low_max, lo);
      if (warp == 0) {
        low[k] = lo;
        vis[k] = x;
      }
    }
    low_max = __reduce_max_sync(~0u, low_max);
    any_vis = __reduce_or_sync(~0u, any_vis);
    // queries
    uint32_t qf[kShared ? 1 : NT][D / 16][2];
    float coef[NT][2];
    if constexpr (kShared) {
      float* units = team_ml;  // [8 NT], until the first join
#pragma unroll 1
      for (int q = warp; q < NT; q += W) {
        const int n = 8 * q + g;
        uint32_t f[D / 16][2];
        const float unit = load_query<D>(f, n < R ? p.q + query_at<D>(p, e, kv_head, base + n) : nullptr, lane);
        if (t == 0) units[n] = unit;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) shared_q[(q * (D / 16) + k) * 32 + lane] = make_uint2(f[k][0], f[k][1]);
      }
      dev::named_barrier_sync(1, W * 32);
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c) coef[q][c] = units[8 * q + 2 * t + c] * p.scale_log2;
    } else {
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const int n = 8 * q + g;
        const float unit = load_query<D>(qf[q], n < R ? p.q + query_at<D>(p, e, kv_head, base + n) : nullptr, lane);
        coef[q][0] = __shfl_sync(~0u, unit, 8 * t) * p.scale_log2;
        coef[q][1] = __shfl_sync(~0u, unit, 8 * t + 4) * p.scale_log2;
      }
      dev::named_barrier_sync(1, W * 32);
    }
    auto queries = [&](int q, int k) {
      if constexpr (kShared) return shared_q[(q * (D / 16) + k) * 32 + lane];
      else return make_uint2(qf[q][k][0], qf[q][k][1]);
    };
    TeamState<D, NT> st;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      st.m[q][0] = st.m[q][1] = -INFINITY;
      st.l[q][0] = st.l[q][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[j][q][c] = 0.0f;
    }
    if (has_tail && team == (taken + blocks) % kTeams) {  // the team whose turn comes next after the blocks
      const uint16_t* tail = v.tail(p.layer, p.seqs ? p.seqs[e] : e, kv_head);
      const int in_tail = len - sp.full * kKv8Block, rows = in_tail + 32 - __clz((int)any_vis);  // at most 63 + 8
      if (rows > 0) team_tail<D, NT>(st, ts, tail, false, in_tail, len, rows, p, e, kv_head, base, R, low, vis, wi, team, lane);
      if (rows > 64) team_tail<D, NT>(st, ts, tail, true, in_tail, len, rows, p, e, kv_head, base, R, low, vis, wi, team, lane);
    }
    bool ok = true;
    int k = b0 + ((team - taken) % kTeams + kTeams) % kTeams;  // S is a multiple of the teams
    for (int buf = 0; k < b1; k += kTeams, buf ^= 1) {
      const int at = taken + (k - b0), stage = at % S;
      // after a wait that ran out the warp goes on without waits (the team's barriers need it) but releases no stage,
      // so that the producer stops too; what it sums is not used
      if (ok) ok = __all_sync(~0u, dev::mbar_wait_bounded(&misc.full[stage], (uint32_t)((at / S) & 1), &misc.wait_ns));
      const int blk = k < sp.head_blocks ? k : sp.from + (k - sp.head_blocks);
      const int token0 = blk * kKv8Block;
      team_block<FMT, D, NT>(st, ts, ring + (size_t)stage * kRecord, queries, coef, low, token0,
                             token0 < low_max && token0 + kKv8Block > p.sinks, p.sinks, buf, wi, team, lane);
      __syncwarp();
      if (ok && lane == 0) dev::mbar_arrive(&misc.empty[stage]);
    }
    if (!ok && lane == 0) misc.fail = 1;
    taken += blocks;

    // join: the sums over a column's lanes and the team's warps, the weighted values as they are
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = st.l[q][c];
        l += __shfl_xor_sync(~0u, l, 4);
        l += __shfl_xor_sync(~0u, l, 8);
        l += __shfl_xor_sync(~0u, l, 16);
        if (g == 0) ts.top[wi][8 * q + 2 * t + c] = l;
      }
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          merge[(size_t)(team * kQueries + 8 * q + 2 * t + (c & 1)) * kRow + 16 * (wi * (D / 64) + j) + g + 8 * (c >> 1)] =
              st.o[j][q][c];
    dev::named_barrier_sync(1, W * 32);
    if (wi == 0) {
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (g == 0) {
            const int n = 8 * q + 2 * t + c;
            team_ml[2 * (team * kQueries + n)] = st.m[q][c];
            team_ml[2 * (team * kQueries + n) + 1] = ((ts.top[0][n] + ts.top[1][n]) + (ts.top[2][n] + ts.top[3][n])) * kUnit;
          }
    }
    dev::named_barrier_sync(1, W * 32);
    if (misc.fail) {
      if (tid == 0) report_wait(p);
      return;
    }
    finish<D, true>(p, misc, pl, merge, kTeams * kQueries * kRow, team_ml, kTeams, kQueries, e, head, ib, per, tid, W * 32);
    dev::named_barrier_sync(1, W * 32);  // the buffers are free again
    u = stop;
  }
}

// The parts that attn_team_kernel left, joined: a warp per query (head_dim 256: two), grid (items, warps /
// kJoinWarps).  With 12 to 40 queries one CTA alone takes 5 to 13 us over an item's parts (up to 0.4 MB) while
// the others have ended.
constexpr int kJoinWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Kv8Attn p) {
  begin_after_prior();
  const uint32_t failed = dev::ld_relaxed_u32(p.failed);  // beside the header's read and the place's
  const int2 where = p.joins[blockIdx.x];
  uint32_t magic;
  if (!is_ours(p.v, &magic)) return;  // nothing was left
  const int e = (int)blockIdx.x / p.heads, head = (int)blockIdx.x % p.heads, base = head % p.chunks * p.queries;
  constexpr int kParts = D > 128 ? D / 128 : 1;  // warps of one query
  const int Q = p.queries, lane = threadIdx.x & 31, w = (int)blockIdx.y * kJoinWarps + ((int)threadIdx.x >> 5);
  const int n = w / kParts, d0 = w % kParts * 128;
  const int np = where.y;
  // (after a wait that ran out a place may be one of an earlier launch: nothing outside the parts is read)
  if (where.x < 0 || np > p.ctas - (where.x >> 1)) return;
  if (np <= 1 || n >= min(Q, p.rows * p.group - base)) return;
  // the first part's slot, and the first slots of the CTAs that follow
  const size_t slot = (size_t)Q * (D + 4), step = 2 * slot;
  const float* parts = p.parts + (size_t)(where.x >> 1) * step;
  const size_t first = (where.x & 1) ? slot : 0;
  constexpr int kLanes = D / kParts / 4;  // lanes that hold four elements each
  const float* at = parts + (size_t)Q * D + 2 * n;
  const float* from = parts + (size_t)n * D + d0 + 4 * (lane % kLanes);
  constexpr int kAhead = 20;
  float4 y[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < np) y[i] = __ldcg(reinterpret_cast<const float4*>(from + i * step + (i == 0 ? first : 0)));
  float m = -INFINITY;
#pragma unroll 1
  for (int c = lane; c < np; c += 32) m = fmaxf(m, __ldcg(at + c * step + (c == 0 ? first : 0)));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  float4 o = {0, 0, 0, 0};
  float l = 0.0f;
#pragma unroll 1
  for (int cc = 0; cc < np; cc += 32) {
    const int c = cc + lane;
    float f = 0.0f;
    if (c < np) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(at + c * step + (c == 0 ? first : 0)));
      f = part_factor(ml.x, ml.y, m);
      l += f * ml.y;
    }
    const int some = min(32, np - cc);
    auto add = [&](int i, const float4& v) {
      const float fi = __shfl_sync(~0u, f, i);
      o.x += fi * v.x;
      o.y += fi * v.y;
      o.z += fi * v.z;
      o.w += fi * v.w;
    };
    int i = 0;
    if (cc == 0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < some) add(k, y[k]);
      i = min(some, kAhead);
    }
#pragma unroll 4
    for (; i < some; ++i) add(i, __ldcg(reinterpret_cast<const float4*>(from + (cc + i) * step)));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
  // After a wait that ran out some CTA left no parts, or no place of them: what is there may be an earlier launch's, of this
  // item or of another.  So nothing is joined, in this launch or (it is reported again) before the workspace is zero-filled.
  if (failed != 0) {
    if (lane == 0) flag(p.v, WOQ_DEVERR_TIMEOUT);
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = p.out + query_at<D>(p, e, head / p.chunks, base + n) + d0;
  if (lane < kLanes)
    *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

template <int D>
cudaError_t launch_join(const Kv8Attn& p, cudaStream_t stream) {
  const dim3 grid((unsigned)(p.n * p.heads), (unsigned)((p.queries * (D > 128 ? D / 128 : 1) + kJoinWarps - 1) / kJoinWarps));
  return launch(join_kernel<D>, grid, 32 * kJoinWarps, 0, stream, p);
}

// REGISTERS: what a kernel that hands registers from warp to warp was written for; with fewer its waits for them would not end.
template <void (*KERNEL)(Kv8Attn), int REGISTERS = 0>
cudaError_t launch_attn(const Kv8Attn& p, int ctas, int threads, int smem, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (device & 63);
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, max_dynamic_smem());
    if (e != cudaSuccess) return e;
    if (REGISTERS) {
      cudaFuncAttributes attr;
      e = cudaFuncGetAttributes(&attr, KERNEL);
      if (e != cudaSuccess) return e;
      if (attr.numRegs != REGISTERS) return cudaErrorLaunchOutOfResources;
    }
    configured.fetch_or(bit);
  }
  return launch(KERNEL, dim3((unsigned)ctas), threads, (size_t)smem, stream, p);
}

// The instances of a cache of FMT codes, by head size (and a team's query tiles).
template <int FMT>
cudaError_t launch_attn_any(const Kv8Attn& p, int ctas, int smem, cudaStream_t s) {
  const int threads = (p.warps + 1) * 32;
  switch (p.v.dim) {
    case 64: return launch_attn<attn_kernel<FMT, 64>>(p, ctas, threads, smem, s);
    case 128: return launch_attn<attn_kernel<FMT, 128>>(p, ctas, threads, smem, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int FMT, int D, int NT>
cudaError_t launch_team(const Kv8Attn& p, int ctas, int smem, cudaStream_t s) {
  using Shape = TeamShape<D>;
  const cudaError_t e = launch_attn<attn_team_kernel<FMT, D, NT>, Shape::kLaunch>(p, ctas, Shape::kThreads, smem, s);
  return e != cudaSuccess || !p.joined ? e : launch_join<D>(p, s);
}

template <int FMT>
cudaError_t launch_team_any(const Kv8Attn& p, int ctas, int smem, cudaStream_t s) {
  switch (p.v.dim * 8 + p.tiles) {
    case 64 * 8 + 2: return launch_team<FMT, 64, 2>(p, ctas, smem, s);
    case 64 * 8 + 3: return launch_team<FMT, 64, 3>(p, ctas, smem, s);
    case 64 * 8 + 4: return launch_team<FMT, 64, 4>(p, ctas, smem, s);
    case 64 * 8 + 5: return launch_team<FMT, 64, 5>(p, ctas, smem, s);
    case 128 * 8 + 2: return launch_team<FMT, 128, 2>(p, ctas, smem, s);
    case 128 * 8 + 3: return launch_team<FMT, 128, 3>(p, ctas, smem, s);
    case 128 * 8 + 4: return launch_team<FMT, 128, 4>(p, ctas, smem, s);
    case 128 * 8 + 5: return launch_team<FMT, 128, 5>(p, ctas, smem, s);
    case 256 * 8 + 1: return launch_team<FMT, 256, 1>(p, ctas, smem, s);
    case 256 * 8 + 2: return launch_team<FMT, 256, 2>(p, ctas, smem, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kv8
}  // namespace woq
