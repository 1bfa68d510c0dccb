// Rotary positions and append: from a qkv linear's output to queries in bf16 and to the cache.
//
// A pair of elements (a, b) is turned by table entry (c, s): a c - b s and b c + a s, each product
// and sum rounded to fp32 (no fused multiply-add, so the result is the same wherever it is
// computed), then to bf16.  Everything here is a stream bound by HBM (prompt) or by one chain of
// dependent loads (draft rows); the table is read through L2.
//
// Full blocks are quantised as a whole, from 64 rows of bf16 in shared memory: the largest
// magnitudes of keys and values, one scale each, and the codes in the record's order.  Rows are
// kept with their 16-byte vectors XORed by the place of the row in a core (row_swizzle), which
// makes both the row-wise writes and the core-wise reads free of bank conflicts.
#include "woq_internal.h"
#include "woq_kv8_device.cuh"

namespace woq {
namespace kv8 {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(256) rope_table_kernel(double theta, int half, int positions, float2* table) {
  const long long n = (long long)half * positions;
  for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < n; u += (long long)gridDim.x * blockDim.x) {
    const int i = (int)(u % half);
    const double f = pow(theta, -(double)(2 * i) / (double)(2 * half));
    double s, c;
    sincos((double)(u / half) * f, &s, &c);
    table[u] = make_float2((float)c, (float)s);
  }
}

// Elements d, d + 1 of a head's row, as fp32.
template <bool F32>
__device__ __forceinline__ float2 load2(const void* base, long long at) {
  if constexpr (F32) {
    return *reinterpret_cast<const float2*>(static_cast<const float*>(base) + at);
  } else {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + at);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
}

// The lane's part of one row's angles: frequencies 2 lane + 64 j and the one behind it, j = 0, 1.
struct Angles {
  float4 cs[2];  // c, s, c, s
};

__device__ __forceinline__ Angles load_angles(const Kv8Rope& r, const uint8_t* axis, int row, int rows, int lane,
                                              bool* bad) {
  Angles a;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * lane + 64 * j;
    if (i >= r.half) break;
    int p0 = r.pos[(size_t)axis[i] * rows + row], p1 = r.pos[(size_t)axis[i + 1] * rows + row];
    if (p0 < 0 || p0 >= r.positions) { *bad = true; p0 = 0; }
    if (p1 < 0 || p1 >= r.positions) { *bad = true; p1 = 0; }
    const float2* t = reinterpret_cast<const float2*>(r.table);
    const float2 x = __ldg(t + (size_t)p0 * r.half + i), y = __ldg(t + (size_t)p1 * r.half + i + 1);
    a.cs[j] = make_float4(x.x, x.y, y.x, y.y);
  }
  return a;
}

__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// Rotate and round one head's row (elements from `at`): emit(d, pair) for each pair of
// neighbouring elements d, d + 1.  One warp.
template <bool F32, class Emit>
__device__ __forceinline__ void rotate_row(const void* x, long long at, int dim, const Kv8Rope& r, const Angles& ang,
                                           int lane, Emit emit) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * lane + 64 * j;
    if (i >= r.half) break;
    const float4 cs = ang.cs[j];
    if (r.interleaved) {
      const float2 u = load2<F32>(x, at + 2 * i), w = load2<F32>(x, at + 2 * i + 2);
      const float2 p = turn(u.x, u.y, cs.x, cs.y), q = turn(w.x, w.y, cs.z, cs.w);
      emit(2 * i, pack_bf16(p.x, p.y));
      emit(2 * i + 2, pack_bf16(q.x, q.y));
    } else {
      const float2 u = load2<F32>(x, at + i), w = load2<F32>(x, at + r.half + i);
      const float2 p = turn(u.x, w.x, cs.x, cs.y), q = turn(u.y, w.y, cs.z, cs.w);
      emit(i, pack_bf16(p.x, q.x));
      emit(r.half + i, pack_bf16(p.y, q.y));
    }
  }
  for (int d = 2 * r.half + 2 * lane; d < dim; d += 64) {
    const float2 u = load2<F32>(x, at + d);
    emit(d, pack_bf16(u.x, u.y));
  }
}

template <bool F32, class Emit>
__device__ __forceinline__ void plain_row(const void* x, long long at, int dim, int lane, Emit emit) {
#pragma unroll 4
  for (int d = 2 * lane; d < dim; d += 64) {
    const float2 u = load2<F32>(x, at + d);
    emit(d, pack_bf16(u.x, u.y));
  }
}

// 64 rows of bf16 in shared memory, rows of D elements, 16-byte vectors swizzled.
__device__ __forceinline__ int row_swizzle(int token) { return ((token >> 4) << 1) | (token & 1); }
__device__ __forceinline__ int tile_at(int token, int d, int D) {  // element offset
  return token * D + (((d >> 3) ^ row_swizzle(token)) << 3) + (d & 7);
}

struct BlockShared {
  float top[2][kWarps];
  int bad;
  float scale[2], mul[2];
};

// Scales and codes of the block in kt, vt (shared memory) into rec.  All threads; barriers inside.
// bad: some row is not finite (its key NaN, its value 0): the key scale is NaN, so that every row
// that sees the block gets NaN.
template <int FMT>
__device__ void quantise_block(const uint16_t* kt, const uint16_t* vt, int D, bool bad, uint8_t* rec, BlockShared& sh) {
  uint32_t top[2] = {0, 0};
  for (int u = threadIdx.x; u < 64 * D / 8; u += kThreads) {
    const uint4 a = reinterpret_cast<const uint4*>(kt)[u], b = reinterpret_cast<const uint4*>(vt)[u];
    top[0] = dev::bf16x2_absmax(top[0], dev::bf16x2_absmax(dev::bf16x2_absmax(a.x, a.y), dev::bf16x2_absmax(a.z, a.w)));
    top[1] = dev::bf16x2_absmax(top[1], dev::bf16x2_absmax(dev::bf16x2_absmax(b.x, b.y), dev::bf16x2_absmax(b.z, b.w)));
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t m = __reduce_max_sync(~0u, __float_as_uint(dev::bf16x2_absmax_to_float(top[w])));
    if ((threadIdx.x & 31) == 0) sh.top[w][threadIdx.x >> 5] = __uint_as_float(m);
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float m = 0.0f;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.top[threadIdx.x][w]);
    float mul;
    const float s = block_scale<FMT>(m, &mul);
    sh.scale[threadIdx.x] = s;
    // a multiplier of 0 also stands for "take the division": amax below the corrected quotient's range
    sh.mul[threadIdx.x] = FMT == WOQ_KV8_INT8 && m < kQuotientMinAmax ? 0.0f : mul;
  }
  __syncthreads();
  const int chunks = 64 * D / 16;
  uint4* out = reinterpret_cast<uint4*>(rec);
  const float s0 = sh.scale[0], m0 = sh.mul[0], s1 = sh.scale[1], m1 = sh.mul[1];
  for (int c = threadIdx.x; c < chunks; c += kThreads) {
    const int core = c >> 3, p = (core / (D / 16)) * 8 + (c & 7), d = (core % (D / 16)) * 16;
    const int t = kv8_token_of_row(p);
    const uint4 a = *reinterpret_cast<const uint4*>(kt + tile_at(t, d, D));
    const uint4 b = *reinterpret_cast<const uint4*>(kt + tile_at(t, d + 8, D));
    uint4 w = {0, 0, 0, 0};
    if (!bad) {
      w.x = codes4<FMT>(a.x, a.y, s0, m0, m0 == 0.0f);
      w.y = codes4<FMT>(a.z, a.w, s0, m0, m0 == 0.0f);
      w.z = codes4<FMT>(b.x, b.y, s0, m0, m0 == 0.0f);
      w.w = codes4<FMT>(b.z, b.w, s0, m0, m0 == 0.0f);
    }
    out[c] = w;
  }
  for (int c = threadIdx.x; c < chunks; c += kThreads) {
    const int core = c >> 3, d = (core >> 2) * 8 + (c & 7), t = (core & 3) * 16;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = vt[tile_at(t + 4 * i + j, d, D)];
      w[i] = codes4<FMT>(x[0] | x[1] << 16, x[2] | x[3] << 16, s1, m1, m1 == 0.0f);
    }
    out[chunks + c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (threadIdx.x == 0) {
    const uint32_t ks = bad ? 0x7FC00000u : __float_as_uint(s0);
    *reinterpret_cast<uint4*>(rec + 128 * (size_t)D) = make_uint4(ks, __float_as_uint(s1), 0u, 0u);
  }
}

__device__ __forceinline__ void quantise_any(const Kv8View& v, const uint16_t* kt, const uint16_t* vt, bool bad,
                                             uint8_t* rec, BlockShared& sh) {
  if (v.fmt == WOQ_KV8_INT8) quantise_block<WOQ_KV8_INT8>(kt, vt, v.dim, bad, rec, sh);
  else quantise_block<WOQ_KV8_E4M3>(kt, vt, v.dim, bad, rec, sh);
}

// Rows r0 .. r1 - 1 of a tail into the tiles; returns whether this thread met one that is not finite.
__device__ bool tail_to_tiles(const uint16_t* tail, int r0, int r1, int D, uint16_t* kt, uint16_t* vt) {
  bool bad = false;
  for (int u = threadIdx.x; u < (r1 - r0) * (D / 8); u += kThreads) {
    const int r = r0 + u / (D / 8), d = (u % (D / 8)) * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(tail + (size_t)r * D + d);
    bad |= bf16_pair_not_finite(x.x) || bf16_pair_not_finite(x.y) || bf16_pair_not_finite(x.z) ||
           bf16_pair_not_finite(x.w);
    *reinterpret_cast<uint4*>(kt + tile_at(r, d, D)) = x;
  }
  const uint16_t* tv = tail + (size_t)kKv8Tail * D;
  for (int u = threadIdx.x; u < (r1 - r0) * D; u += kThreads) {
    const int d = u / (r1 - r0), r = r0 + u % (r1 - r0);
    vt[tile_at(r, d, D)] = tv[(size_t)d * kKv8Tail + r];
  }
  return bad;
}

// --------------------------------------------------------------------------- prompt

__device__ __forceinline__ void stage_axes(const Kv8Rope& r, uint8_t* axis) {
  for (int i = threadIdx.x; i < r.half; i += blockDim.x) axis[i] = r.axis_of[i];
  __syncthreads();
}

// Queries of a prompt: a warp per row, the row's angles in registers for all of its heads.
template <bool F32>
__global__ void __launch_bounds__(kThreads) prompt_q_kernel(const __grid_constant__ Kv8Append p) {
  __shared__ uint8_t axis[128];
  if (!header_ok(p.v)) return;
  stage_axes(p.rope, axis);
  const int lane = threadIdx.x & 31, row = blockIdx.x * kWarps + (threadIdx.x >> 5), D = p.v.dim;
  if (row >= p.rows) return;
  bool bad = false;
  const Angles ang = load_angles(p.rope, axis, row, p.rows, lane, &bad);
  if (__any_sync(~0u, bad) && lane == 0) flag(p.v, WOQ_DEVERR_POSITION);
  const long long at = (long long)row * p.row_stride;
  uint16_t* out = p.q_out + (size_t)row * p.q_heads * D;
#pragma unroll 4
  for (int h = 0; h < p.q_heads; ++h)
    rotate_row<F32>(p.qkv, at + (long long)h * D, D, p.rope, ang, lane,
                    [&](int d, uint32_t x) { *reinterpret_cast<uint32_t*>(out + (size_t)h * D + d) = x; });
}

// Keys and values of a prompt: grid (blocks, heads).  Block b of the sequence goes to its page if
// it is full, else to the tail.  The first block may have rows in the tail already; the CTA that reads
// those also writes the tail's new rows, after it (no other CTA writes what it reads).
template <bool F32>
__global__ void __launch_bounds__(kThreads) prompt_kv_kernel(const __grid_constant__ Kv8Append p) {
  extern __shared__ __align__(16) uint16_t tiles[];
  __shared__ uint8_t axis[128];
  __shared__ BlockShared sh;
  const Kv8View& v = p.v;
  if (!header_ok(v)) return;
  const int seq = p.n, T = p.rows, D = v.dim, head = blockIdx.y;
  const int len = v.lens_p()[seq], start = len - T;
  if (v.reserved_p()[seq] != T || start < 0) {
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
    return;
  }
  stage_axes(p.rope, axis);
  uint16_t *kt = tiles, *vt = tiles + 64 * D;
  uint16_t* tail = v.tail(p.layer, seq, head);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = start / kKv8Block, last = (len - 1) / kKv8Block, full = len / kKv8Block;
  const bool joined = start % kKv8Block != 0 && first < full && last == full;  // CTA 0 does the last block too
  int b = first + (int)blockIdx.x;
  if (b > last || (joined && b == last)) return;
  for (;;) {
    const int r0 = b == first ? start - first * kKv8Block : 0;  // rows of this call: r0 .. r1 - 1
    const int r1 = b == full ? len - full * kKv8Block : kKv8Block;
    bool bad = b < full && tail_to_tiles(tail, 0, r0, D, kt, vt);
#pragma unroll 2
    for (int r = r0 + warp; r < r1; r += kWarps) {
      const int row = b * kKv8Block + r - start;
      const long long at = (long long)row * p.row_stride + (long long)(p.q_heads + head) * D;
      bool far = false, odd = false;
      const Angles ang = load_angles(p.rope, axis, row, T, lane, &far);
      rotate_row<F32>(p.qkv, at, D, p.rope, ang, lane, [&](int d, uint32_t x) {
        odd |= bf16_pair_not_finite(x);
        *reinterpret_cast<uint32_t*>(kt + tile_at(r, d, D)) = x;
      });
      plain_row<F32>(p.qkv, at + (long long)v.heads * D, D, lane, [&](int d, uint32_t x) {
        odd |= bf16_pair_not_finite(x);
        *reinterpret_cast<uint32_t*>(vt + tile_at(r, d, D)) = x;
      });
      if (__any_sync(~0u, far) && lane == 0) flag(v, WOQ_DEVERR_POSITION);
      if (__any_sync(~0u, odd)) {  // the row's key becomes NaN and its value 0
        for (int d = 2 * lane; d < D; d += 64) {
          *reinterpret_cast<uint32_t*>(kt + tile_at(r, d, D)) = 0x7FC07FC0u;
          *reinterpret_cast<uint32_t*>(vt + tile_at(r, d, D)) = 0u;
        }
        bad = true;
      }
    }
    const bool any_bad = __syncthreads_or(bad);
    if (b < full) {
      quantise_any(v, kt, vt, any_bad, v.record(v.table_row(seq)[b], p.layer, head), sh);
    } else {
      for (int u = threadIdx.x; u < (r1 - r0) * (D / 8); u += kThreads) {
        const int r = r0 + u / (D / 8), d = (u % (D / 8)) * 8;
        *reinterpret_cast<uint4*>(tail + (size_t)r * D + d) = *reinterpret_cast<const uint4*>(kt + tile_at(r, d, D));
      }
      uint16_t* tv = tail + (size_t)kKv8Tail * D;
      for (int u = threadIdx.x; u < (r1 - r0) * D; u += kThreads) {
        const int d = u / (r1 - r0), r = r0 + u % (r1 - r0);
        tv[(size_t)d * kKv8Tail + r] = vt[tile_at(r, d, D)];
      }
    }
    if (!joined || b == last || blockIdx.x != 0) return;
    __syncthreads();
    b = last;
  }
}

// --------------------------------------------------------------------------- draft rows

// One warp per (row, query head or kv head).
template <bool F32>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ Kv8Append p) {
  __shared__ uint8_t axis[128];
  const Kv8View& v = p.v;
  stage_axes(p.rope, axis);
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  if (!header_ok(v)) return;
  const int lane = threadIdx.x & 31, D = v.dim, slots = p.q_heads + v.heads;
  const long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long rows = (long long)p.n * p.rows;
  if (u >= rows * slots) return;
  const int row = (int)(u / slots), slot = (int)(u % slots), e = row / p.rows, m = row % p.rows;
  const int seq = p.seqs ? p.seqs[e] : e;
  bool bad = seq < 0 || seq >= v.seqs;
  if (p.seqs)
    for (int i = lane; i < e; i += 32) bad |= p.seqs[i] == seq;
  if (__any_sync(~0u, bad)) {
    if (lane == 0) flag(v, WOQ_DEVERR_STATE);
    return;
  }
  const long long at = (long long)row * p.row_stride;
  bool far = false;
  const Angles ang = load_angles(p.rope, axis, row, (int)rows, lane, &far);
  if (__any_sync(~0u, far) && lane == 0) flag(v, WOQ_DEVERR_POSITION);
  if (slot < p.q_heads) {
    uint16_t* out = p.q_out + ((size_t)row * p.q_heads + slot) * D;
    rotate_row<F32>(p.qkv, at + (long long)slot * D, D, p.rope, ang, lane,
                    [&](int d, uint32_t x) { *reinterpret_cast<uint32_t*>(out + d) = x; });
    return;
  }
  const int head = slot - p.q_heads;
  const long long kat = at + (long long)(p.q_heads + head) * D, vat = kat + (long long)v.heads * D;
  const int r = v.lens_p()[seq] % kKv8Block + m;  // at most 63 + 7
  uint16_t* tail = v.tail(p.layer, seq, head);
  uint16_t* tk = tail + (size_t)r * D;
  uint16_t* tv = tail + (size_t)kKv8Tail * D + r;
  bool odd = false;
  rotate_row<F32>(p.qkv, kat, D, p.rope, ang, lane, [&](int d, uint32_t x) {
    odd |= bf16_pair_not_finite(x);
    *reinterpret_cast<uint32_t*>(tk + d) = x;
  });
  uint32_t vals[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = 2 * lane + 64 * j;
    if (d >= D) break;
    const float2 x = load2<F32>(p.qkv, vat + d);
    vals[j] = pack_bf16(x.x, x.y);
    odd |= bf16_pair_not_finite(vals[j]);
  }
  const bool any = __any_sync(~0u, odd);  // the row's key becomes NaN and its value 0
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = 2 * lane + 64 * j;
    if (d >= D) break;
    if (any) *reinterpret_cast<uint32_t*>(tk + d) = 0x7FC07FC0u;
    tv[(size_t)d * kKv8Tail] = any ? 0 : (uint16_t)vals[j];
    tv[(size_t)(d + 1) * kKv8Tail] = any ? 0 : (uint16_t)(vals[j] >> 16);
  }
}

// --------------------------------------------------------------------------- accepted rows

// moves[] of accept_meta_kernel, in one (entry, head, layer): kept rows go to the end of the
// tokens (each to a row at or below its own, in order); a block that is full goes to its page and
// the rows behind it to the tail's beginning.
__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ Kv8View v) {
  extern __shared__ __align__(16) uint16_t tiles[];
  __shared__ BlockShared sh;
  if (!header_ok(v)) return;
  const int4 m = v.moves_p()[blockIdx.x];
  const uint32_t keep = (uint32_t)m.y;
  if (keep == 0) return;
  const int D = v.dim, at = m.x % kKv8Block, kept = __popc(keep);
  uint16_t* tail = v.tail(blockIdx.z, m.w, blockIdx.y);
  uint16_t* tv = tail + (size_t)kKv8Tail * D;
  if ((keep & (keep + 1)) != 0) {  // not already in place
    for (int d = threadIdx.x; d < D; d += kThreads) {  // a thread moves one element of every row
      uint32_t left = keep;
      for (int j = 0; j < kept; ++j) {
        const int from = __ffs(left) - 1;
        left &= left - 1;
        tail[(size_t)(at + j) * D + d] = tail[(size_t)(at + from) * D + d];
        tv[(size_t)d * kKv8Tail + at + j] = tv[(size_t)d * kKv8Tail + at + from];
      }
    }
  }
  if (m.z < 0) return;
  __syncthreads();
  uint16_t *kt = tiles, *vt = tiles + 64 * D;
  const bool bad = __syncthreads_or(tail_to_tiles(tail, 0, kKv8Block, D, kt, vt));
  quantise_any(v, kt, vt, bad, v.record(m.z, blockIdx.z, blockIdx.y), sh);
  const int rest = at + kept - kKv8Block;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    for (int j = 0; j < rest; ++j) {
      tail[(size_t)j * D + d] = tail[(size_t)(kKv8Block + j) * D + d];
      tv[(size_t)d * kKv8Tail + j] = tv[(size_t)d * kKv8Tail + kKv8Block + j];
    }
  }
}

}  // namespace kv8

cudaError_t launch_rope_table(double theta, int half, int positions, float* table, cudaStream_t s) {
  const long long n = (long long)half * positions;
  const long long blocks = (n + 255) / 256;
  kv8::rope_table_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(theta, half, positions,
                                                                                  reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

cudaError_t launch_kv8_append_rows(const Kv8Append& p, cudaStream_t s) {
  const long long units = (long long)p.n * p.rows * (p.q_heads + p.v.heads);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)((units + kv8::kWarps - 1) / kv8::kWarps));
  lc.blockDim = dim3(kv8::kThreads);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return p.f32 ? cudaLaunchKernelEx(&lc, kv8::rows_kernel<true>, p) : cudaLaunchKernelEx(&lc, kv8::rows_kernel<false>, p);
}

// The tiles of a block take 256 D bytes: above 48 KB the kernel's limit is raised (head_dim 256).
template <class K>
static cudaError_t allow_tiles(K kernel, int bytes) {
  return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                           : cudaSuccess;
}

cudaError_t launch_kv8_prompt(const Kv8Append& p, cudaStream_t s) {
  const int smem = 256 * p.v.dim;
  const dim3 grid((unsigned)((p.rows - 1) / kKv8Block + 2), (unsigned)p.v.heads);
  cudaError_t e;
  if (p.f32) {
    if ((e = allow_tiles(kv8::prompt_kv_kernel<true>, smem)) != cudaSuccess) return e;
    kv8::prompt_kv_kernel<true><<<grid, kv8::kThreads, smem, s>>>(p);
  } else {
    if ((e = allow_tiles(kv8::prompt_kv_kernel<false>, smem)) != cudaSuccess) return e;
    kv8::prompt_kv_kernel<false><<<grid, kv8::kThreads, smem, s>>>(p);
  }
  if ((e = cudaGetLastError()) != cudaSuccess || p.q_heads == 0) return e;
  const unsigned blocks = (unsigned)((p.rows + kv8::kWarps - 1) / kv8::kWarps);
  if (p.f32) kv8::prompt_q_kernel<true><<<blocks, kv8::kThreads, 0, s>>>(p);
  else kv8::prompt_q_kernel<false><<<blocks, kv8::kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv8_accept_rows(const Kv8View& v, int n, cudaStream_t s) {
  const int smem = 256 * v.dim;
  const cudaError_t e = allow_tiles(kv8::accept_kernel, smem);
  if (e != cudaSuccess) return e;
  kv8::accept_kernel<<<dim3((unsigned)n, (unsigned)v.heads, (unsigned)v.layers), kv8::kThreads, smem, s>>>(v);
  return cudaGetLastError();
}

}  // namespace woq
