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
  begin_after_prior();
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

// The row's positions on each axis; one outside the table is reported and taken as 0.
struct Places {
  int p[4];
  __device__ __forceinline__ int of(int axis) const { return axis < 2 ? (axis ? p[1] : p[0]) : (axis == 2 ? p[2] : p[3]); }
};

__device__ __forceinline__ Places load_places(const Kv8Rope& r, int row, int rows, bool* bad) {
  Places a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a.p[i] = r.half > 0 && i < r.axes ? r.pos[(size_t)i * rows + row] : 0;
    if (a.p[i] < 0 || (r.half > 0 && a.p[i] >= r.positions)) {
      *bad = true;
      a.p[i] = 0;
    }
  }
  return a;
}

__device__ __forceinline__ Angles load_angles(const Kv8Rope& r, const uint8_t* axis, int row, int rows, int lane,
                                              bool* bad) {
  Angles a;
  const Places pl = load_places(r, row, rows, bad);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * lane + 64 * j;
    if (i >= r.half) break;
    const int p0 = pl.of(axis[i]), p1 = pl.of(axis[i + 1]);
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

// The same in 16-byte vectors, for heads that are rotated as a whole: half / 8 lanes a row, each for eight
// frequencies i0 .. i0 + 7 and their sixteen elements, two runs of eight (i0 and half + i0, or 2 i0 and
// 2 i0 + 8 if interleaved).
struct Angles8 {
  float2 cs[8];
};

__device__ __forceinline__ Angles8 load_angles8(const Kv8Rope& r, const uint8_t* axis, const Places& pl, int i0) {
  Angles8 a;
  const float2* t = reinterpret_cast<const float2*>(r.table);
  if (r.axes == 1) {
    const float4* from = reinterpret_cast<const float4*>(t + (size_t)pl.p[0] * r.half + i0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = __ldg(from + j);
      a.cs[2 * j] = make_float2(x.x, x.y);
      a.cs[2 * j + 1] = make_float2(x.z, x.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) a.cs[j] = __ldg(t + (size_t)pl.of(axis[i0 + j]) * r.half + i0 + j);
  }
  return a;
}

// Eight neighbouring elements from a 16-byte boundary.
template <bool F32>
struct Run8 {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, long long at) {
    const uint4* p = F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at)
                         : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    w[0] = __ldcs(p);
    if constexpr (F32) w[1] = __ldcs(p + 1);
  }
  __device__ __forceinline__ float operator[](int i) const {  // i a compile-time constant
    if constexpr (F32) {
      const uint4& v = w[i >> 2];
      return __uint_as_float((i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w);
    } else {
      const uint32_t v = (i >> 1) == 0 ? w[0].x : (i >> 1) == 1 ? w[0].y : (i >> 1) == 2 ? w[0].z : w[0].w;
      return __uint_as_float((i & 1) ? v & 0xFFFF0000u : v << 16);
    }
  }
  __device__ __forceinline__ uint4 rounded() const {
    return make_uint4(pack_bf16((*this)[0], (*this)[1]), pack_bf16((*this)[2], (*this)[3]), pack_bf16((*this)[4], (*this)[5]),
                      pack_bf16((*this)[6], (*this)[7]));
  }
};

template <bool F32>
__device__ __forceinline__ void rotate8(const Run8<F32>& x, const Run8<F32>& y, const Angles8& a, bool interleaved,
                                        uint4* u, uint4* v) {
  uint32_t o[8];
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = turn(x[2 * j], x[2 * j + 1], a.cs[j].x, a.cs[j].y);
      const float2 q = turn(y[2 * j], y[2 * j + 1], a.cs[4 + j].x, a.cs[4 + j].y);
      o[j] = pack_bf16(p.x, p.y);
      o[4 + j] = pack_bf16(q.x, q.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = turn(x[2 * j], y[2 * j], a.cs[2 * j].x, a.cs[2 * j].y);
      const float2 q = turn(x[2 * j + 1], y[2 * j + 1], a.cs[2 * j + 1].x, a.cs[2 * j + 1].y);
      o[j] = pack_bf16(p.x, q.x);
      o[4 + j] = pack_bf16(p.y, q.y);
    }
  }
  *u = make_uint4(o[0], o[1], o[2], o[3]);
  *v = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ bool not_finite8(const uint4& x) {
  return bf16_pair_not_finite(x.x) || bf16_pair_not_finite(x.y) || bf16_pair_not_finite(x.z) || bf16_pair_not_finite(x.w);
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
template <int FMT, int D>
__device__ __forceinline__ void quantise_block(const uint16_t* kt, const uint16_t* vt, bool bad, uint8_t* rec, BlockShared& sh) {
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
    *reinterpret_cast<uint4*>(rec + 128 * (size_t)D) = make_uint4(ks, __float_as_uint(s1), __float_as_uint(s1 * kUnit), 0u);
  }
}

// D: head_dim, or 0: as the cache says.
template <int D>
__device__ __forceinline__ void quantise_any(const Kv8View& v, const uint16_t* kt, const uint16_t* vt, bool bad, uint8_t* rec,
                                             BlockShared& sh) {
  if constexpr (D == 0) {
    if (v.dim == 64) quantise_any<64>(v, kt, vt, bad, rec, sh);
    else if (v.dim == 128) quantise_any<128>(v, kt, vt, bad, rec, sh);
    else quantise_any<256>(v, kt, vt, bad, rec, sh);
  } else {
    if (v.fmt == WOQ_KV8_INT8) quantise_block<WOQ_KV8_INT8, D>(kt, vt, bad, rec, sh);
    else quantise_block<WOQ_KV8_E4M3, D>(kt, vt, bad, rec, sh);
  }
}

// Rows 0 .. r1 - 1 of a tail into the tiles, row r from row from[r] (shared memory; the first `at` are in place);
// returns whether this thread met a key that is not finite.
__device__ bool tail_to_tiles(const uint16_t* tail, int r1, int at, const uint8_t* from, int D, uint16_t* kt, uint16_t* vt) {
  bool bad = false;
#pragma unroll 4
  for (int u = threadIdx.x; u < r1 * (D / 8); u += kThreads) {
    const int r = u / (D / 8), d = (u % (D / 8)) * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(tail + (size_t)(r < at ? r : from[r]) * D + d);
    bad |= not_finite8(x);
    *reinterpret_cast<uint4*>(kt + tile_at(r, d, D)) = x;
  }
  const uint16_t* tv = tail + (size_t)kKv8Tail * D;
  const int octets = (r1 + 7) / 8;
#pragma unroll 4
  for (int u = threadIdx.x; u < octets * D; u += kThreads) {  // lanes take neighbouring elements
    const int d = u % D, r = (u / D) * 8;
    uint32_t x[4];
    if (r + 8 <= at) {
      const uint4 y = *reinterpret_cast<const uint4*>(tv + (size_t)d * kKv8Tail + r);
      x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = r + 2 * i < r1 ? tv[(size_t)d * kKv8Tail + (r + 2 * i < at ? r + 2 * i : from[r + 2 * i])] : 0u;
        const uint32_t hi = r + 2 * i + 1 < r1 ? tv[(size_t)d * kKv8Tail + (r + 2 * i + 1 < at ? r + 2 * i + 1 : from[r + 2 * i + 1])] : 0u;
        x[i] = lo | hi << 16;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r + i < r1) vt[tile_at(r + i, d, D)] = (uint16_t)(x[i >> 1] >> (16 * (i & 1)));
  }
  return bad;
}

// --------------------------------------------------------------------------- prompt

__device__ __forceinline__ void stage_axes(const Kv8Rope& r, uint8_t* axis) {
  for (int i = threadIdx.x; i < r.half; i += blockDim.x) axis[i] = r.axis_of[i];
  __syncthreads();
}

// A prompt's rows in one launch: CTAs of keys and values, one per (block, head), and of queries, a warp per row, in
// turn.  LANES > 0: heads rotated as a whole, of 16 LANES elements, LANES lanes a head with
// 16-byte loads; else element pairs.
//
// Bound by HBM, so by the bytes under way: a thread issues the loads of its part of a full block (8 to 16
// vectors), or of kSteps heads, before it works on the first: 8,191 rows of 40 + 2 x 8 heads take 46 us (117 MB
// in, 101 MB out: 4.7 TB/s), 67 with the codes' read-back; as two launches with two to four vectors under way that took 99.
// By element pairs, 4-byte loads of bf16: the same rows with rot_dim 64 of 128 195 us, without rotation 175 (fp32: 254, 231).

// The row's angles stay in registers for all of its heads; a warp turns 32 / LANES heads at once.
template <bool F32, int LANES>
__device__ __forceinline__ void prompt_queries(const Kv8Append& p, const uint8_t* axis, int row, int lane) {
  if (row >= p.rows) return;
  bool bad = false;
  const long long at = (long long)row * p.row_stride;
  const int D = p.v.dim;
  uint16_t* out = p.q_out + (size_t)row * p.q_heads * D;
  if constexpr (LANES > 0) {
    constexpr int kD = 16 * LANES, kStep = 32 / LANES, kSteps = F32 ? 3 : 5;
    const int i0 = (lane % LANES) * 8;
    const int d0 = p.rope.interleaved ? 2 * i0 : i0, d1 = p.rope.interleaved ? d0 + 8 : 8 * LANES + i0;
    const Places pl = load_places(p.rope, row, p.rows, &bad);
    const Angles8 ang = load_angles8(p.rope, axis, pl, i0);
    for (int h0 = lane / LANES; h0 < p.q_heads; h0 += kStep * kSteps) {
      Run8<F32> x[kSteps], y[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int h = min(h0 + i * kStep, p.q_heads - 1);
        x[i].load(p.qkv, at + h * kD + d0);
        y[i].load(p.qkv, at + h * kD + d1);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int h = h0 + i * kStep;
        if (h >= p.q_heads) break;
        uint4 u, v;
        rotate8<F32>(x[i], y[i], ang, p.rope.interleaved, &u, &v);
        *reinterpret_cast<uint4*>(out + h * kD + d0) = u;
        *reinterpret_cast<uint4*>(out + h * kD + d1) = v;
      }
    }
  } else {
    const Angles ang = load_angles(p.rope, axis, row, p.rows, lane, &bad);
#pragma unroll 4
    for (int h = 0; h < p.q_heads; ++h)
      rotate_row<F32>(p.qkv, at + (long long)h * D, D, p.rope, ang, lane,
                      [&](int d, uint32_t x) { *reinterpret_cast<uint32_t*>(out + (size_t)h * D + d) = x; });
  }
  if (__any_sync(~0u, bad) && lane == 0) flag(p.v, WOQ_DEVERR_POSITION);
}

// Rows r0 .. r1 - 1 of block b (row r is row first_row + r of the call) into the tiles, keys rotated; a row with an
// element that is not finite sets odd_row[r].
template <bool F32, int LANES>
__device__ __forceinline__ void rows_to_tiles(const Kv8Append& p, const uint8_t* axis, int head, int first_row, int r0, int r1,
                                              uint16_t* kt, uint16_t* vt, int* odd_row, bool* far) {
  constexpr int D = 16 * LANES, kKeyRows = kThreads / LANES, kValueRows = kThreads / (2 * LANES);
  constexpr int kKeys = 64 / kKeyRows, kValues = 64 / kValueRows;  // passes
  const int i0 = ((int)threadIdx.x % LANES) * 8, kr = (int)threadIdx.x / LANES;
  const int d0 = p.rope.interleaved ? 2 * i0 : i0, d1 = p.rope.interleaved ? d0 + 8 : 8 * LANES + i0;
  const int vd = ((int)threadIdx.x % (2 * LANES)) * 8, vr = (int)threadIdx.x / (2 * LANES);
  const long long base = (long long)first_row * p.row_stride + (long long)(p.q_heads + head) * D;
  const long long vbase = base + (long long)p.v.heads * D + vd;
  Run8<F32> x[kKeys], y[kKeys], w[kValues];
  Places pl[kKeys];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int r = kr + i * kKeyRows;
    if (r < r0 || r >= r1) continue;
    x[i].load(p.qkv, base + (long long)r * p.row_stride + d0);
    y[i].load(p.qkv, base + (long long)r * p.row_stride + d1);
    pl[i] = load_places(p.rope, first_row + r, p.rows, far);
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int r = vr + i * kValueRows;
    if (r >= r0 && r < r1) w[i].load(p.qkv, vbase + (long long)r * p.row_stride);
  }
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int r = kr + i * kKeyRows;
    if (r < r0 || r >= r1) continue;
    const Angles8 ang = load_angles8(p.rope, axis, pl[i], i0);
    uint4 u, v;
    rotate8<F32>(x[i], y[i], ang, p.rope.interleaved, &u, &v);
    if (not_finite8(u) || not_finite8(v)) odd_row[r] = 1;
    *reinterpret_cast<uint4*>(kt + tile_at(r, d0, D)) = u;
    *reinterpret_cast<uint4*>(kt + tile_at(r, d1, D)) = v;
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int r = vr + i * kValueRows;
    if (r < r0 || r >= r1) continue;
    const uint4 u = w[i].rounded();
    if (not_finite8(u)) odd_row[r] = 1;
    *reinterpret_cast<uint4*>(vt + tile_at(r, vd, D)) = u;
  }
}

template <bool F32>
__device__ __forceinline__ void rows_to_tiles_by_pairs(const Kv8Append& p, const uint8_t* axis, int head, int first_row, int r0,
                                                       int r1, uint16_t* kt, uint16_t* vt, int* odd_row, bool* far) {
  const int D = p.v.dim, lane = threadIdx.x & 31;
#pragma unroll 2
  for (int r = r0 + (int)(threadIdx.x >> 5); r < r1; r += kWarps) {
    const int row = first_row + r;
    const long long at = (long long)row * p.row_stride + (long long)(p.q_heads + head) * D;
    bool odd = false;
    const Angles ang = load_angles(p.rope, axis, row, p.rows, lane, far);
    rotate_row<F32>(p.qkv, at, D, p.rope, ang, lane, [&](int d, uint32_t x) {
      odd |= bf16_pair_not_finite(x);
      *reinterpret_cast<uint32_t*>(kt + tile_at(r, d, D)) = x;
    });
    plain_row<F32>(p.qkv, at + (long long)p.v.heads * D, D, lane, [&](int d, uint32_t x) {
      odd |= bf16_pair_not_finite(x);
      *reinterpret_cast<uint32_t*>(vt + tile_at(r, d, D)) = x;
    });
    if (odd) odd_row[r] = 1;
  }
}

// Block b of the sequence goes to its page if it is full, else to the tail.  The first block may have rows in the tail
// already; the CTA that reads those also writes the tail's new rows, after it (no other CTA writes what it
// reads).
template <bool F32, int LANES>
__device__ __forceinline__ void prompt_block(const Kv8Append& p, const uint8_t* axis, int block, int head, uint16_t* tiles,
                                             int* odd_row, BlockShared& sh) {
  const Kv8View& v = p.v;
  const int seq = p.n, T = p.rows, D = LANES > 0 ? 16 * LANES : v.dim;
  const int len = v.lens_p()[seq], reserved = v.reserved_p()[seq], start = len - T;  // beside the header's read
  if (!header_ok(v)) return;
  if (reserved != T || start < 0) {
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
    return;
  }
  uint16_t *kt = tiles, *vt = tiles + 64 * D;
  uint16_t* tail = v.tail(p.layer, seq, head);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = start / kKv8Block, last = (len - 1) / kKv8Block, full = len / kKv8Block;
  const bool joined = start % kKv8Block != 0 && first < full && last == full;  // the first CTA does the last block too
  int b = first + block;
  if (b > last || (joined && b == last)) return;
  for (;;) {
    const int r0 = b == first ? start - first * kKv8Block : 0;  // rows of this call: r0 .. r1 - 1
    const int r1 = b == full ? len - full * kKv8Block : kKv8Block;
    const int page = b < full ? v.table_row(seq)[b] : 0;
    bool bad = b < full && tail_to_tiles(tail, r0, r0, nullptr, D, kt, vt), far = false;
    if (threadIdx.x < kKv8Block) odd_row[threadIdx.x] = 0;
    __syncthreads();
    if constexpr (LANES > 0) rows_to_tiles<F32, LANES>(p, axis, head, b * kKv8Block - start, r0, r1, kt, vt, odd_row, &far);
    else rows_to_tiles_by_pairs<F32>(p, axis, head, b * kKv8Block - start, r0, r1, kt, vt, odd_row, &far);
    if (__any_sync(~0u, far) && lane == 0) flag(v, WOQ_DEVERR_POSITION);
    __syncthreads();
    const int mine = (int)threadIdx.x < kKv8Block ? odd_row[threadIdx.x] : 0;
    if (__syncthreads_or(mine)) {  // a key that is not finite, or its value: the key becomes NaN and the value 0
      bad = true;
      for (int r = r0 + warp; r < r1; r += kWarps) {
        if (!odd_row[r]) continue;
        for (int d = 2 * lane; d < D; d += 64) {
          *reinterpret_cast<uint32_t*>(kt + tile_at(r, d, D)) = 0x7FC07FC0u;
          *reinterpret_cast<uint32_t*>(vt + tile_at(r, d, D)) = 0u;
        }
      }
    }
    const bool any_bad = __syncthreads_or(bad);
    if (b < full) {
      quantise_any<LANES * 16>(v, kt, vt, any_bad, v.record(page, p.layer, head), sh);
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
    if (!joined || b == last || block != 0) return;
    __syncthreads();
    b = last;
  }
}

template <bool F32, int LANES>
__global__ void __launch_bounds__(kThreads, F32 ? 2 : 3) prompt_kernel(const __grid_constant__ Kv8Append p, int blocks) {
  extern __shared__ __align__(16) uint16_t tiles[];
  __shared__ uint8_t axis[128];
  __shared__ int odd_row[kKv8Block];
  __shared__ BlockShared sh;
  stage_axes(p.rope, axis);
  begin_after_prior();
  // the two kinds in turn, so that an SM has some of each (the ones wait for chains of loads, the others for bandwidth)
  const int kv = blocks * p.v.heads, queries = (int)gridDim.x - kv, both = 2 * min(kv, queries), i = (int)blockIdx.x;
  const bool is_kv = i < both ? (i & 1) == 0 : kv > queries;
  const int k = i < both ? i >> 1 : i - both / 2;
  if (is_kv) prompt_block<F32, LANES>(p, axis, k / p.v.heads, k % p.v.heads, tiles, odd_row, sh);
  else if (header_ok(p.v)) prompt_queries<F32, LANES>(p, axis, k * kWarps + (int)(threadIdx.x >> 5), threadIdx.x & 31);
}

// --------------------------------------------------------------------------- draft rows

// One warp per (row, query head or kv head).
template <bool F32>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ Kv8Append p) {
  __shared__ uint8_t axis[128];
  const Kv8View& v = p.v;
  stage_axes(p.rope, axis);
  begin_after_prior();
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
  __shared__ uint8_t from[kKv8Tail];
  begin_after_prior();
  const int4 m = v.moves_p()[blockIdx.x];  // beside the header's read
  const uint32_t keep = (uint32_t)m.y;
  if (!header_ok(v) || keep == 0) return;
  const int D = v.dim, at = m.x % kKv8Block, kept = __popc(keep);
  if (threadIdx.x < WOQ_KV8_ROWS && (int)threadIdx.x < kept)  // where the kept rows are
    from[at + threadIdx.x] = (uint8_t)(at + __fns(keep, 0, (int)threadIdx.x + 1));
  __syncthreads();
  uint16_t* tail = v.tail(blockIdx.z, m.w, blockIdx.y);
  if (m.z >= 0) {  // rows 0 .. 63 to the page
    uint16_t *kt = tiles, *vt = tiles + 64 * D;
    const bool bad = __syncthreads_or(tail_to_tiles(tail, kKv8Block, at, from, D, kt, vt));
    quantise_any<0>(v, kt, vt, bad, v.record(m.z, blockIdx.z, blockIdx.y), sh);
  } else if ((keep & (keep + 1)) == 0) {
    return;  // in place already
  }
  // the other kept rows, each to its place in the tail: a thread moves one element of all of them (at most 8,
  // read before the first is written; rows that move lie at or behind the places they move to)
  const int first = m.z >= 0 ? kKv8Block : at, count = at + kept - first, to = m.z >= 0 ? 0 : at;
  for (int u = threadIdx.x; u < 2 * D; u += kThreads) {
    uint16_t* x = u < D ? tail + u : tail + (size_t)kKv8Tail * D + (size_t)(u - D) * kKv8Tail;
    const int step = u < D ? D : 1;
    uint16_t y[WOQ_KV8_ROWS];
#pragma unroll
    for (int j = 0; j < WOQ_KV8_ROWS; ++j)
      if (j < count) y[j] = x[from[first + j] * step];
#pragma unroll
    for (int j = 0; j < WOQ_KV8_ROWS; ++j)
      if (j < count) x[(to + j) * step] = y[j];
  }
}

}  // namespace kv8

cudaError_t launch_rope_table(double theta, int half, int positions, float* table, cudaStream_t s) {
  const long long n = (long long)half * positions;
  const long long blocks = (n + 255) / 256;
  return kv8::launch(kv8::rope_table_kernel, (unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s, theta, half, positions,
                     reinterpret_cast<float2*>(table));
}

cudaError_t launch_kv8_append_rows(const Kv8Append& p, cudaStream_t s) {
  const long long units = (long long)p.n * p.rows * (p.q_heads + p.v.heads);
  const unsigned blocks = (unsigned)((units + kv8::kWarps - 1) / kv8::kWarps);
  return kv8::launch(p.f32 ? kv8::rows_kernel<true> : kv8::rows_kernel<false>, blocks, kv8::kThreads, 0, s, p);
}

// The tiles of a block take 256 D bytes: above 48 KB the kernel's limit is raised (head_dim 256).
template <class K>
static cudaError_t allow_tiles(K kernel, int bytes) {
  return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                           : cudaSuccess;
}

template <bool F32, int LANES>
static cudaError_t launch_prompt(const Kv8Append& p, cudaStream_t s) {
  const int smem = 256 * p.v.dim, blocks = (p.rows - 1) / kKv8Block + 2;  // whatever the first token's place in its block
  const cudaError_t e = allow_tiles(kv8::prompt_kernel<F32, LANES>, smem);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)blocks * p.v.heads + (p.q_heads > 0 ? (p.rows + kv8::kWarps - 1) / kv8::kWarps : 0);
  return kv8::launch(kv8::prompt_kernel<F32, LANES>, (unsigned)ctas, kv8::kThreads, smem, s, p, blocks);
}

cudaError_t launch_kv8_prompt(const Kv8Append& p, cudaStream_t s) {
  const int lanes = p.rope.half * 2 == p.v.dim ? p.v.dim / 16 : 0;
  switch (lanes + (p.f32 ? 1 : 0)) {
    case 4: return launch_prompt<false, 4>(p, s);
    case 5: return launch_prompt<true, 4>(p, s);
    case 8: return launch_prompt<false, 8>(p, s);
    case 9: return launch_prompt<true, 8>(p, s);
    case 16: return launch_prompt<false, 16>(p, s);
    case 17: return launch_prompt<true, 16>(p, s);
    default: return p.f32 ? launch_prompt<true, 0>(p, s) : launch_prompt<false, 0>(p, s);
  }
}

cudaError_t launch_kv8_accept_rows(const Kv8View& v, int n, cudaStream_t s) {
  const int smem = 256 * v.dim;
  const cudaError_t e = allow_tiles(kv8::accept_kernel, smem);
  if (e != cudaSuccess) return e;
  return kv8::launch(kv8::accept_kernel, dim3((unsigned)n, (unsigned)v.heads, (unsigned)v.layers), kv8::kThreads, smem, s, v);
}

}  // namespace woq
