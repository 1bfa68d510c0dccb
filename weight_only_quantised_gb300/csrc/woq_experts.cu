// Experts' products over packed int4 / int6 weights (include/woq_block.h):
//   h_e,t = silu(G_e x_t) * U_e x_t,   part = D_e h,   y_t = sum_j w_tj part_tj.
//
// A decode step's few rows choose many experts, so a launch is bound by the bytes of the chosen experts' weights, each
// read once.  Three steps behind a plan of one CTA that lists the chosen experts with their rows:
//   gate and up (with silu and product), down, and the weighted sum of each row's places.
// A CTA works on a few 16-row tiles of one expert over all of K, its warps on the groups in turn: a warp loads its tiles'
// weights straight into the registers that the matrix instructions take them from (the packed layout was made for
// m16n8k16 fragments: lane 4 g + t reads quarter t of rows g and g + 8), so all loads of a group are under way at once
// and nothing passes through shared memory but the warps' partial sums at the end.
//   A: weights, nibbles made bf16 exactly (128 + w + 8 by one LOP3, less 136);  B: the rows of x, 8 at a time;
//   products are exact and sums fp32; a group's sum is multiplied by its row's scale in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "woq_block.h"
#include "woq_block_internal.h"
#include "woq_device.cuh"
#include "woq_kv8_device.cuh"
#include "woq_layout.h"
#include "woq_prologue.cuh"

namespace woq {
namespace experts {

constexpr int kWarps = 8;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ bool matrix_ok(const uint8_t* m, int bits, int N, int K) {
  const PackedHeader* h = reinterpret_cast<const PackedHeader*>(m);
  return h->magic == kMagic && h->version == kLayoutVersion && h->bits == (uint32_t)bits && h->N == (uint32_t)N &&
         h->K == (uint32_t)K;
}

// One CTA: places by expert, and the items (up to kExpertRows places of one expert).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Experts p) {
  __shared__ int s_next[1024], s_sums[33];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  if (tid == 0) s_bad = 0;
  s_next[tid] = 0;
  __syncthreads();
  int flags = 0;
  if (tid < p.experts && !(matrix_ok(p.gate_up + (size_t)tid * p.gate_up_stride, p.bits, 2 * p.inner, p.hidden) &&
                           matrix_ok(p.down + (size_t)tid * p.down_stride, p.bits, p.hidden, p.inner)))
    flags = WOQ_DEVERR_HEADER;
  for (int i = tid; i < p.entries; i += kPlanThreads) {
    const int e = p.ids[i];
    if ((unsigned)e < (unsigned)p.experts) atomicAdd(&s_next[e], 1);
    else if (e != -1) flags |= WOQ_DEVERR_STATE;
  }
  if (flags) atomicOr(&s_bad, flags);
  __syncthreads();
  const int count = s_next[tid];
  int total, items;
  const int first = kv8::block_exclusive_sum(count, s_sums, &total);
  __syncthreads();
  const int item = kv8::block_exclusive_sum((count + kExpertRows - 1) / kExpertRows, s_sums, &items);
  s_next[tid] = first;
  __syncthreads();
  for (int i = 0; i < count; i += kExpertRows)
    p.item[item + i / kExpertRows] = ExpertItem{tid, first + i, count - i < kExpertRows ? count - i : kExpertRows, 0};
  // The order of an expert's places may differ from run to run; each is a column of its own, so no result does.
  for (int i = tid; i < p.entries; i += kPlanThreads) {
    const int e = p.ids[i];
    if ((unsigned)e < (unsigned)p.experts) p.order[atomicAdd(&s_next[e], 1)] = i;
  }
  if (tid == 0) {
    const bool stop = s_bad & WOQ_DEVERR_HEADER;
    p.status[1] = stop ? 0u : (uint32_t)items;
    p.status[2] = stop;
    if (s_bad) atomicOr(p.status, (uint32_t)s_bad);
  }
}

__device__ __forceinline__ uint4 load_weights(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load_weights8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// A word of eight weights k0 .. k0+7 as bf16 pairs (0,2) (1,3) (4,6) (5,7); u: int6's word of top bits, i: the word's
// number.  Nibble b is the bf16 128 + b with exponent 0x4300; the top bit of the code is flipped, so that b = w + 8 (32).
template <int BITS>
__device__ __forceinline__ void unpack8(uint32_t v, uint32_t u, int i, uint32_t (&a)[4]) {
  if constexpr (BITS == 4) {
    const uint32_t off = 0x43084308u, sub = 0x43084308u;  // 128 + 8
    a[0] = less((v & 0x000F000Fu) ^ off, sub);
    a[1] = less(((v >> 8) & 0x000F000Fu) ^ off, sub);
    a[2] = less(((v >> 4) & 0x000F000Fu) ^ off, sub);
    a[3] = less(((v >> 12) & 0x000F000Fu) ^ off, sub);
  } else {
    const uint32_t off = 0x43204320u, sub = 0x43204320u;  // 128 + 32
    const uint32_t w = (i & 1) ? u >> 4 : u;              // bits 0..1: the low nibbles' top bits, 2..3: the high ones'
    a[0] = less(((v & 0x000F000Fu) | ((w << 4) & 0x00300030u)) ^ off, sub);
    a[1] = less((((v >> 8) & 0x000F000Fu) | ((w >> 4) & 0x00300030u)) ^ off, sub);
    a[2] = less((((v >> 4) & 0x000F000Fu) | ((w << 2) & 0x00300030u)) ^ off, sub);
    a[3] = less((((v >> 12) & 0x000F000Fu) | ((w >> 6) & 0x00300030u)) ^ off, sub);
  }
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The weights of one 16-row tile and group as a lane holds them.
template <int BITS>
struct Tile {
  uint4 w[2];
  uint2 hi[2];
  uint32_t scale[2];
};

// Rows row0 .. row0 + 15 of the matrix, group g.
template <int BITS>
__device__ __forceinline__ void load_tile(Tile<BITS>& t, const uint8_t* matrix, int groups, int row0, int g, int lane) {
  const uint8_t* block = matrix + kHeaderBytes + ((size_t)(row0 >> 7) * groups + g) * block_bytes(BITS);
  const int r = row0 & 127, j = r >> 5, q = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int l = (r & 31) + (lane >> 2) + 8 * i;
    t.w[i] = load_weights(block + w4_chunk_offset(q, j, l));
    if (BITS == 6) t.hi[i] = load_weights8(block + hi_chunk_offset(q, j, l));
    t.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(block) + 4 * l + j);
  }
}

// GATED: rows of gate and up, silu and product, h; else the down projection's parts.
// A CTA takes TILES 16-row tiles (of gate, and the same of up) of one item.
template <int BITS, bool GATED, int TILES>
__global__ void __launch_bounds__(kWarps * 32) product_kernel(const Experts p) {
  constexpr int kMats = GATED ? 2 : 1, kRows = 16 * TILES;
  __shared__ float s_sum[kWarps][kMats][kRows][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  if (blockIdx.y >= p.status[1]) return;
  const ExpertItem it = p.item[blockIdx.y];
  const int K = GATED ? p.hidden : p.inner, groups = K / kGroup;
  const int row0 = blockIdx.x * kRows;
  const uint8_t* matrix = GATED ? p.gate_up + (size_t)it.expert * p.gate_up_stride : p.down + (size_t)it.expert * p.down_stride;
  // the row of x (or h) that this lane's column of B is
  const int col = lane >> 2;
  const uint16_t* b_row = nullptr;
  if (col < it.rows) {
    const int place = p.order[it.first + col];
    b_row = GATED ? p.x + (size_t)(place / p.k) * K : p.h + (size_t)place * K;
  }
  float acc[kMats * TILES][4];
#pragma unroll
  for (int i = 0; i < kMats * TILES; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int g = warp; g < groups; g += kWarps) {
    Tile<BITS> tile[kMats * TILES];
#pragma unroll
    for (int i = 0; i < kMats * TILES; ++i)
      load_tile<BITS>(tile[i], matrix, groups, row0 + (i / TILES) * p.inner + (i % TILES) * 16, g, lane);
    uint32_t b[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (b_row) v = *reinterpret_cast<const uint4*>(b_row + (size_t)g * kGroup + (lane & 3) * 32 + i * 8);
      b[i][0] = __byte_perm(v.x, v.y, 0x5410);  // k 0, 2
      b[i][1] = __byte_perm(v.x, v.y, 0x7632);  // 1, 3
      b[i][2] = __byte_perm(v.z, v.w, 0x5410);  // 4, 6
      b[i][3] = __byte_perm(v.z, v.w, 0x7632);  // 5, 7
    }
#pragma unroll
    for (int i = 0; i < kMats * TILES; ++i) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const uint32_t w[2][4] = {{tile[i].w[0].x, tile[i].w[0].y, tile[i].w[0].z, tile[i].w[0].w},
                                {tile[i].w[1].x, tile[i].w[1].y, tile[i].w[1].z, tile[i].w[1].w}};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) unpack8<BITS>(w[r][j], BITS == 6 ? (j < 2 ? tile[i].hi[r].x : tile[i].hi[r].y) : 0u, j, a[r]);
        mma(d, a[0][0], a[1][0], a[0][1], a[1][1], b[j][0], b[j][1]);
        mma(d, a[0][2], a[1][2], a[0][3], a[1][3], b[j][2], b[j][3]);
      }
      const float s0 = dev::half_bits_to_float(tile[i].scale[0]), s1 = dev::half_bits_to_float(tile[i].scale[1]);
      acc[i][0] = fmaf(s0, d[0], acc[i][0]);
      acc[i][1] = fmaf(s0, d[1], acc[i][1]);
      acc[i][2] = fmaf(s1, d[2], acc[i][2]);
      acc[i][3] = fmaf(s1, d[3], acc[i][3]);
    }
  }
#pragma unroll
  for (int i = 0; i < kMats * TILES; ++i) {
    const int r = (i % TILES) * 16 + (lane >> 2), c = (lane & 3) * 2;
    *reinterpret_cast<float2*>(&s_sum[warp][i / TILES][r][c]) = make_float2(acc[i][0], acc[i][1]);
    *reinterpret_cast<float2*>(&s_sum[warp][i / TILES][r + 8][c]) = make_float2(acc[i][2], acc[i][3]);
  }
  __syncthreads();
  for (int i = tid; i < kRows * it.rows; i += kWarps * 32) {
    const int c = i / kRows, r = i % kRows;
    const int place = p.order[it.first + c];
    float v[kMats];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      v[m] = s_sum[0][m][r][c];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) v[m] += s_sum[w][m][r][c];
    }
    if constexpr (GATED) p.h[(size_t)place * p.inner + row0 + r] = (uint16_t)pro::f32_to_bf16_bits(v[0] / (1.0f + expf(-v[0])) * v[1]);
    else p.parts[(size_t)place * p.hidden + row0 + r] = v[0];
  }
}

// y_t = sum over its places, in their order.
__global__ void __launch_bounds__(256) sum_kernel(const Experts p) {
  const int row = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  if (c >= p.hidden || p.status[2]) return;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j = 0; j < p.k; ++j) {
    const size_t place = (size_t)row * p.k + j;
    if ((unsigned)p.ids[place] >= (unsigned)p.experts) continue;
    const float w = p.weights[place];
    const float4 v = *reinterpret_cast<const float4*>(p.parts + place * p.hidden + c);
    y.x = fmaf(w, v.x, y.x);
    y.y = fmaf(w, v.y, y.y);
    y.z = fmaf(w, v.z, y.z);
    y.w = fmaf(w, v.w, y.w);
  }
  *reinterpret_cast<uint2*>(p.y + (size_t)row * p.hidden + c) =
      make_uint2(pro::f32_to_bf16_bits(y.x) | pro::f32_to_bf16_bits(y.y) << 16,
                 pro::f32_to_bf16_bits(y.z) | pro::f32_to_bf16_bits(y.w) << 16);
}

template <int BITS>
static cudaError_t launch_bits(const Experts& p, cudaStream_t s) {
  cudaError_t e = kv8::launch(plan_kernel, dim3(1), kPlanThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  e = kv8::launch(product_kernel<BITS, true, 1>, dim3((unsigned)(p.inner / 16), (unsigned)p.items), kWarps * 32, 0, s, p);
  if (e != cudaSuccess) return e;
  e = kv8::launch(product_kernel<BITS, false, 1>, dim3((unsigned)(p.hidden / 16), (unsigned)p.items), kWarps * 32, 0, s, p);
  if (e != cudaSuccess) return e;
  return kv8::launch(sum_kernel, dim3((unsigned)p.rows, (unsigned)((p.hidden + 1023) / 1024)), 256, 0, s, p);
}

}  // namespace experts

cudaError_t launch_experts(const Experts& p, cudaStream_t s) {
  return p.bits == 4 ? experts::launch_bits<4>(p, s) : experts::launch_bits<6>(p, s);
}

}  // namespace woq
