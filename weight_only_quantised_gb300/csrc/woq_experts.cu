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
#include <math.h>
#include <stdlib.h>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "woq_block.h"
#include "woq_block_internal.h"
#include "woq_device.cuh"
#include "woq_internal.h"
#include "woq_kv8_device.cuh"
#include "woq_layout.h"
#include "woq_prologue.cuh"

namespace woq {
namespace experts {

constexpr int kWarps = 16;
constexpr int kPlanThreads = 1024;
constexpr int kSmallEntries = 256;  // places that every CTA sorts out for itself

__device__ __forceinline__ bool matrix_ok(const uint8_t* m, int bits, int N, int K) {
  const PackedHeader* h = reinterpret_cast<const PackedHeader*>(m);
  return h->magic == kMagic && h->version == kLayoutVersion && h->bits == (uint32_t)bits && h->N == (uint32_t)N &&
         h->K == (uint32_t)K;
}

// One CTA: places by expert, and the items (up to kExpertRows places of one expert).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Experts p) {
  __shared__ int s_next[1024], s_sums[33];
  const int tid = threadIdx.x;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  s_next[tid] = 0;
  __syncthreads();
  for (int i = tid; i < p.entries; i += kPlanThreads) {
    const int e = p.ids[i];
    if ((unsigned)e < (unsigned)p.experts) atomicAdd(&s_next[e], 1);
  }
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
  if (tid == 0) p.status[1] = (uint32_t)items;
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

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Which experts are worked on, and for which places: with up to kSmallEntries places every CTA sorts them out for itself
// (shared memory), else plan_kernel has (global memory).
struct Plan {
  int items;
  int expert[kSmallEntries];
  int rows[kSmallEntries];
  int place[kSmallEntries][kExpertRows];
  // scratch
  alignas(16) int ids[kSmallEntries];
  int number[kSmallEntries];
  int starts[kSmallEntries / 32];
};

// One place a thread.  A place's turn is the number of places before it with the same expert; every kExpertRows-th
// starts an item.
__device__ __forceinline__ void plan_here(const Experts& p, Plan& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool here = tid < kSmallEntries;
  int e = -1;
  if (tid < p.entries) {
    e = p.ids[tid];
    if ((unsigned)e >= (unsigned)p.experts) e = -1;
  }
  if (here) s.ids[tid] = e, s.rows[tid] = 0;
  __syncthreads();
  int turn = 0, leader = tid;
  if (e >= 0) {
    const int4* v = reinterpret_cast<const int4*>(s.ids);
    for (int i = 0; i < tid; i += 4) {
      const int4 o = v[i >> 2];
      const int w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (w[j] == e && i + j < tid) {
          if (turn % kExpertRows == 0) leader = i + j;
          ++turn;
        }
    }
    if (turn % kExpertRows == 0) leader = tid;
  }
  const bool start = e >= 0 && leader == tid;
  const unsigned starts = __ballot_sync(~0u, start);
  if (here && lane == 0) s.starts[warp] = __popc(starts);
  __syncthreads();
  if (here) {
    int number = __popc(starts & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) number += s.starts[w];
    s.number[tid] = number;
    if (start) s.expert[number] = e;
    if (tid == kSmallEntries - 1) s.items = number + start;
  }
  __syncthreads();
  if (e >= 0) {
    const int item = s.number[leader];
    s.place[item][turn % kExpertRows] = tid;
    atomicAdd(&s.rows[item], 1);
  }
  __syncthreads();
}

// A stage of a warp's ring: the weights of one group (128 k) for two 16-row tiles, as lanes take them; every lane reads back
// only what it copied itself, so a warp's ring needs no barrier.
template <int BITS>
constexpr int kStageBytes = 2048 + 512 + (BITS == 6 ? 1024 : 0);
template <int BITS>
constexpr int kStageCount = BITS == 4 ? 4 : 3;
constexpr int kPartBytes = 2 * kWarps * 32 * 32;  // two buffers of the warps' sums, 8 floats a lane
template <int BITS>
constexpr int kSharedBytes = kWarps * kStageCount<BITS> * kStageBytes<BITS> + kPartBytes + (int)((sizeof(Plan) + 15) / 16 * 16);

// GATED: rows of gate and up, silu and product, h; else the down projection's parts.  One CTA per SM; a team of `split`
// warps works on units (an item's 16 rows of gate and the same of up, or 32 rows of down) in turn.
template <int BITS, bool GATED, bool SMALL>
__global__ void __launch_bounds__(kWarps * 32, 1) product_kernel(const Experts p) {
  extern __shared__ __align__(16) uint8_t s_mem[];
  constexpr int kStage = kStageBytes<BITS>, kStages = kStageCount<BITS>, kBlock = BITS == 4 ? kBlockBytesW4 : kBlockBytesW6;
  float4* const s_part = reinterpret_cast<float4*>(s_mem + kWarps * kStages * kStage);
  Plan& s = *reinterpret_cast<Plan*>(s_mem + kWarps * kStages * kStage + kPartBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The down projection's launch may read the ids (and the plan), which were there before the one it waits for began.
  if (GATED) dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  int items;
  if constexpr (SMALL) {
    plan_here(p, s);
    items = s.items;
  } else {
    items = (int)p.status[1];
  }
  const int K = GATED ? p.hidden : p.inner, groups = K / kGroup;
  const int slices = GATED ? p.inner / 16 : p.hidden / 32;
  const int units = items * slices;
  const int split = GATED ? p.split_up : p.split_down, teams = (int)gridDim.x * (kWarps / split);
  const int team = (int)blockIdx.x + (int)gridDim.x * (warp / split), member = warp & (split - 1);
  const uint8_t* const matrices = GATED ? p.gate_up : p.down;
  const size_t stride = GATED ? p.gate_up_stride : p.down_stride;
  // from the first tile to the second
  const size_t next_w = GATED ? (size_t)(p.inner / kTileRows) * groups * kBlock : 256;
  const size_t next_s = GATED ? next_w : 128;
  const int q = lane & 3, col = lane >> 2;

  // The copies run stages ahead of the work.
  int ahead_unit = team, ahead_g = member;
  const uint8_t *src_w = nullptr, *src_s = nullptr, *src_h = nullptr;
  const auto locate = [&]() {
    const int item = ahead_unit / slices, row0 = (ahead_unit - item * slices) * (GATED ? 16 : 32);
    const int expert = SMALL ? s.expert[item] : p.item[item].expert;
    const uint8_t* block = matrices + (size_t)expert * stride + kHeaderBytes + ((size_t)(row0 >> 7) * groups + ahead_g) * kBlock;
    const int j = (row0 & 127) >> 5, l = (row0 & 31) + col;
    src_w = block + w4_chunk_offset(q, j, l);
    src_s = block + 8 * l + 2 * (j & 2);
    src_h = block + hi_chunk_offset(q, j, l);
  };
  if (ahead_unit < units) locate();
  const uint32_t ring = dev::smem_addr(s_mem) + warp * (kStages * kStage);
  int fill = 0;
  const auto copy = [&]() {
    if (ahead_unit < units) {
      const uint32_t at = ring + fill * kStage;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // rows g and g + 8
          copy16(at + (m * 2 + i) * 512 + lane * 16, src_w + m * next_w + i * 128);
          copy4(at + 2048 + (m * 2 + i) * 128 + lane * 4, src_s + m * next_s + i * 64);
          if (BITS == 6) copy8(at + 2560 + (m * 2 + i) * 256 + lane * 8, src_h + m * next_s + i * 64);
        }
      ahead_g += split;
      if (ahead_g < groups) {
        const size_t step = (size_t)split * kBlock;
        src_w += step, src_s += step, src_h += step;
      } else {
        ahead_unit += teams;
        ahead_g = member;
        if (ahead_unit < units) locate();
      }
    }
    copies_commit();
    fill = fill + 1 == kStages ? 0 : fill + 1;
  };
  for (int i = 0; i < kStages - 1; ++i) copy();
  if (!GATED) dev::pdl_wait_prior_grids();  // h; the weights before it

  int take = 0, buffer = 0;
  for (int unit = team; unit < units; unit += teams) {
    const int item = unit / slices, row0 = (unit - item * slices) * (GATED ? 16 : 32);
    const int rows = SMALL ? s.rows[item] : p.item[item].rows;
    const int first = SMALL ? 0 : p.item[item].first;
    const int shift = (row0 & 32) ? 16 : 0;  // of the scale in its pair (j odd)
    // the row of x (or h) that this lane's column of B is
    const uint16_t* b_row = nullptr;
    if (col < rows) {
      const int place = SMALL ? s.place[item][col] : p.order[first + col];
      b_row = (GATED ? p.x + (size_t)(place / p.k) * K : p.h + (size_t)place * K) + q * 32;
    }
    uint4 bv[4];
    const auto load_b = [&](int g) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bv[i] = b_row ? *reinterpret_cast<const uint4*>(b_row + (size_t)g * kGroup + i * 8) : make_uint4(0u, 0u, 0u, 0u);
    };
    load_b(member);
    float acc[2][4] = {};
    for (int g = member; g < groups; g += split) {
      copies_wait<kStages - 2>();
      const uint8_t* const st = s_mem + (size_t)warp * (kStages * kStage) + take * kStage;
      uint4 w[2][2];
      uint2 hi[2][2];
      uint32_t scale[2][2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[m][i] = *reinterpret_cast<const uint4*>(st + (m * 2 + i) * 512 + lane * 16);
          scale[m][i] = *reinterpret_cast<const uint32_t*>(st + 2048 + (m * 2 + i) * 128 + lane * 4);
          if (BITS == 6) hi[m][i] = *reinterpret_cast<const uint2*>(st + 2560 + (m * 2 + i) * 256 + lane * 8);
        }
      take = take + 1 == kStages ? 0 : take + 1;
      copy();  // into the stage that the step before this one read
      uint32_t b[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[i][0] = __byte_perm(bv[i].x, bv[i].y, 0x5410);  // k 0, 2
        b[i][1] = __byte_perm(bv[i].x, bv[i].y, 0x7632);  // 1, 3
        b[i][2] = __byte_perm(bv[i].z, bv[i].w, 0x5410);  // 4, 6
        b[i][3] = __byte_perm(bv[i].z, bv[i].w, 0x7632);  // 5, 7
      }
      if (g + split < groups) load_b(g + split);
      float d[2][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v = j == 0 ? w[m][i].x : j == 1 ? w[m][i].y : j == 2 ? w[m][i].z : w[m][i].w;
            unpack8<BITS>(v, BITS == 6 ? (j < 2 ? hi[m][i].x : hi[m][i].y) : 0u, j, a[i]);
          }
          mma(d[m], a[0][0], a[1][0], a[0][1], a[1][1], b[j][0], b[j][1]);
          mma(d[m], a[0][2], a[1][2], a[0][3], a[1][3], b[j][2], b[j][3]);
        }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float s0 = dev::half_bits_to_float(scale[m][0] >> shift & 0xFFFFu), s1 = dev::half_bits_to_float(scale[m][1] >> shift & 0xFFFFu);
        acc[m][0] = fmaf(s0, d[m][0], acc[m][0]);
        acc[m][1] = fmaf(s0, d[m][1], acc[m][1]);
        acc[m][2] = fmaf(s1, d[m][2], acc[m][2]);
        acc[m][3] = fmaf(s1, d[m][3], acc[m][3]);
      }
    }
    if (split > 1) {
      // the others' sums to the team's first warp; two buffers, so that one barrier per unit is enough
      float4* const part = s_part + (size_t)buffer * (kWarps * 64) + lane;
      buffer ^= 1;
      if (member) {
        part[warp * 64] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        part[warp * 64 + 32] = make_float4(acc[1][0], acc[1][1], acc[1][2], acc[1][3]);
      }
      dev::named_barrier_sync(1 + warp / split, split * 32);
      if (member) continue;
      for (int w = warp + 1; w < warp + split; ++w) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float4 v = part[w * 64 + m * 32];
          acc[m][0] += v.x, acc[m][1] += v.y, acc[m][2] += v.z, acc[m][3] += v.w;
        }
      }
    }
    // columns 2 q and 2 q + 1, rows col and col + 8 of each tile
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (q * 2 + c >= rows) continue;
      const int place = SMALL ? s.place[item][q * 2 + c] : p.order[first + q * 2 + c];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + col + 8 * i;
        if constexpr (GATED) {
          const float v = acc[0][2 * i + c];
          p.h[(size_t)place * p.inner + r] = (uint16_t)pro::f32_to_bf16_bits(v / (1.0f + expf(-v)) * acc[1][2 * i + c]);
        } else {
          p.parts[(size_t)place * p.hidden + r] = acc[0][2 * i + c];
          p.parts[(size_t)place * p.hidden + r + 16] = acc[1][2 * i + c];
        }
      }
    }
  }
}

// y_t = sum over its places, in their order.  The headers of the row's matrices are looked at here, before the wait for
// the products: a row with one that does not match keeps its y.
__global__ void __launch_bounds__(256) sum_kernel(const Experts p) {
  const int row = blockIdx.x, tid = threadIdx.x, c = (blockIdx.y * 256 + tid) * 4;
  const size_t first = (size_t)row * p.k;
  dev::pdl_launch_dependents();
  int flags = 0;
  if (tid < p.k) {
    const int e = p.ids[first + tid];
    if ((unsigned)e < (unsigned)p.experts) {
      if (!matrix_ok(p.gate_up + (size_t)e * p.gate_up_stride, p.bits, 2 * p.inner, p.hidden) ||
          !matrix_ok(p.down + (size_t)e * p.down_stride, p.bits, p.hidden, p.inner))
        flags = WOQ_DEVERR_HEADER;
    } else if (e != -1) {
      flags = WOQ_DEVERR_STATE;
    }
  }
  dev::pdl_wait_prior_grids();
  if (flags) atomicOr(p.status, (uint32_t)flags);
  if (__syncthreads_or(flags & WOQ_DEVERR_HEADER) || c >= p.hidden) return;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j = 0; j < p.k; ++j) {
    const size_t place = first + j;
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

// Warps that share the groups of a unit: the split that has the fewest steps one behind another, a unit's beginning and
// end counted as three.  The order of a row's sums goes by it, so it comes from the call's shape and not from what was chosen:
// the units are those of as many items as n places give where every expert is as likely.
static int choose_split(const Experts& p, int sms, int slices, int groups) {
  const double items = p.experts * (1.0 - pow(1.0 - 1.0 / p.experts, p.entries)) + (double)p.entries / (2 * kExpertRows);
  const int units = (int)((items < p.items ? items : p.items) * slices);
  int best = 1, least = 0x7FFFFFFF;
  for (int s = 1; s <= kWarps && s <= groups; s *= 2) {
    const int teams = sms * (kWarps / s);
    const int steps = (units + teams - 1) / teams * ((groups + s - 1) / s + 3);
    if (steps < least) least = steps, best = s;
  }
  return best;
}

template <int BITS, bool SMALL>
static cudaError_t launch_all(Experts p, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  p.split_up = choose_split(p, sms, p.inner / 16, p.hidden / kGroup);
  p.split_down = choose_split(p, sms, p.hidden / 32, p.inner / kGroup);
  if (const char* v = getenv("XT"); v && atoi(v)) p.split_up = atoi(v) % 100, p.split_down = atoi(v) / 100;
  cudaError_t e = cudaSuccess;
  if (!SMALL) e = kv8::launch(plan_kernel, dim3(1), kPlanThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  constexpr int kBytes = kSharedBytes<BITS>;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  e = cudaFuncSetAttribute(product_kernel<BITS, true, SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(product_kernel<BITS, false, SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  e = kv8::launch(product_kernel<BITS, true, SMALL>, dim3((unsigned)sms), kWarps * 32, kBytes, s, p);
  if (e != cudaSuccess) return e;
  e = kv8::launch(product_kernel<BITS, false, SMALL>, dim3((unsigned)sms), kWarps * 32, kBytes, s, p);
  if (e != cudaSuccess) return e;
  return kv8::launch(sum_kernel, dim3((unsigned)p.rows, (unsigned)((p.hidden + 1023) / 1024)), 256, 0, s, p);
}

template <int BITS>
static cudaError_t launch_bits(const Experts& p, cudaStream_t s) {
  return p.entries <= kSmallEntries ? launch_all<BITS, true>(p, s) : launch_all<BITS, false>(p, s);
}

}  // namespace experts

cudaError_t launch_experts(const Experts& p, cudaStream_t s) {
  return p.bits == 4 ? experts::launch_bits<4>(p, s) : experts::launch_bits<6>(p, s);
}

}  // namespace woq
