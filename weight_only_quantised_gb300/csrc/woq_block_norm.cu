// Norms before and after a block, with its gate and residual scale, in one pass (include/woq_block.h).
//
//   n = u rsqrt(mean(u^2) + eps) (post + offset),  r' = alpha r + beta gate n,
//   h = r' rsqrt(mean(r'^2) + eps) (pre + offset)
//
// A row is read once: one CTA holds its u and r in registers through both reductions.
#include <cuda_bf16.h>

#include "woq_block_internal.h"
#include "woq_device.cuh"
#include "woq_kv8_device.cuh"
#include "woq_prologue.cuh"

namespace woq {
namespace block {

template <bool F32>
__device__ __forceinline__ void load8(const void* base, size_t at, float* v) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t at, const float* v) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pro::f32_to_bf16_bits(v[2 * i]) | pro::f32_to_bf16_bits(v[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Sum over the CTA, the same in every thread (fixed order).
__device__ __forceinline__ float block_sum(float x, float* parts) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = x;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  x = lane < (int)(blockDim.x >> 5) ? parts[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

template <bool UF32, bool RF32, int VECS>
__global__ void __launch_bounds__(1024) norm_kernel(const BlockNorm p) {
  __shared__ float s_parts[2][32];
  const int row = blockIdx.x;
  const size_t at = (size_t)row * p.dim;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  float u[VECS][8], r[VECS][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c < p.dim) {
      load8<UF32>(p.u, at + c, u[i]);
      load8<RF32>(p.r, at + c, r[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = r[i][j] = 0.0f;
    }
  }
  float f = 1.0f;
  if (p.post) {
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
    f = 1.0f / sqrtf(block_sum(ss, s_parts[0]) / (float)p.dim + p.eps);
  }
  const size_t gate_at = (size_t)(row / p.rows_per_gate) * p.dim;
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c >= p.dim) continue;
    float w[8];
    if (p.post) {
      load8<false>(p.post, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = u[i][j] * f * (w[j] + p.offset);
    }
    if (p.gate) {
      load8<false>(p.gate, gate_at + c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] *= w[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[i][j] = fmaf(p.alpha, r[i][j], p.beta * u[i][j]);
      ss = fmaf(r[i][j], r[i][j], ss);
    }
    store8<RF32>(p.r_out, at + c, r[i]);
  }
  if (!p.out) return;
  f = 1.0f / sqrtf(block_sum(ss, s_parts[1]) / (float)p.dim + p.eps);
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c >= p.dim) continue;
    float w[8];
    load8<false>(p.pre, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * f * (w[j] + p.offset);
    store8<false>(p.out, at + c, r[i]);
  }
}

template <int VECS>
static cudaError_t launch_vecs(const BlockNorm& p, cudaStream_t s) {
  const int vectors = p.dim / 8;
  const int threads = ((vectors + VECS - 1) / VECS + 31) / 32 * 32;
  auto kernel = p.u_f32 ? (p.r_f32 ? norm_kernel<true, true, VECS> : norm_kernel<true, false, VECS>)
                        : (p.r_f32 ? norm_kernel<false, true, VECS> : norm_kernel<false, false, VECS>);
  return kv8::launch(kernel, dim3((unsigned)p.rows), threads, 0, s, p);
}

}  // namespace block

cudaError_t launch_block_norm(const BlockNorm& p, cudaStream_t s) {
  const int vectors = p.dim / 8;
  if (vectors <= 1024) return block::launch_vecs<1>(p, s);
  return block::launch_vecs<2>(p, s);
}

}  // namespace woq
