// Norms before and after a block, with its gate and residual scale, in one pass (include/woq_block.h).
//
//   n = u rsqrt(mean(u^2) + eps) (post + offset),  r' = alpha r + beta gate n,
//   h = r' rsqrt(mean(r'^2) + eps) (pre + offset)
//
// A row is read once: one CTA holds its u and r in registers through both sums.  Bound by DRAM and the latency of the
// sums: 8,190 x 5120 bf16 gated 62 to 63 us (0.80 of the copy rate), 2,049 x 4096 fp32 21.6 to 22.4 (0.80), one row 2.3 on the device.
// Above 5,120 elements a row one CTA stays on an SM and nothing covers its sums: 7,000 x 6144 bf16 70 us (0.73), 5,000 x 7168 86 (0.50).
// Rows that stay with a CTA, the next one on its way meanwhile (in registers or through cp.async), were slower: 80 us.
#include <cuda_bf16.h>

#include "woq_block_internal.h"
#include "woq_device.cuh"
#include "woq_internal.h"
#include "woq_kv8_device.cuh"
#include "woq_prologue.cuh"

namespace woq {
namespace block {

typedef dev::f32x2 Pair;

__device__ __forceinline__ Pair pair_of(uint32_t bf16x2) { return dev::f2_pack(bf16x2 << 16, bf16x2 & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16_of(Pair v) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(__uint_as_float(dev::f2_hi(v))), "f"(__uint_as_float(dev::f2_lo(v))));
  return d;
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t at, const Pair* v) {
  if constexpr (F32) {
    ulonglong2* p = reinterpret_cast<ulonglong2*>(static_cast<float*>(base) + at);
    p[0] = make_ulonglong2(v[0], v[1]);
    p[1] = make_ulonglong2(v[2], v[3]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(bf16_of(v[0]), bf16_of(v[1]), bf16_of(v[2]), bf16_of(v[3]));
  }
}

__device__ __forceinline__ float sum_of(Pair v) { return __uint_as_float(dev::f2_lo(v)) + __uint_as_float(dev::f2_hi(v)); }

// Sum over the CTA, the same in every thread (fixed order).
__device__ __forceinline__ float block_sum(float x, float* parts) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = x;
  __syncthreads();
  x = parts[threadIdx.x & 31];  // behind the last warp's there are zeros
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Eight elements as they lie in memory (bf16 takes half the registers so, and a third CTA fits an SM).
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at * (F32 ? 4 : 2));
    v[0] = p[0];
    if (F32) v[F32] = p[1];
  }
  __device__ __forceinline__ Pair pair(int j) const {
    const uint4 w = v[F32 ? j >> 1 : 0];
    if constexpr (F32) return j & 1 ? dev::f2_pack(w.z, w.w) : dev::f2_pack(w.x, w.y);
    else return pair_of(j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w);
  }
};

// A row a CTA, VECS vectors of 8 a thread; everything that a row takes is asked for at once.  post and pre come after the wait for
// the prior grid too: they may be what a linear has just written (a scale that depends on the condition).
template <bool UF32, bool RF32, int VECS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 640 ? 1 : THREADS > 512 ? (UF32 || RF32 ? 2 : 3) : (UF32 || RF32 ? 3 : 4)) norm_kernel(const BlockNorm p) {
  __shared__ float s_parts[2][32];
  const int warps = blockDim.x >> 5;
  for (int i = threadIdx.x; i < 64; i += blockDim.x)
    if ((i & 31) >= warps) s_parts[i >> 5][i & 31] = 0.0f;  // what block_sum adds behind the last warp's
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  const size_t at = (size_t)blockIdx.x * p.dim;
  uint4 post[VECS] = {}, gate[VECS] = {}, pre[VECS] = {};
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (p.post && c < p.dim) post[i] = *reinterpret_cast<const uint4*>(p.post + c);
    if (p.out && c < p.dim) pre[i] = *reinterpret_cast<const uint4*>(p.pre + c);
  }
  Raw<UF32> u[VECS] = {};
  Raw<RF32> r0[VECS] = {};
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c < p.dim) {
      u[i].load(p.u, at + c);
      r0[i].load(p.r, at + c);
      if (p.gate) gate[i] = *reinterpret_cast<const uint4*>(p.gate + (size_t)((int)blockIdx.x / p.rows_per_gate) * p.dim + c);
    }
  }
  float f = p.beta;
  Pair ss = 0;
  if (p.post) {
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = dev::f2_fma(u[i].pair(j), u[i].pair(j), ss);
    f *= rsqrtf(fmaf(block_sum(sum_of(ss), s_parts[0]), p.inv_dim, p.eps));
  }
  const Pair fs = dev::f2_splat(f), alpha = dev::f2_splat(p.alpha), offset = dev::f2_splat(p.offset);
  Pair r[VECS][4];
  ss = 0;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c >= p.dim) continue;
    const uint32_t pw[4] = {post[i].x, post[i].y, post[i].z, post[i].w}, gw[4] = {gate[i].x, gate[i].y, gate[i].z, gate[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Pair v = dev::f2_mul(u[i].pair(j), fs);
      if (p.post) v = dev::f2_mul(v, dev::f2_add(pair_of(pw[j]), offset));
      if (p.gate) v = dev::f2_mul(v, pair_of(gw[j]));
      r[i][j] = dev::f2_fma(alpha, r0[i].pair(j), v);
      ss = dev::f2_fma(r[i][j], r[i][j], ss);
    }
    store8<RF32>(p.r_out, at + c, r[i]);
  }
  if (!p.out) return;
  const Pair g = dev::f2_splat(rsqrtf(fmaf(block_sum(sum_of(ss), s_parts[1]), p.inv_dim, p.eps)));
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c >= p.dim) continue;
    const uint32_t qw[4] = {pre[i].x, pre[i].y, pre[i].z, pre[i].w};
    Pair w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = dev::f2_mul(dev::f2_mul(r[i][j], g), dev::f2_add(pair_of(qw[j]), offset));
    store8<false>(p.out, at + c, w);
  }
}

template <bool UF32, bool RF32>
static cudaError_t launch_types(const BlockNorm& p, cudaStream_t s) {
  const int vectors = p.dim / 8, vecs = vectors <= 1024 ? 1 : 2;
  const int threads = ((vectors + vecs - 1) / vecs + 31) / 32 * 32;
  // a vector a thread up to 8,192 elements (with two or four, 8,190 x 5120 takes 77 or 89 us; with one 62).  Bounds of 512 and 640 threads
  // leave room for three and four CTAs: 9,000 x 4096 bf16 50.5 us, by the kernel of 1,024 56.6; 8,190 x 5120 60 and 73.5.
  auto kernel = vecs == 2 ? norm_kernel<UF32, RF32, 2, 1024> : threads <= 512 ? norm_kernel<UF32, RF32, 1, 512> : threads <= 640 ? norm_kernel<UF32, RF32, 1, 640> : norm_kernel<UF32, RF32, 1, 1024>;
  return kv8::launch(kernel, dim3((unsigned)p.rows), threads, 0, s, p);
}

}  // namespace block

cudaError_t launch_block_norm(const BlockNorm& p, cudaStream_t s) {
  if (p.u_f32) return p.r_f32 ? block::launch_types<true, true>(p, s) : block::launch_types<true, false>(p, s);
  return p.r_f32 ? block::launch_types<false, true>(p, s) : block::launch_types<false, false>(p, s);
}

}  // namespace woq
