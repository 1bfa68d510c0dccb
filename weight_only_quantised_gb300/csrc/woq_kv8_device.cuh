// Device helpers shared by the cache's kernels: the header check, block scans, codes and scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "woq_device.cuh"
#include "woq_kv8_layout.h"
#include "woq_quotient.h"

namespace woq {
namespace kv8 {

// Every kernel of the cache is launched with programmatic dependent launch and passes through this: it may be
// scheduled while the kernel before it ends, writes nothing and keeps nothing that it read until that one has completed (the
// attention plans from lengths that it read before, and checks them afterwards), and only then
// lets its own successor be scheduled (in that order: a linear reads its weights before its own wait, so
// whoever wrote them must be complete by the time this kernel lets it start).
__device__ __forceinline__ void begin_after_prior() {
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
}

template <class... P, class... A>
inline cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, P(args)...);
}

__device__ __forceinline__ void flag(const Kv8View& v, uint32_t bits) { atomicOr(v.status(), bits); }

// Whether the buffer is a cache of this config.  A cache of another config gets the status bit;
// a buffer that is no cache is not written.
__device__ __forceinline__ bool header_ok(const Kv8View& v) {
  const uint4 h = *reinterpret_cast<const uint4*>(v.base);
  if (h.y != kKv8Magic) return false;
  if (h.z != v.hash) {
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_HEADER);
    return false;
  }
  return true;
}

__device__ __forceinline__ bool bf16_pair_not_finite(uint32_t p) {
  return (p & 0x7F80u) == 0x7F80u || (p & 0x7F800000u) == 0x7F800000u;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Scale of a block whose largest magnitude (a bf16 value) is amax, and what multiplies a value
// before it is rounded to a code (int8: the reciprocal for the corrected quotient).
template <int FMT>
__device__ __forceinline__ float block_scale(float amax, float* mul) {
  if (!(amax > 0.0f)) {
    *mul = 0.0f;
    return 0.0f;
  }
  if constexpr (FMT == WOQ_KV8_INT8) {
    const float s = __fdiv_rn(amax, 127.0f);
    *mul = __frcp_rn(s);
    return s;
  } else {
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 127 - (((b >> 16) & 0x7Fu) <= 0x60u ? 8 : 7);  // 448 = 1.75 * 2^8
    if (e < -126) e = -126;
    *mul = __uint_as_float((uint32_t)(127 - e) << 23);
    return __uint_as_float((uint32_t)(127 + e) << 23);
  }
}

// Codes of four bf16 values (two packed pairs).  int8: rne of the IEEE quotient, by the corrected
// quotient where it is exact (amax >= 2^-116: woq_quotient.h) and by the division below.  e4m3:
// x / s is exact (s a power of two), so the conversion's rounding is the only one.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(uint32_t p01, uint32_t p23, float s, float mul, bool exact_div) {
  const float x0 = __uint_as_float(p01 << 16), x1 = __uint_as_float(p01 & 0xFFFF0000u);
  const float x2 = __uint_as_float(p23 << 16), x3 = __uint_as_float(p23 & 0xFFFF0000u);
  if constexpr (FMT == WOQ_KV8_INT8) {
    if (s == 0.0f) return 0u;
    if (exact_div) {
      return dev::quant_byte_exact(x0, s) | dev::quant_byte_exact(x1, s) << 8 | dev::quant_byte_exact(x2, s) << 16 |
             dev::quant_byte_exact(x3, s) << 24;
    }
    const uint32_t q0 = __float_as_uint(corrected_quotient(x0, s, mul) + dev::kRoundMagic);
    const uint32_t q1 = __float_as_uint(corrected_quotient(x1, s, mul) + dev::kRoundMagic);
    const uint32_t q2 = __float_as_uint(corrected_quotient(x2, s, mul) + dev::kRoundMagic);
    const uint32_t q3 = __float_as_uint(corrected_quotient(x3, s, mul) + dev::kRoundMagic);
    return __byte_perm(__byte_perm(q0, q1, 0x0040), __byte_perm(q2, q3, 0x0040), 0x5410);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1 * mul), "f"(x0 * mul));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3 * mul), "f"(x2 * mul));
    return (uint32_t)lo | (uint32_t)hi << 16;
  }
}

// Two codes (the low 16 bits of c) as a pair of f16: exact.
template <int FMT>
__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t c) {
  if constexpr (FMT == WOQ_KV8_INT8) {
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1024 + 128
    uint32_t u = __byte_perm(c ^ 0x8080u, 0x64646464u, 0x4140);
    const __half2 h = __hsub2(*reinterpret_cast<__half2*>(&u), off);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)c));
    return d;
  }
}

// Four codes as two pairs of f16: exact.  int8: byte + 128 in the low bits of 1024, then less 1152.
template <int FMT>
__device__ __forceinline__ void f16x4_of_codes(uint32_t c, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == WOQ_KV8_INT8) {
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1024 + 128
    c ^= 0x80808080u;
    uint32_t u = __byte_perm(c, 0x64646464u, 0x4140), w = __byte_perm(c, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<__half2*>(&u), off), b = __hsub2(*reinterpret_cast<__half2*>(&w), off);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
  }
}

// Exclusive sum over the block (blockDim.x a multiple of 32, at most 1024); *total over all threads.
__device__ __forceinline__ int block_exclusive_sum(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(~0u, y, d);
    if (lane >= d) y += z;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < warps ? warp_sums[lane] : 0;
    int s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(~0u, s, d);
      if (lane >= d) s += z;
    }
    warp_sums[lane] = s - w;
    if (lane == 31) warp_sums[32] = s;
  }
  __syncthreads();
  *total = warp_sums[32];
  return warp_sums[warp] + y - x;
}

}  // namespace kv8
}  // namespace woq
