// Routing of rows to experts (include/woq_block.h): scores, groups, the k best and their weights, a warp per row.
//
// Which experts are chosen is decided as in exact arithmetic.  Without a bias the choice goes by the logits, which
// both scores grow with.  With one, scores c are formed in fp32; e^x is good to 2 ulp (CUDA's expf), so that
//   sigmoid: s is within 2^-21 s, softmax: within 2^-17 s (the sum's rounding and the exponent's included), c within that and 2^-24 |c|.
// Where two neighbours of the order (the k chosen and the next) lie nearer than both errors and do not have the very
// same logit and bias, the row is done again in fp64: about one row in a thousand.
#include <cuda_bf16.h>

#include "woq_block_internal.h"
#include "woq_device.cuh"
#include "woq_kv8_device.cuh"

namespace woq {
namespace route {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xFFFFFFFFu;

// Unsigned order of a float (no NaN; -0 and 0 differ: add 0 first).
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v);
  return b ^ ((unsigned long long)((long long)b >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (unsigned long long)hi << 32 | lo;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float fmin(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ float fmax(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double fmin(double a, double b) { return ::fmin(a, b); }
__device__ __forceinline__ double fmax(double a, double b) { return ::fmax(a, b); }


constexpr float kInf = __builtin_huge_valf();

// Type that orders a score: 0 is an expert that cannot be chosen (any more).
template <class F>
struct Key {
  typedef uint32_t type;
};
template <>
struct Key<double> {
  typedef unsigned long long type;
};

__device__ __forceinline__ float logit(const Route& p, size_t at) {
  const float v = p.f32 ? __ldg(static_cast<const float*>(p.logits) + at)
                        : dev::bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(p.logits) + at));
  return v + 0.0f;  // -0 and 0 are one value
}

template <int PER>
__device__ __forceinline__ void load_row(const Route& p, int row, int lane, float (&l)[PER]) {
  const size_t at = (size_t)row * p.stride;
#pragma unroll
  for (int j = 0; j < PER; ++j) l[j] = lane + 32 * j < p.experts ? logit(p, at + lane + 32 * j) : -kInf;
}

// Largest logit and the softmax's denominator (0 and 1 for the sigmoid, and for a row without experts).
template <class F, int PER>
__device__ __forceinline__ void softmax_terms(const Route& p, const float (&l)[PER], float* m, F* sum) {
  *m = 0.0f;
  *sum = 1;
  if (!p.softmax) return;
  float x = -kInf;
#pragma unroll
  for (int j = 0; j < PER; ++j) x = fmaxf(x, l[j]);  // NaN aside
  x = warp_max(x);
  if (x == -kInf) return;
  *m = x;
  F t = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) t += l[j] > -kInf && l[j] < kInf ? exp_of((F)l[j] - (F)x) : (F)0;  // x +inf: not used
  *sum = warp_sum(t);
}

// c of one expert that may be chosen (NaN and, under softmax, +inf come first).
template <class F>
__device__ __forceinline__ F value(const Route& p, float l, int e, float m, F sum) {
  if (l != l || (p.softmax && l == kInf)) return (F)kInf;
  F s;
  if (p.softmax) s = m == kInf ? (F)0 : exp_of((F)l - (F)m) / sum;
  else s = (F)1 / ((F)1 + exp_of(-(F)l));
  const F c = s + (p.bias ? (F)__ldg(p.bias + e) : (F)0);
  return c != c ? (F)kInf : c;
}

// The choice of one row.  l: the lane's logits (expert lane + 32 j); chosen: lane i < k gets the i-th expert, else -1.
// Returns whether F tells every score that matters from its neighbour.
template <class F, int PER>
__device__ __forceinline__ bool choose(const Route& p, const float (&l)[PER], float m, F sum, F* shared, int lane, int* chosen) {
  typedef typename Key<F>::type K;
  const bool by_logit = p.bias == nullptr;
  const float rel = p.softmax ? 0x1p-16f : 0x1p-19f;  // twice the relative error of s in fp32, and more
  bool sure = true;
  unsigned kept = kAll;
  if (p.groups > 1) {
    const bool max_logit = by_logit && p.group_best == 1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 32 * j;
      if (e >= p.experts) continue;
      shared[e] = l[j] == -kInf ? (F)-kInf : max_logit ? (l[j] != l[j] ? (F)kInf : (F)l[j]) : value<F>(p, l[j], e, m, sum);
    }
    __syncwarp();
    F best = -kInf, next = -kInf;  // of group `lane`
    if (lane < p.groups) {
      const F* c = shared + lane * p.group_size;
      int i = lane % p.group_size;  // lanes start at different members: fewer bank conflicts
      for (int n = 0; n < p.group_size; ++n) {
        next = fmax(next, fmin(best, c[i]));
        best = fmax(best, c[i]);
        if (++i == p.group_size) i = 0;
      }
    }
    __syncwarp();
    const F score = p.group_best == 1 ? best : next == (F)-kInf ? (F)-kInf : best + next;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const F other = __shfl_sync(kAll, score, g);
      rank += other > score || (other == score && g < lane);
    }
    const bool group = lane < p.groups, in = group && rank < p.top_groups;
    kept = __ballot_sync(kAll, in);
    if (sizeof(F) == 4 && !max_logit && p.top_groups < p.groups) {
      const float big = warp_max(group && score > -kInf && score < kInf ? fmaxf(fabsf((float)best), fabsf((float)next)) : 0.0f);
      const float low = -warp_max(in ? -(float)score : -kInf);  // of the kept
      const float high = warp_max(group && !in ? (float)score : -kInf);
      // s <= 1, and two of them at most make a group's score
      if (low < kInf && high > -kInf && low - high <= 4.0f * rel + 0x1p-20f * big) sure = false;
    }
  }
  K key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    key[j] = 0;
    if (l[j] == -kInf || e >= p.experts || (p.groups > 1 && !(kept >> (e / p.group_size) & 1))) continue;
    key[j] = order(by_logit ? (l[j] != l[j] ? (F)kInf : (F)l[j]) : value<F>(p, l[j], e, m, sum) + (F)0);
  }
  K top = 0;
  int at = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (key[j] > top) top = key[j], at = j;
  *chosen = -1;
  float last = 0.0f, last_l = 0.0f, last_b = 0.0f;
  const bool check = sizeof(F) == 4 && !by_logit;
  const int rounds = check ? p.k + 1 : p.k;  // the next one too, to compare with
  for (int n = 0; n < rounds; ++n) {
    const K best = warp_max(top);
    if (best == 0) break;
    const int e = (int)__reduce_min_sync(kAll, top == best ? (unsigned)(lane + 32 * at) : kAll);
    if (lane == n && n < p.k) *chosen = e;
    if (check) {
      float mine = l[0];
#pragma unroll
      for (int j = 1; j < PER; ++j)
        if (j == e >> 5) mine = l[j];
      const float el = __shfl_sync(kAll, mine, e & 31), eb = __ldg(p.bias + e);
      const uint32_t bits = (uint32_t)best;
      const float c = __uint_as_float(bits & 0x80000000u ? bits ^ 0x80000000u : ~bits);
      if (n > 0 && last < kInf && !(el == last_l && eb == last_b)) {
        const float near = rel * (fabsf(last - last_b) + fabsf(c - eb)) + 0x1p-21f * (fabsf(last) + fabsf(c));
        if (last - c <= near) sure = false;
      }
      last = c, last_l = el, last_b = eb;
    }
    if ((e & 31) == lane) {
      top = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (j == e >> 5) key[j] = 0;
        if (key[j] > top) top = key[j], at = j;
      }
    }
  }
  return sure;
}

template <int PER>
__device__ __noinline__ int choose_in_64_bits(const Route& p, int row, double* shared, int lane) {
  float l[PER], m;
  load_row<PER>(p, row, lane, l);
  double sum;
  int chosen;
  softmax_terms<double, PER>(p, l, &m, &sum);
  choose<double, PER>(p, l, m, sum, shared, lane, &chosen);
  return chosen;
}

template <int PER>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const Route p) {
  extern __shared__ double s_scores[];  // with groups: [kWarps][experts]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kWarps + warp;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  if (row >= p.rows) return;
  const size_t out = (size_t)row * p.k + lane;
  if (p.live && row >= __ldg(p.live)) {
    if (lane < p.k) {
      p.ids[out] = -1;
      p.weights[out] = 0.0f;
    }
    return;
  }
  double* shared = s_scores + warp * p.experts;
  float l[PER], m, sum;
  load_row<PER>(p, row, lane, l);
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) bad |= l[j] != l[j] || (p.softmax && l[j] == kInf);
  bad = __any_sync(kAll, bad);
  softmax_terms<float, PER>(p, l, &m, &sum);
  int chosen;
  if (!choose<float, PER>(p, l, m, sum, reinterpret_cast<float*>(shared), lane, &chosen))
    chosen = choose_in_64_bits<PER>(p, row, shared, lane);
  // weights, from the chosen logits
  const bool has = chosen >= 0;
  const float x = has ? logit(p, (size_t)row * p.stride + chosen) : -kInf;
  float w = 0.0f;
  if (p.renormalise) {
    // s up to a factor that all share, such that the largest is near 1 (softmax) or its s (a sigmoid that has not underflowed)
    const float most = warp_max(x);
    if (has) {
      if (p.softmax) w = expf(x - most);
      else w = expf(fminf(x, 0.0f) - fminf(most, 0.0f)) / (1.0f + expf(-fabsf(x)));
    }
    const float total = warp_sum(w);
    w = has ? w / total : 0.0f;
  } else if (has) {
    w = p.softmax ? expf(x - m) / sum : 1.0f / (1.0f + expf(-x));
  }
  if (lane < p.k) {
    p.ids[out] = chosen;
    p.weights[out] = !has ? 0.0f : bad ? __int_as_float(0x7FC00000) : w * p.scale;
  }
}

template <int PER>
static cudaError_t launch_per(const Route& p, cudaStream_t s) {
  const size_t smem = p.groups > 1 ? (size_t)kWarps * p.experts * 8 : 0;  // 32 KB at most
  return kv8::launch(route_kernel<PER>, dim3((unsigned)((p.rows + kWarps - 1) / kWarps)), kWarps * 32, smem, s, p);
}

}  // namespace route

cudaError_t launch_route(const Route& p, cudaStream_t s) {
  const int per = (p.experts + 31) / 32;
  if (per <= 1) return route::launch_per<1>(p, s);
  if (per <= 2) return route::launch_per<2>(p, s);
  if (per <= 4) return route::launch_per<4>(p, s);
  if (per <= 8) return route::launch_per<8>(p, s);
  if (per <= 16) return route::launch_per<16>(p, s);
  return route::launch_per<32>(p, s);
}

}  // namespace woq
