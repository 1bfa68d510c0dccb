// Routing of rows to experts (include/woq_block.h): scores, groups, the k best and their weights, a warp per row.
//
// Which experts are chosen is decided as by scores in fp64.  Without a bias the choice goes by the logits, which both scores grow
// with.  With one, scores c are formed in fp32; e^x and 1 / x are good to 2 ulp (CUDA's expf and __fdividef), so that
//   sigmoid: s is within 2^-20.8 s; softmax: within 2^-16.7 s (the sum's rounding and the exponent's included); c within that and 2^-24 |c|.
// Sure is an order whose neighbours lie further apart than both errors (or have the very same logit and bias), and a choice that leaves
// nothing out that its own error (a large s under a negative bias has a large one) could lift to the k-th. Else those that may be among
// the k are put in order in fp64 (sigmoid: some ten scores, a lane each), or the whole row is done again in fp64 (softmax, more than
// 64 such scores, groups too near to tell): one or two rows in a thousand of normally distributed logits and biases.
// The k best: as many lanes' largest scores as are wanted bound them from below; what is not below (some ten) goes to a lane each
// and finds its place by comparing all with all.  Bound by latency, as a row is one chain and few warps stay on an SM: 8,191 rows x 256
// experts in groups 25.6 us (some 1,790 instructions a row, issue 46 %, 30 % of the warps, 80 registers; with one argument of the maximum
// after another 35, the first right version 57), 16,000 x 60 12.3 us (540 a row, issue 55 %, 46 % of the warps, 48 registers).
#include <cuda_bf16.h>

#include "woq_block_internal.h"
#include "woq_device.cuh"
#include "woq_internal.h"
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
__device__ __forceinline__ float warp_max(float v) {  // NaN aside
  float d;
  asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(d) : "f"(v));
  return d;
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

// Plain loads here and below: the kernel may be there before what it reads has been written (it waits for the prior grid), and the
// read-only path is for what nobody writes while a kernel is there.
__device__ __forceinline__ float logit(const Route& p, size_t at) {
  const float v = p.f32 ? static_cast<const float*>(p.logits)[at] : dev::bf16_bits_to_float(static_cast<const uint16_t*>(p.logits)[at]);
  return v + 0.0f;  // -0 and 0 are one value
}

template <int PER>
__device__ __forceinline__ void load_row(const Route& p, int row, int lane, float (&l)[PER], float (&b)[PER]) {
  const size_t at = (size_t)row * p.stride;
#pragma unroll
  for (int j = 0; j < PER; ++j) l[j] = lane + 32 * j < p.experts ? logit(p, at + lane + 32 * j) : -kInf;
#pragma unroll
  for (int j = 0; j < PER; ++j) b[j] = p.bias && lane + 32 * j < p.experts ? p.bias[lane + 32 * j] : 0.0f;
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

__device__ __forceinline__ float inverse(float x) { return __fdividef(1.0f, x); }  // within 2 ulp; 0 from 2^126 on
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

// c of one expert that may be chosen (NaN and, under softmax, +inf come first).
template <class F>
__device__ __forceinline__ F value(const Route& p, float l, float b, float m, F sum) {
  if (l != l || (p.softmax && l == kInf)) return (F)kInf;
  F s;
  if (p.softmax) s = m == kInf ? (F)0 : exp_of((F)l - (F)m) * inverse(sum);
  else s = inverse((F)1 + exp_of(-(F)l));
  const F c = s + (F)b;
  return c != c ? (F)kInf : c;
}

// Scores c of the lane's experts (bit j of `can`: it may be chosen), without a bias the logits themselves.
template <class F, int PER>
__device__ __forceinline__ void scores(const Route& p, const float (&l)[PER], const float (&b)[PER], float m, F sum, bool by_logit, F (&c)[PER],
                                       uint32_t& can) {
  can = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (l[j] != -kInf) can |= 1u << j;  // experts that there are not have -inf too
  if (by_logit) {
#pragma unroll
    for (int j = 0; j < PER; ++j) c[j] = l[j] != l[j] ? (F)kInf : (F)l[j];
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) c[j] = l[j] == -kInf ? (F)-kInf : value<F>(p, l[j], b[j], m, sum);
  }
}

// Which groups are kept (bit g).  c: as of scores (without a bias and with group_best 2: of the scores proper).  Returns whether F
// tells the last one kept from the first one dropped.
template <class F, int PER>
__device__ __forceinline__ bool keep_groups(const Route& p, const F (&c)[PER], F* shared, int lane, unsigned* kept) {
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (lane + 32 * j < p.experts) shared[lane + 32 * j] = c[j];
  __syncwarp();
  // `share` lanes look at each group's members in turn, each beginning at another one (fewer bank conflicts)
  const int share = p.group_share, group = lane / share, part = lane & (share - 1);
  F best = -kInf, next = -kInf;
  if (group < p.groups) {
    const F* const of = shared + group * p.group_size;
    int i = part + share * (group % max(1, p.group_size / share));
    for (int n = part; n < p.group_size; n += share) {
      if (i >= p.group_size) i = part;
      next = fmax(next, fmin(best, of[i]));
      best = fmax(best, of[i]);
      i += share;
    }
  }
  __syncwarp();
  for (int o = 1; o < share; o <<= 1) {
    const F other = __shfl_xor_sync(kAll, best, o), other_next = __shfl_xor_sync(kAll, next, o);
    next = fmax(fmax(next, other_next), fmin(best, other));
    best = fmax(best, other);
  }
  // lane g takes group g
  best = __shfl_sync(kAll, best, min(lane * share, 31));
  next = __shfl_sync(kAll, next, min(lane * share, 31));
  const F score = p.group_best == 1 ? best : next == (F)-kInf ? (F)-kInf : best + next;
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const F other = __shfl_sync(kAll, score, g);
    rank += other > score || (other == score && g < lane);
  }
  const bool real = lane < p.groups, in = real && rank < p.top_groups;
  *kept = __ballot_sync(kAll, in);
  if (sizeof(F) == 8 || (!p.bias && p.group_best == 1) || p.top_groups == p.groups) return true;
  const float rel = p.softmax ? 0x1p-16f : 0x1p-19f;
  const float big = warp_max(real && score > -kInf && score < kInf ? fmaxf(fabsf((float)best), fabsf((float)next)) : 0.0f);
  const float low = -warp_max(in ? -(float)score : -kInf);  // of the kept
  const float high = warp_max(real && !in ? (float)score : -kInf);
  // s <= 1 (two of softmax's together), so two groups' scores are off by 2^-18.9 (2^-16) and their roundings at most
  return !(low < kInf && high > -kInf && low - high <= 1.25f * rel + 0x1p-20f * big);
}

template <int PER>
__device__ __forceinline__ uint32_t in_kept_groups(const Route& p, unsigned kept, int lane) {
  uint32_t in = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    in |= (kept >> ((lane + 32 * j) * p.group_magic >> 20 & 31) & 1u) << j;  // (places behind the last expert: any)
  return in;
}

// The k best of those that `can`.  Lane i gets the i-th one's expert (else -1) and order.
template <class F, int PER>
__device__ __forceinline__ int best_of(const Route& p, const F (&c)[PER], uint32_t can, int lane, typename Key<F>::type* mine,
                                       uint32_t* shared) {
  typedef typename Key<F>::type K;
  K key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = can >> j & 1u ? order(c[j] + (F)0) : (K)0;
  K top = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) top = key[j] > top ? key[j] : top;
  int chosen = -1;
  *mine = 0;
  const int rounds = p.k;
  if constexpr (sizeof(F) == 4 && PER > 2) {
    // As many lanes' largest as are wanted: nothing below the least of these is among the best.  What is not below (some ten
    // experts) goes to a lane each, and is placed by comparing all with all.
    K rest = top, least = 0;
    int lanes = 0;
    while (lanes < rounds) {
      const K best = warp_max(rest);
      if (best == 0) break;
      least = best;
      lanes += __popc(__ballot_sync(kAll, rest == best));
      if (rest == best) rest = 0;
    }
    if (lanes < rounds) least = 1;  // all that can be chosen
    unsigned has[PER];
    int total = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      has[j] = __ballot_sync(kAll, key[j] >= least);
      total += __popc(has[j]);
    }
    if (total <= 32) {
      int base = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (key[j] >= least) {
          const int at = base + __popc(has[j] & ((1u << lane) - 1));
          shared[at] = key[j];
          shared[32 + at] = lane + 32 * j;
        }
        base += __popc(has[j]);
      }
      __syncwarp();
      const K k = lane < total ? shared[lane] : 0;
      const uint32_t e = shared[32 + lane];
      int place = 0;
      // among equals the lower number first: the list runs over j, then over lanes
      for (int i = 0; i < total; ++i) {
        const K other = shared[i];
        place += other > k || (other == k && i < lane);
      }
      if (lane < total) {
        shared[64 + place] = k;
        shared[96 + place] = e;
      }
      __syncwarp();
      const bool mine_too = lane < total && lane < rounds;
      if (mine_too) *mine = shared[64 + lane], chosen = (int)shared[96 + lane];
      __syncwarp();
      return chosen;
    }
  }
  for (int n = 0; n < rounds; ++n) {
    const K best = warp_max(top);
    if (best == 0) break;
    int at = 0;
#pragma unroll
    for (int j = PER - 1; j >= 0; --j) at = key[j] == best ? j : at;
    const unsigned owners = __ballot_sync(kAll, top == best);
    // one lane has it, or the lowest number of those that have
    int e;
    if ((owners & (owners - 1)) == 0) e = __shfl_sync(kAll, lane + 32 * at, __ffs(owners) - 1);
    else e = (int)__reduce_min_sync(kAll, top == best ? (unsigned)(lane + 32 * at) : kAll);
    if (lane == n) chosen = e, *mine = best;
    if ((e & 31) == lane) {
      top = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (j == e >> 5) key[j] = 0;
        top = key[j] > top ? key[j] : top;
      }
    }
  }
  return chosen;
}

// How far a score in fp32 may be off; s is c - b, 2^-120 covers one that underflows.
__device__ __forceinline__ float error_of(const Route& p, float c, float b) {
  return fmaf(p.softmax ? 0x1p-16f : 0x1p-20f, fabsf(c - b), fmaf(0x1p-22f, fabsf(c), 0x1p-120f));
}

// All of a row in 64 bits.
template <int PER>
__device__ __noinline__ int choose_in_64_bits(const Route& p, int row, double* shared, int lane) {
  float l[PER], b[PER], m;
  load_row<PER>(p, row, lane, l, b);
  double sum, c[PER];
  softmax_terms<double, PER>(p, l, &m, &sum);
  uint32_t can, in = kAll;
  scores<double, PER>(p, l, b, m, sum, !p.bias && (p.groups == 1 || p.group_best == 1), c, can);
  if (p.groups > 1) {
    unsigned kept;
    keep_groups<double, PER>(p, c, shared, lane, &kept);
    in = in_kept_groups<PER>(p, kept, lane);
    if (!p.bias && p.group_best == 2) scores<double, PER>(p, l, b, m, sum, true, c, can);
  }
  unsigned long long key;
  const int e = best_of<double, PER>(p, c, can & in, lane, &key, nullptr);
  return lane < p.k ? e : -1;
}

// The order of a few experts in 64 bits: those whose fp32 score is not surely below the k-th's (bits of `few`, 64 at most;
// sigmoid only).  Lane i gets the i-th.
template <int PER>
__device__ __noinline__ int choose_few(const Route& p, int row, uint32_t few, double* shared, int lane) {
  float l[PER], b[PER];
  load_row<PER>(p, row, lane, l, b);
  int before = __popc(few), total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, before, o);
    if (lane >= o) before += y;
  }
  total = __shfl_sync(kAll, before, 31);
  before -= __popc(few);
  int* const experts = reinterpret_cast<int*>(shared + 64);
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (few >> j & 1u) experts[before++] = lane + 32 * j;
  __syncwarp();
  for (int i = lane; i < total; i += 32) {
    const float x = logit(p, (size_t)row * p.stride + experts[i]);
    shared[i] = value<double>(p, x, p.bias[experts[i]], 0.0f, 1.0);
  }
  __syncwarp();
  int chosen = -1;
  int* const out = experts + 64;
  for (int i = lane; i < total; i += 32) {
    const double v = shared[i];
    const int e = experts[i];
    int rank = 0;
    for (int j = 0; j < total; ++j) rank += shared[j] > v || (shared[j] == v && experts[j] < e);
    if (rank < 32) out[rank] = e;
  }
  __syncwarp();
  if (lane < p.k && lane < total) chosen = out[lane];
  return chosen;
}

template <int PER>
__device__ __forceinline__ void route_row(const Route& p, int row, int lane, double* shared) {
  const size_t out = (size_t)row * p.k + lane;
  if (p.live && row >= *p.live) {
    if (lane < p.k) {
      p.ids[out] = -1;
      p.weights[out] = 0.0f;
    }
    return;
  }
  float l[PER], b[PER], m, sum, c[PER];
  load_row<PER>(p, row, lane, l, b);
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) bad |= !(l[j] < kInf) && (l[j] != l[j] || p.softmax);
  bad = __any_sync(kAll, bad);
  softmax_terms<float, PER>(p, l, &m, &sum);
  uint32_t can, kept_members = kAll;
  bool sure = true;
  if (p.groups > 1) {
    unsigned kept;
    scores<float, PER>(p, l, b, m, sum, !p.bias && p.group_best == 1, c, can);
    sure = keep_groups<float, PER>(p, c, reinterpret_cast<float*>(shared), lane, &kept);
    kept_members = in_kept_groups<PER>(p, kept, lane);
    if (!p.bias && p.group_best == 2) scores<float, PER>(p, l, b, m, sum, true, c, can);
  } else {
    scores<float, PER>(p, l, b, m, sum, !p.bias, c, can);
  }
  can &= kept_members;
  uint32_t key;
  int chosen = best_of<float, PER>(p, c, can, lane, &key, reinterpret_cast<uint32_t*>(shared));
  const bool has_x = chosen >= 0;
  const float x = has_x ? logit(p, (size_t)row * p.stride + chosen) : -kInf;
  bool again = !sure;
  uint32_t few = 0;
  if (p.bias) {
    const float eb = has_x ? p.bias[chosen] : 0.0f;
    const float v = __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
    const float err = error_of(p, v, eb);
    // their order: each chosen one against the one before it
    const float v0 = __shfl_up_sync(kAll, v, 1), b0 = __shfl_up_sync(kAll, eb, 1), x0 = __shfl_up_sync(kAll, x, 1), err0 = __shfl_up_sync(kAll, err, 1);
    bool near = lane > 0 && has_x && v0 < kInf && !(x == x0 && eb == b0) && v0 - v <= err0 + err;
    // the choice: what is not surely below all of them, apart from the k-th's equals (the lower numbers of these are chosen)
    const float kth = __shfl_sync(kAll, v, p.k - 1), kth_x = __shfl_sync(kAll, x, p.k - 1), kth_b = __shfl_sync(kAll, eb, p.k - 1);
    const bool full = __shfl_sync(kAll, has_x, p.k - 1);  // else all that can be chosen are
    if (full && kth < kInf) {
      const float least = -warp_max(has_x && v < kInf ? err - v : -kInf);
      uint32_t equal = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        few |= (uint32_t)(c[j] + error_of(p, c[j], b[j]) >= least) << j;
        equal |= (uint32_t)(l[j] == kth_x && b[j] == kth_b) << j;
      }
      few &= can;
      const unsigned others = __reduce_add_sync(kAll, (unsigned)__popc(few & ~equal));
      near |= others != (unsigned)__popc(__ballot_sync(kAll, has_x && !(x == kth_x && eb == kth_b)));
    } else {
      few = can;
    }
    if (__any_sync(kAll, near) && !again) {
      again = p.softmax || bad || __reduce_add_sync(kAll, (unsigned)__popc(few)) > 64u;
      if (!again) chosen = choose_few<PER>(p, row, few, shared, lane);
    }
  }
  if (again) chosen = choose_in_64_bits<PER>(p, row, shared, lane);
  if (lane >= p.k) chosen = -1;
  // weights, from the chosen logits
  const bool has = chosen >= 0;
  const float y = has ? logit(p, (size_t)row * p.stride + chosen) : -kInf;
  float w = 0.0f;
  if (p.renormalise) {
    // s up to a factor that all share, such that the largest is near 1 (softmax) or its s (a sigmoid that has not underflowed)
    const float most = warp_max(y);
    if (has) {
      if (p.softmax) w = expf(y - most);
      else w = expf(fminf(y, 0.0f) - fminf(most, 0.0f)) / (1.0f + expf(-fabsf(y)));
    }
    const float total = warp_sum(w);
    w = has ? w / total : 0.0f;
  } else if (has) {
    w = p.softmax ? expf(y - m) / sum : 1.0f / (1.0f + expf(-y));
  }
  if (lane < p.k) {
    p.ids[out] = chosen;
    p.weights[out] = !has ? 0.0f : bad ? __int_as_float(0x7FC00000) : w * p.scale;
  }
}

template <int PER>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const Route p) {
  extern __shared__ double s_scores[];  // [kWarps][scratch]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < p.rows; row += (long long)gridDim.x * kWarps) {
    route_row<PER>(p, (int)row, lane, s_scores + warp * p.scratch);
    __syncwarp();  // the next row takes the same scratch
  }
}

template <int PER>
static cudaError_t launch_per(Route p, cudaStream_t s) {
  // scores of a row in 64 bits, and at least room for 64 of them with their experts and places
  p.scratch = p.groups > 1 && p.experts > 128 ? p.experts : 128;
  p.group_magic = (int)(((1u << 20) + p.group_size - 1) / p.group_size);  // e * magic >> 20 = e / group_size for e < 1024
  p.group_share = 1;
  while (p.group_share * 2 * p.groups <= 32) p.group_share *= 2;
  const size_t smem = (size_t)kWarps * p.scratch * 8;  // 32 KB at most
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // up to 12 CTAs an SM (no kernel has room for more than 10), each warp then takes several rows: 8,191 x 256 in groups 25.7 us, with up to
  // 4 CTAs 34.8, 6 27.8, 24 25.8; 30,000 x 256 92.9, with 24 88.9
  const long long ctas = (p.rows + kWarps - 1) / kWarps, most = (long long)sms * 12;
  return kv8::launch(route_kernel<PER>, dim3((unsigned)(ctas < most ? ctas : most)), kWarps * 32, smem, s, p);
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
