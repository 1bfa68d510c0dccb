// Experts' products: what surrounds the products of woq_experts.cuh (the plan and x in halves; the weighted sum), and the
// launches.
#include "woq_experts.cuh"

namespace woq {
namespace experts {

cudaError_t launch_products_w4(const Experts& p, bool gated, int sms, cudaStream_t s);
cudaError_t launch_products_w6(const Experts& p, bool gated, int sms, cudaStream_t s);

constexpr int kBeginThreads = 256;
constexpr int kPlanWarps = kBeginThreads / 32;
// Up to so many places each is compared with all others: 64 places 37.6 us (a call of 8 rows of 128 experts), counted 38.9; 128 55.0
// and 55.9, 256 68.5 and 69.0 (most of that difference the time that the longer code takes to arrive).
constexpr int kFewEntries = kBeginThreads;
static_assert(kBeginThreads * 4 == 1024, "four experts a thread");

// The plan, made by one CTA: places by expert, in the order of their numbers, and the items (up to p.item_rows places of one expert).
// Which places share an item decides where the products of a row are cut between CTAs, and so the order of its sums: it must not go by
// which of several warps comes first.

// Up to a place a thread: the rank of each by comparing it with all others, then a thread a rank.
__device__ __forceinline__ void plan_few(const Experts& p) {
  __shared__ int4 s_keys[kBeginThreads / 4];  // expert 256 + place
  __shared__ int s_sorted[kBeginThreads + 1];
  __shared__ uint32_t s_firsts[kBeginThreads / 32], s_lasts[kBeginThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.entries;
  const bool busy = warp * 32 < n;
  int e = tid < n ? p.ids[tid] : -1;
  if ((unsigned)e >= (unsigned)p.experts) e = 1024;  // none: behind all
  const int key = e << 8 | tid;
  reinterpret_cast<int*>(s_keys)[tid] = key;
  if (tid == 0) s_sorted[n] = 1024;
  if (lane == 0) s_firsts[warp] = s_lasts[warp] = 0;
  __syncthreads();
  if (busy) {
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
      const int4 o = s_keys[j >> 2];
      rank += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
    }
    if (tid < n) {
      s_sorted[rank] = e;
      if (e < 1024) p.order[rank] = tid;
    }
  }
  __syncthreads();
  const int expert = busy && tid < n ? s_sorted[tid] : 1024;
  const bool here = expert < 1024;
  const unsigned firsts = __ballot_sync(~0u, here && (tid == 0 || s_sorted[tid - 1] != expert));
  if (lane == 0) s_firsts[warp] = firsts;
  __syncthreads();
  int in_item = 0;  // places of the expert before this one, in its item
  if (here) {
    int w = warp;
    uint32_t m = firsts & (2u << lane) - 1;
    while (m == 0) m = s_firsts[--w];  // the expert's first place is in an earlier word
    in_item = (tid - (w * 32 + 31 - __clz(m))) & (p.item_rows - 1);  // 8, 16 or 32
  }
  const bool last = here && (in_item == p.item_rows - 1 || s_sorted[tid + 1] != expert);
  const unsigned lasts = __ballot_sync(~0u, last);
  if (lane == 0) s_lasts[warp] = lasts;
  __syncthreads();
  int item = __popc(lasts & (1u << lane) - 1), items = 0;
#pragma unroll
  for (int i = 0; i < kBeginThreads / 32; ++i) {
    const int here_too = __popc(s_lasts[i]);
    item += i < warp ? here_too : 0;
    items += here_too;
  }
  if (last) p.item[item] = ExpertItem{expert, tid - in_item, in_item + 1, 0};
  if (tid == 0) p.status[1] = (uint32_t)items;
}

// Any number: each warp has a run of places and counts them for itself; thread i looks after experts 4 i .. 4 i + 3.
__device__ __forceinline__ void plan_many(const Experts& p) {
  __shared__ int4 s_counts[kPlanWarps][1024 / 4];  // of each warp's run; then where the next of them goes
  __shared__ int s_sums[33];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.entries + 32 * kPlanWarps - 1) / (32 * kPlanWarps) * 32;
  for (int w = 0; w < kPlanWarps; ++w) s_counts[w][tid] = make_int4(0, 0, 0, 0);
  __syncthreads();
  int* const mine = reinterpret_cast<int*>(s_counts[warp]);
  const int begin = min(warp * run, p.entries), end = min(begin + run, p.entries);
  // Sixteen ids of a lane are on their way at a time, of places from + lane + 32 j (-1: none); a run of no more is loaded once.
  constexpr int kAtOnce = 16;
  int e[kAtOnce];
  const auto load = [&](int from) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) e[j] = from + 32 * j + lane < end ? p.ids[from + 32 * j + lane] : -1;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if ((unsigned)e[j] >= (unsigned)p.experts) e[j] = -1;
  };
  for (int from = begin; from < end; from += 32 * kAtOnce) {
    load(from);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (e[j] >= 0) atomicAdd(mine + e[j], 1);
  }
  __syncthreads();
  const int most = p.item_rows;
  int count[4] = {}, sum = 0, items = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    const int4 c = s_counts[w][tid];
    count[0] += c.x, count[1] += c.y, count[2] += c.z, count[3] += c.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sum += count[j];
    items += (count[j] + most - 1) / most;
  }
  // both sums in one scan: entries (at most 32,768) above items (at most 5,120)
  int total;
  const int before = kv8::block_exclusive_sum(sum << 13 | items, s_sums, &total);
  int first = before >> 13, item = before & 0x1FFF;
  int4 at = make_int4(first, first + count[0], first + count[0] + count[1], first + count[0] + count[1] + count[2]);
  for (int w = 0; w < kPlanWarps; ++w) {
    const int4 c = s_counts[w][tid];
    s_counts[w][tid] = at;
    at.x += c.x, at.y += c.y, at.z += c.z, at.w += c.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    for (int i = 0; i < count[j]; i += most, ++item)
      p.item[item] = ExpertItem{4 * tid + j, first + i, count[j] - i < most ? count[j] - i : most, 0};
    first += count[j];
  }
  __syncthreads();
  for (int from = begin; from < end; from += 32 * kAtOnce) {
    if (run > 32 * kAtOnce) load(from);
#pragma unroll
    for (int q = 0; q < kAtOnce; q += 4) {
      if (from + 32 * q >= end) break;
      unsigned same[4];  // the lanes with this expert
#pragma unroll
      for (int j = 0; j < 4; ++j) same[j] = __match_any_sync(~0u, e[q + j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int id = e[q + j], next = id >= 0 ? mine[id] : 0, ahead = __popc(same[j] & ((1u << lane) - 1));
        __syncwarp();
        if (id >= 0) {
          if (ahead == 0) mine[id] = next + __popc(same[j]);
          p.order[next + ahead] = from + 32 * (q + j) + lane;
        }
        __syncwarp();
      }
    }
  }
  if (tid == 0) p.status[1] = (uint32_t)(total & 0x1FFF);
}

// Before gate and up: the plan (CTA 0), and x in halves, a warp per group.
__global__ void __launch_bounds__(kBeginThreads) begin_kernel(const Experts p) {
  dev::pdl_launch_dependents();
  dev::pdl_wait_prior_grids();
  if (blockIdx.x == 0) {
    if (p.entries <= kFewEntries) plan_few(p);
    else plan_many(p);
    return;
  }
  const int lane = threadIdx.x & 31;
  const size_t group = (size_t)(blockIdx.x - 1) * (kBeginThreads / 32) + (threadIdx.x >> 5);
  if (group >= (size_t)p.rows * (p.hidden / kGroup)) return;
  const uint2 x = *reinterpret_cast<const uint2*>(p.x + group * kGroup + lane * 4);
  const int e = group_exponent(__reduce_max_sync(~0u, most_field(most2(x.x, x.y))));
  uint32_t high, low;
  int sum;
  halves4(x.x, x.y, e, high, low, sum);
  sum = __reduce_add_sync(~0u, sum);
  uint8_t* const to = p.x_halves + group * 256 + (lane >> 2) * 32 + (lane & 3) * 4;
  *reinterpret_cast<uint32_t*>(to) = high;
  *reinterpret_cast<uint32_t*>(to + 16) = low;
  if (lane == 0) p.x_meta[group] = group_meta(e, sum, p.bits);
}

__device__ __forceinline__ bool matrix_ok(const uint8_t* m, int bits, int N, int K) {
  const PackedHeader* h = reinterpret_cast<const PackedHeader*>(m);
  return h->magic == kMagic && h->version == kLayoutVersion && h->bits == (uint32_t)bits && h->N == (uint32_t)N &&
         h->K == (uint32_t)K;
}

// y_t = sum over its places, in their order.  The row's ids, weights and the headers of its matrices are looked at before the
// wait for the products: a row with a header that does not match keeps its y.
__global__ void __launch_bounds__(256) sum_kernel(const Experts p) {
  __shared__ int s_here[32];
  __shared__ float s_weight[32];
  const int row = blockIdx.x, tid = threadIdx.x, c = (blockIdx.y * 256 + tid) * 4;
  const size_t first = (size_t)row * p.k;
  dev::pdl_launch_dependents();
  int flags = 0;
  if (tid < p.k) {
    const int e = p.ids[first + tid];
    const bool here = (unsigned)e < (unsigned)p.experts;
    s_here[tid] = here;
    s_weight[tid] = p.weights[first + tid];
    if (here) {
      if (!matrix_ok(p.gate_up + (size_t)e * p.gate_up_stride, p.bits, 2 * p.inner, p.hidden) ||
          !matrix_ok(p.down + (size_t)e * p.down_stride, p.bits, p.hidden, p.inner))
        flags = WOQ_DEVERR_HEADER;
    } else if (e != -1) {
      flags = WOQ_DEVERR_STATE;
    }
  }
  const bool bad = __syncthreads_or(flags & WOQ_DEVERR_HEADER);
  dev::pdl_wait_prior_grids();
  // a wait that ran out, in this call or in an earlier one: every call that writes nothing says so
  const bool gave_up = p.status[2] != 0;
  if (gave_up && tid == 0) flags |= WOQ_DEVERR_TIMEOUT;
  if (flags) atomicOr(p.status, (uint32_t)flags);
  if (bad || c >= p.hidden || gave_up) return;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* const parts = p.parts + first * p.hidden + c;
  for (int j = 0; j < p.k; j += 8) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < p.k && s_here[j + i]) v[i] = *reinterpret_cast<const float4*>(parts + (size_t)(j + i) * p.hidden);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < p.k && s_here[j + i]) {
        const float w = s_weight[j + i];
        y.x = fmaf(w, v[i].x, y.x);
        y.y = fmaf(w, v[i].y, y.y);
        y.z = fmaf(w, v[i].z, y.z);
        y.w = fmaf(w, v[i].w, y.w);
      }
  }
  *reinterpret_cast<uint2*>(p.y + (size_t)row * p.hidden + c) =
      make_uint2(pro::f32_to_bf16_bits(y.x) | pro::f32_to_bf16_bits(y.y) << 16,
                 pro::f32_to_bf16_bits(y.z) | pro::f32_to_bf16_bits(y.w) << 16);
}

}  // namespace experts

cudaError_t launch_experts(const Experts& p, cudaStream_t s) {
  using namespace experts;
  int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (sms > kMostCtas) sms = kMostCtas;
  const auto products = p.bits == 4 ? launch_products_w4 : launch_products_w6;
  const long long groups = (long long)p.rows * (p.hidden / kGroup);
  cudaError_t e = kv8::launch(begin_kernel, dim3((unsigned)(1 + (groups + 7) / 8)), kBeginThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  e = products(p, true, sms, s);
  if (e != cudaSuccess) return e;
  e = products(p, false, sms, s);
  if (e != cudaSuccess) return e;
  return kv8::launch(sum_kernel, dim3((unsigned)p.rows, (unsigned)((p.hidden + 1023) / 1024)), 256, 0, s, p);
}

}  // namespace woq
