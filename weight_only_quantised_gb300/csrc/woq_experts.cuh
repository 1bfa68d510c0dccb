// Experts' products over packed int4 / int6 weights (include/woq_block.h):
//   h_e,t = silu(G_e x_t) * U_e x_t,   part = D_e h,   y_t = sum_j w_tj part_tj.
//
// A decode step's few rows choose many experts, so a launch is bound by the bytes of the chosen experts' weights, each read
// once: two blocks of 128 x 128 weights arrive at an SM every 740 cycles, and what is done for them has to stay below that.
//   - A, the weights, as 8-bit floats: the codes 0 .. 15 of e4m3 are themselves times 2^-9 (the subnormals, and the least
//     exponent), so a nibble with its top bit flipped is w + 8 with nothing but a mask: 3 operations per 8 weights.  int6's two
//     top bits are a product of their own, worth 16.  (mma.sync has no 8-bit floats on this part, the compiler converts them to
//     f16; with bf16 operands, 9 to 11 operations per 8 weights, it was issue bound: 8 rows of 128 experts 48 us, here 37.5.)
//   - B, the rows: x is the sum of a high and a low half in e4m3 (4 significant bits each, bf16 has 8), two columns of B, under
//     a power of two per row and group of 128.  Exact, but for elements below 2^-13 of the group's largest, which are off by at
//     most 2^-17 of it.  h is taken apart the same way from fp32, with one rounding (2^-8 at most, of a bf16's kind).
//   - tcgen05.mma kind::f8f6f4, A in tensor memory: D[128 rows of weights][2 columns a row] in fp32, one per group, then
//     acc += scale (D_high + D_low / 16 - 8 sum(high + low / 16)) 2^e in fp32, a thread a row of weights.  M 128, N 16 to 64, K 32 takes 32 cycles
//     whatever N is.
// Roles of a CTA (one per SM): two pairs of teams of four warps, which make A from a block (shared memory -> registers -> tensor
// memory) and add up D, in each pair one team for gate and one for up (down: two neighbouring tiles), the pairs in turn, as
// a step takes a team 1,500 cycles of latency; a warp that copies blocks (bulk copies of 8 KB); one that issues the
// products; two that bring B; and four that take a unit's sums from the teams and finish it (2 us and more of latency,
// during which the teams go on).  The copying and the issuing warp run as whole warps with one elected lane: from a branch on the
// lane, two copies took 700 cycles and eight products 1,400.
// The steps (a group of a pair of tiles of an item) are dealt out evenly to the CTAs; a unit that several share is finished
// by the one that comes last, from all their sums in CTA order, and nobody waits for another CTA.
#pragma once

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

constexpr int kTeamThreads = 128;
// warps 0 .. 15: the teams
constexpr int kProducer = 16, kIssuer = 17, kBringer = 18, kBringers = 2, kFinisher = 20, kFinishers = 4;
constexpr int kThreads = (kFinisher + kFinishers) * 32;
constexpr int kColumns = 512;  // of tensor memory

// ---------------------------------------------------------------------------------------- halves

// What a group's elements are multiplied by before they become e4m3: 2^7 over the power of two of the largest magnitude
// (e: its exponent field), 16 times that for the low halves; and what undoes it.  Groups below 2^-116 share one factor.
__device__ __forceinline__ int group_exponent(uint32_t field) { return max((int)field, 11); }
__device__ __forceinline__ float group_factor(int e) { return __int_as_float((261 - e) << 23); }
__device__ __forceinline__ float group_undo(int e) { return __int_as_float(e == 255 ? 0x7FC00000 : (e - 7) << 23); }  // inf, NaN: NaN

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Largest magnitudes of two pairs of bf16, NaN if there is one (signs are not kept).
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t most_field(uint32_t m) { return max(m & 0x7FFFu, m >> 16 & 0x7FFFu) >> 7; }

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x4(uint32_t p01, uint32_t p23) {
  return (uint32_t)e4m3x2(__uint_as_float(p01 << 16), __uint_as_float(p01 & 0xFFFF0000u)) |
         (uint32_t)e4m3x2(__uint_as_float(p23 << 16), __uint_as_float(p23 & 0xFFFF0000u)) << 16;
}

// Four e4m3 summed: a multiple of 2^-9 below 2^11, exact in fp32.
__device__ __forceinline__ float sum_of_codes(uint32_t c) {
  uint32_t lo, hi;
  kv8::f16x4_of_codes<WOQ_KV8_E4M3>(c, lo, hi);
  return (dev::half_bits_to_float(lo & 0xFFFFu) + dev::half_bits_to_float(lo >> 16)) +
         (dev::half_bits_to_float(hi & 0xFFFFu) + dev::half_bits_to_float(hi >> 16));
}
__device__ __forceinline__ void of_codes(uint16_t c, float& lo, float& hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(c));
  lo = dev::half_bits_to_float(d & 0xFFFFu), hi = dev::half_bits_to_float(d >> 16);
}
// What halves hold, high + low / 16, in units of 2^-13 (the low ones' last bit): whole numbers, so sums of them are exact
// and go by no order.
__device__ __forceinline__ int held_units(float high, float low) { return __float2int_rn(fmaf(high, 8192.0f, low * 512.0f)); }

// Of four bf16 (two pairs): their high halves (the value without its last four bits), their low ones (the rest, times 16), and
// the sum of what both hold, in units of 2^-13.
__device__ __forceinline__ void halves4(uint32_t x01, uint32_t x23, int e, uint32_t& high, uint32_t& low, int& sum) {
  const uint32_t f = (uint32_t)(261 - e) << 7, f2 = f | f << 16, f16 = f2 + 0x02000200u, zero = 0x80008000u;
  const uint32_t h01 = x01 & 0xFFF0FFF0u, h23 = x23 & 0xFFF0FFF0u;
  high = e4m3x4(fma2(h01, f2, zero), fma2(h23, f2, zero));
  low = e4m3x4(fma2(h01, f16 ^ zero, fma2(x01, f16, zero)), fma2(h23, f16 ^ zero, fma2(x23, f16, zero)));
  sum = held_units(sum_of_codes(high), sum_of_codes(low));
}

// A group of a row in halves: 8 x [16 high][16 low], 256 bytes; beside it what undoes the factor and what takes the codes'
// offset off: -8 or -32 times the sum of what the halves hold (not of what they were made from: the products see the halves, and a
// rounding must not count w + 8 times), in codes' units.  Rounded once from the whole number, as a sum of products with codes
// that are all 0 is, so those give 0.
__device__ __forceinline__ float2 group_meta(int e, int units, int bits) {
  return make_float2(group_undo(e), (float)units * (bits == 4 ? -0x1p-19f : -0x1p-17f));
}

// ----------------------------------------------------------------------------------- tensor memory

__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Sixteen columns of the thread's row: there after tmem_loaded.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
// Waits for every load of the thread; r: so that nothing uses them before.
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (128 x N, fp32) = or += A (tensor memory, 128 x 32 e4m3) B (shared memory, N x 32 e4m3).
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(dev::smem_addr(bar)) : "memory");
}
// B as core matrices of 8 columns x 16 bytes: 128 bytes from one to the next along k, 1024 from 8 columns to the next 8.
__device__ __forceinline__ uint64_t b_descriptor(uint32_t at) {
  return (uint64_t)(at >> 4 & 0x3FFF) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46;
}
template <int N>
constexpr uint32_t kIdesc = 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(128 >> 4) << 24;  // fp32 sums, A and B e4m3 along k, M = 128

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.b32 %0, 1, 0, p;}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void fence_for_products() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------------------- products

// Sizes of a kernel for N columns of B (items of N / 2 rows).
template <int BITS, int N>
struct Shape {
  static constexpr int kRows = N / 2;  // of an item
  static constexpr int kBlock = BITS == 4 ? kBlockBytesW4 : kBlockBytesW6;
  static constexpr int kB = 2 * kBlock, kUndo = kB + N * 128, kLess = kUndo + kRows * 4, kStage = (kLess + kRows * 4 + 127) / 128 * 128;
  static constexpr int kACols = BITS == 4 ? 32 : 64, kDCols = BITS == 4 ? N : 2 * N;
  // Of A and of D, a team: with two of A the next block becomes A while the last one's products are under way.
  static constexpr int kTeamCols = kColumns / 4, kBuffers = 2 * kACols + kDCols <= kTeamCols ? 2 : 1;
  static constexpr int kSums = kBuffers * (kACols + kDCols) <= kTeamCols ? kBuffers : 1;
  static_assert(kBuffers * kACols + kSums * kDCols <= kTeamCols, "tensor memory");
  // [stages][exchange: units' sums by pairs, then the finishers' maxima and sums][barriers and flags]
  static constexpr int kUnits = N == 16 ? 2 : 1;  // units' sums that there is room for
  static constexpr int kExchange = kUnits * 2 * kRows * 256 * 4 + 2 * 4 * kRows * 4;
  static constexpr int kMisc = 1024;
  static constexpr int kRoom = 227 * 1024 - kExchange - kMisc;
  // An even number, so that a stage always serves the same pair: a wait for a parity two phases ahead returns at once.
  static constexpr int kStages = (kRoom / kStage < 12 ? kRoom / kStage : 12) / 2 * 2;
  static_assert(kStages >= 2 * kBuffers + 2, "a stage is held until its sums are taken");
  static constexpr int kBytes = kStages * kStage + kExchange + kMisc;
};

struct Barriers {
  uint64_t weights[12], operands[12], empty[12];  // operands: a step's B (one arrival) and its two A (eight)
  uint64_t done[2][2];                            // a pair's products
  uint64_t given[2][2], taken[2][2];              // a pair's sums of a unit, to the finishers
  uint64_t finishers;                             // where their warps meet
  uint32_t tmem;
  int fail, last;
};
static_assert(sizeof(Barriers) <= 1024, "misc");

// GATED: rows of gate and up, silu and product, h in halves; else the down projection's parts.
template <int BITS, bool GATED, int N>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const Experts p) {
  typedef Shape<BITS, N> Z;
  extern __shared__ __align__(128) uint8_t s_mem[];
  float* const s_unit = reinterpret_cast<float*>(s_mem + Z::kStages * Z::kStage);  // [units][pair][rows][256]
  uint32_t* const s_most = reinterpret_cast<uint32_t*>(s_unit + Z::kUnits * 2 * Z::kRows * 256);
  int* const s_sums = reinterpret_cast<int*>(s_most + 4 * Z::kRows);
  Barriers& s = *reinterpret_cast<Barriers*>(s_mem + Z::kStages * Z::kStage + Z::kExchange);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint64_t limit = p.wait_ns;

  if (tid == 0) {
    for (int i = 0; i < Z::kStages; ++i) {
      dev::mbar_init(&s.weights[i], 1);
      dev::mbar_init(&s.operands[i], 9);
      dev::mbar_init(&s.empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) dev::mbar_init(&s.done[i >> 1][i & 1], 1);
    for (int i = 0; i < 4; ++i) {
      dev::mbar_init(&s.given[i >> 1][i & 1], 8);
      dev::mbar_init(&s.taken[i >> 1][i & 1], kFinishers);
    }
    dev::mbar_init(&s.finishers, kFinishers);
    s.fail = 0;
    dev::fence_mbar_init();
  }
  if (warp == kIssuer)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_addr(&s.tmem)), "n"(kColumns) : "memory");
  // The down projection's launch may read the plan, which was there before the one it waits for began.
  if (GATED) dev::pdl_wait_prior_grids();
  dev::pdl_launch_dependents();
  const int items = (int)p.status[1];
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;

  const int K = GATED ? p.hidden : p.inner, groups = K / kGroup;
  const int tiles = GATED ? p.inner / kTileRows : p.hidden / kTileRows, slices = GATED ? tiles : (tiles + 1) / 2;
  const int units = items * slices, total = units * groups;
  const int cta = blockIdx.x, grid = gridDim.x;
  // Shares of whole units where the longest is not much longer than those of steps: putting a unit together takes as long as
  // some eight steps.  Share c has `each` of them, and one more if c < more.  128 experts, 1 / 8 / 500 rows: 21.0 / 37.6 / 166 us, with a bound
  // of 0 steps 22.3 / 41.5 / 205, of 16 20.5 / 38.2 / 160; 3 rows of 8 large experts 68.3, of whole units only 89.6.
  const bool whole = (units + grid - 1) / grid * groups <= total / grid + 8;
  const int least = whole ? groups : 1, each = (whole ? units : total) / grid, more = (whole ? units : total) - each * grid;
  const int begin = (each * cta + min(cta, more)) * least, end = begin + (each + (cta < more)) * least;
  const auto cta_of = [&](int step) { return step < more * (each + 1) ? step / (each + 1) : more + (step - more * (each + 1)) / each; };
  const auto failed = [&]() {
    *(volatile int*)&s.fail = 1;
    atomicOr(p.status, (uint32_t)WOQ_DEVERR_TIMEOUT);
    p.status[2] = 1;  // y is not written then
  };
  const auto gave_up = [&]() { return *(volatile int*)&s.fail != 0; };
  // By whole warps: false once a wait has run out, here or elsewhere in the CTA.  Warps that run ahead or behind sleep a little between
  // tries: with 23 warps that try all the time, a wait that is over at once takes 72 cycles instead of 16.
  const bool sleeps = warp == kProducer || warp >= kBringer;
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    bool ok = dev::mbar_try_wait(bar, parity);
    if (!ok) {
      const uint64_t t0 = dev::global_timer_ns();
      while (!(ok = dev::mbar_try_wait(bar, parity)) && !gave_up()) {
        if (sleeps) __nanosleep(40);
        if (dev::global_timer_ns() - t0 > limit) failed();
      }
    }
    return (bool)__all_sync(~0u, ok);
  };

  int issued = 0, last = -1;  // the producer's copies; the issuer's newest products: pair, buffer and parity
  if (warp == kProducer) {
    if (begin < end) {
      const uint8_t* const matrices = GATED ? p.gate_up : p.down;
      const size_t stride = GATED ? p.gate_up_stride : p.down_stride;
      int unit = begin / groups, g = begin - unit * groups;
      int at_item = -1, expert = 0;
      const uint8_t *src0, *src1;
      const auto locate = [&]() {
        const int item = unit / slices, slice = unit - item * slices;
        if (item != at_item) expert = p.item[item].expert, at_item = item;
        const uint8_t* const m = matrices + (size_t)expert * stride + kHeaderBytes;
        const int t0 = GATED ? slice : 2 * slice, t1 = GATED ? slice + tiles : 2 * slice + 1;
        src0 = m + ((size_t)t0 * groups + g) * Z::kBlock;
        src1 = GATED || t1 < tiles ? m + ((size_t)t1 * groups + g) * Z::kBlock : nullptr;
      };
      locate();
      int stage = 0;
      uint32_t parity = 1;
      for (int i = begin; i < end; ++i) {
        if (!wait(&s.empty[stage], parity)) break;
        if (p.fault_cta != cta) {
          if (elected()) {
            uint8_t* const at = s_mem + (size_t)stage * Z::kStage;
            dev::mbar_arrive_expect_tx(&s.weights[stage], src1 ? 2 * Z::kBlock : Z::kBlock);
            dev::bulk_copy_g2s(at, src0, Z::kBlock, &s.weights[stage]);
            if (src1) dev::bulk_copy_g2s(at + Z::kBlock, src1, Z::kBlock, &s.weights[stage]);
          }
          __syncwarp();
          ++issued;
        }
        if (++g == groups) {
          g = 0;
          ++unit;
          if (i + 1 < end) locate();
        } else {
          src0 += Z::kBlock;
          if (src1) src1 += Z::kBlock;
        }
        if (++stage == Z::kStages) stage = 0, parity ^= 1;
      }
    }
  } else if (warp == kIssuer) {
    int stage = 0;
    uint32_t stage_parity = 0;
    const uint32_t base = dev::smem_addr(s_mem);
    for (int i = 0; i < end - begin; ++i) {
      if (!wait(&s.operands[stage], stage_parity)) break;
      tmem_fence_after();
      const uint64_t b = b_descriptor(base + stage * Z::kStage + Z::kB);
      const int pair = i & 1, turn = i >> 1, buffer = turn % Z::kBuffers;
      if (elected()) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t at = tmem + (pair * 2 + w) * Z::kTeamCols, a = at + buffer * Z::kACols;
          const uint32_t d = at + Z::kBuffers * Z::kACols + turn % Z::kSums * Z::kDCols;
#pragma unroll
          for (int k = 0; k < 4; ++k) mma(d, a + 8 * k, b + k * (256 >> 4), kIdesc<N>, k > 0);
          if (BITS == 6) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma(d + N, a + 32 + 8 * k, b + k * (256 >> 4), kIdesc<N>, k > 0);
          }
        }
        mma_commit(&s.done[pair][buffer]);
      }
      __syncwarp();
      last = (pair * 2 + buffer) * 2 + (turn / Z::kBuffers & 1);
      if (++stage == Z::kStages) stage = 0, stage_parity ^= 1;
    }
  } else if (warp >= kBringer && warp < kFinisher) {
    if (!GATED) dev::pdl_wait_prior_grids();  // h
    const int me = warp - kBringer;
    const auto arrive = [&](int stage) {
      fence_for_products();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&s.operands[stage]);
    };
    const auto free_stage = [&](int n) { return wait(&s.empty[n % Z::kStages], ((uint32_t)(n / Z::kStages) & 1u) ^ 1u); };  // for step n of this CTA
    // pieces of 16 bytes: piece lane & 15 of two rows at a time
    const uint8_t* const halves = GATED ? p.x_halves : p.h_halves;
    const float* const meta = reinterpret_cast<const float*>(GATED ? p.x_meta : p.h_meta);
    const int half = lane >> 4, piece = lane & 15;
    const uint32_t base = dev::smem_addr(s_mem), to = Z::kB + (piece >> 1) * 128 + half * 32 + (piece & 1) * 16;
    constexpr int kAhead = Z::kStages >= 10 ? 2 : 1;  // copies of this many steps are under way
    uint32_t from[Z::kRows / 2], from_meta = 0;       // of rows 2 j + half, bytes (below 2^31); of row `lane`, floats
    int item = -1, rows = 0, pending = 0, i = begin + me;
    bool ok = true;
    for (; i < end; i += kBringers) {
      const int unit = i / groups, g = i - unit * groups, at_item = unit / slices;
      if (at_item != item) {
        item = at_item;
        const ExpertItem it = p.item[item];
        rows = it.rows;
#pragma unroll
        for (int j = 0; j < Z::kRows / 2; ++j) {
          const int r = 2 * j + half, place = r < rows ? p.order[it.first + r] : 0;
          from[j] = (uint32_t)(GATED ? place / p.k : place) * (uint32_t)groups * 256u + (uint32_t)piece * 16u;
        }
        const int place = lane < rows ? p.order[it.first + lane] : 0;
        from_meta = (uint32_t)(GATED ? place / p.k : place) * (uint32_t)groups * 2u;
      }
      const int n = i - begin;
      if (!(ok = free_stage(n))) break;
      const uint32_t at = base + (n % Z::kStages) * Z::kStage;
      const uint8_t* const src = halves + (size_t)g * 256;
#pragma unroll
      for (int j = 0; j < Z::kRows / 2; ++j)
        if (2 * j + half < rows) copy16(at + to + (j >> 1) * 1024 + (j & 1) * 64, src + from[j]);
      if (lane < rows) {
        copy4(at + Z::kUndo + lane * 4, meta + from_meta + 2 * g);
        copy4(at + Z::kLess + lane * 4, meta + from_meta + 2 * g + 1);
      }
      copies_commit();
      if (++pending > kAhead) {
        copies_wait<kAhead>();
        arrive((n - kAhead * kBringers) % Z::kStages);
        --pending;
      }
    }
    copies_wait<0>();
    // the last steps (if the loop ended early nobody waits for them any more)
    if (ok)
      for (; pending > 0; --pending) arrive((i - begin - pending * kBringers) % Z::kStages);
  } else if (warp >= kFinisher) {
    if (!GATED) dev::pdl_wait_prior_grids();  // the sums of split units lie where the launch before had its own
    const int me = tid - kFinisher * 32, quad = warp - kFinisher;
    uint32_t phase = 0;
    const auto meet = [&]() {  // false: something has failed, here or elsewhere
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&s.finishers);
      phase ^= 1;
      return wait(&s.finishers, phase ^ 1);
    };
    int turns[2] = {0, 0};  // units that each pair has given
    for (int step = begin; step < end;) {
      const int unit = step / groups, first_step = unit * groups, last_step = min(first_step + groups, end);
      // a pair that had a step of it
      const bool gave[2] = {last_step - step > 1 || !((step - begin) & 1), last_step - step > 1 || ((step - begin) & 1)};
      const int item = unit / slices, slice = unit - item * slices;
      const ExpertItem it = p.item[item];
      const int rows = it.rows, places = lane < rows ? p.order[it.first + lane] : 0;  // lane t: of row t
      const auto place_of = [&](int t) { return (size_t)__shfl_sync(~0u, places, t); };
      int buffer[2];
      bool ok = true;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        buffer[w] = turns[w] % Z::kUnits;
        if (gave[w]) ok = ok && wait(&s.given[buffer[w]][w], (uint32_t)(turns[w] / Z::kUnits) & 1u);
      }
      if (!ok) break;
      step = last_step;
      // this thread's rows: me of the first tile, and of the second 128 on
      float* const sums0 = s_unit + (buffer[0] * 2) * (Z::kRows * 256) + me;
      float* const sums1 = s_unit + (buffer[1] * 2 + 1) * (Z::kRows * 256) + me;
      float* const sums = gave[0] ? sums0 : sums1;
      // the CTAs of the unit's first and last step
      const int a = whole ? cta : cta_of(first_step), b = whole ? cta : cta_of(first_step + groups - 1);
      if (gave[0] && gave[1]) {
#pragma unroll 4
        for (int i = 0; i < 2 * rows; ++i) sums[i * 128] += sums1[i * 128];
      }
      bool mine = true;
      if (a != b) {
        constexpr size_t kWords = (size_t)Z::kRows * 256;
        float* const part = p.split_sums + ((size_t)cta * 2 + (first_step >= begin ? 1 : 0)) * kWords + me;
#pragma unroll 4
        for (int i = 0; i < 2 * rows; ++i) __stcg(part + i * 128, sums[i * 128]);
        if (!meet()) break;
        if (me == 0) {
          __threadfence();  // of all that the meeting has brought together
          const uint32_t before = dev::atomic_add_acq_rel_gpu(p.split_counts + a, 1u);
          s.last = before == (uint32_t)(b - a);
          if (s.last) p.split_counts[a] = 0;
        }
        if (!meet()) break;
        mine = s.last;
        if (mine) {
          // in CTA order; eight loads are under way at a time
          const float* const parts = p.split_sums + me;
          for (int i = 0; i < 2 * rows; i += 2) {
            float v0 = 0.0f, v1 = 0.0f;
            for (int c = a; c <= b; c += 4) {
              float w[4][2];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* const from = parts + ((size_t)(c + j) * 2 + (c + j == a ? 1 : 0)) * kWords + i * 128;
                w[j][0] = c + j <= b ? __ldcg(from) : 0.0f;
                w[j][1] = c + j <= b ? __ldcg(from + 128) : 0.0f;
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) v0 += w[j][0], v1 += w[j][1];
            }
            sums[i * 128] = v0;
            sums[i * 128 + 128] = v1;
          }
        }
      }
      // codes were taken as 2^-9 of themselves
      if (mine) {
        if constexpr (!GATED) {
          const bool second = 2 * slice + 1 < tiles;
#pragma unroll 4
          for (int t = 0; t < rows; ++t) {
            float* const to = p.parts + place_of(t) * p.hidden + 2 * slice * kTileRows + me;
            to[0] = 512.0f * sums[t * 256];
            if (second) to[kTileRows] = 512.0f * sums[t * 256 + 128];
          }
        } else {
          // h = silu(gate) up of 128 neighbouring elements of each row: a group of down's, taken apart here
#pragma unroll 4
          for (int t = 0; t < rows; ++t) {
            const float v = 512.0f * sums[t * 256], h = __fdividef(v, 1.0f + expf(-v)) * (512.0f * sums[t * 256 + 128]);
            sums[t * 256] = h;
            const uint32_t m = __reduce_max_sync(~0u, __float_as_uint(h) & 0x7FFFFFFFu);
            if (lane == 0) s_most[quad * Z::kRows + t] = m;
          }
          if (!meet()) break;
          const auto exponent = [&](int t) {
            const uint32_t* const m = s_most + t;
            return group_exponent(max(max(m[0], m[Z::kRows]), max(m[2 * Z::kRows], m[3 * Z::kRows])) >> 23);
          };
          // two rows at a time (the last of an odd number twice)
#pragma unroll 2
          for (int t = 0; t < rows; t += 2) {
            const int t1 = min(t + 1, rows - 1);
            const float v0 = sums[t * 256] * group_factor(exponent(t)), v1 = sums[t1 * 256] * group_factor(exponent(t1));
            const uint16_t high = e4m3x2(v0, v1);
            float h0, h1, l0, l1;
            of_codes(high, h0, h1);
            const uint16_t low = e4m3x2((v0 - h0) * 16.0f, (v1 - h1) * 16.0f);
            of_codes(low, l0, l1);
            uint8_t* const to = p.h_halves + (size_t)slice * 256 + (me >> 4) * 32 + (me & 15);
            const size_t row_bytes = (size_t)(p.inner / kGroup) * 256;
            uint8_t *const to0 = to + place_of(t) * row_bytes, *const to1 = to + place_of(t1) * row_bytes;
            to0[0] = (uint8_t)high;
            to0[16] = (uint8_t)low;
            to1[0] = (uint8_t)(high >> 8);
            to1[16] = (uint8_t)(low >> 8);
            const int sum0 = __reduce_add_sync(~0u, held_units(h0, l0)), sum1 = __reduce_add_sync(~0u, held_units(h1, l1));
            if (lane == 0) s_sums[quad * Z::kRows + t] = sum0, s_sums[quad * Z::kRows + t1] = sum1;
          }
          if (!meet()) break;
          if (me < rows) {
            const int* const q = s_sums + me;
            p.h_meta[(size_t)places * (p.inner / kGroup) + slice] =
                group_meta(exponent(me), q[0] + q[Z::kRows] + q[2 * Z::kRows] + q[3 * Z::kRows], BITS);
          }
          if (!meet()) break;  // the maxima and sums may be written again
        }
      }
      __syncwarp();
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (gave[w]) {
          if (lane == 0) dev::mbar_arrive(&s.taken[buffer[w]][w]);
          ++turns[w];
        }
    }
  } else {
    // ------------------------------------------------------------------------------- the teams
    const int team = warp >> 2, pair = team >> 1, side = team & 1, quad = warp & 3, row = quad * 32 + lane;  // row of the tile
    const uint32_t my_tmem = tmem + ((uint32_t)(quad * 32) << 16) + team * Z::kTeamCols;
    dev::f32x2 acc[Z::kRows / 2] = {};  // two rows each
    constexpr int kLag = Z::kBuffers - 1;  // the pair's steps from making A to adding up D
    const int steps = end - begin > pair ? (end - begin - pair + 1) / 2 : 0;  // the pair's: every other one
    int g = (begin + pair) % groups, unit_buffer = 0;                         // of the step that is added up
    uint32_t unit_parity = 0;
    int stage = pair, stored = 0, added_stage = pair, buffer = 0, added_buffer = 0;
    uint32_t parity = 0, added_parity = 0;
    for (int n = 0; n < steps + kLag; ++n) {
      if (n < steps) {
        if (!wait(&s.weights[stage], parity)) break;
        const uint8_t* const block = s_mem + (size_t)stage * Z::kStage + side * Z::kBlock;
        const uint32_t at = my_tmem + buffer * Z::kACols;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a[16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(block + w4_chunk_offset(half * 2 + c, quad, lane));
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            constexpr uint32_t flip = BITS == 4 ? 0x08080808u : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a[c * 8 + 2 * j] = (w[j] & 0x0F0F0F0Fu) ^ flip;
              a[c * 8 + 2 * j + 1] = (w[j] >> 4 & 0x0F0F0F0Fu) ^ flip;
            }
          }
          tmem_store16(at + half * 16, a);
          if constexpr (BITS == 6) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint2 u2 = *reinterpret_cast<const uint2*>(block + hi_chunk_offset(half * 2 + c, quad, lane));
              const uint32_t u[2] = {u2.x, u2.y};
#pragma unroll
              for (int j = 0; j < 8; ++j) a[c * 8 + j] = (u[j >> 2] >> (2 * (j & 3)) & 0x03030303u) ^ 0x02020202u;
            }
            tmem_store16(at + 32 + half * 16, a);
          }
        }
        stored = stage;
        if ((stage += 2) >= Z::kStages) stage -= Z::kStages, parity ^= 1;
      }
      const auto announce = [&]() {  // the A that was stored
        tmem_wait_stores();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&s.operands[stored]);
        if (++buffer == Z::kBuffers) buffer = 0;
      };
      if (kLag == 0) announce();
      if (n >= kLag) {
        // with two buffers the store goes on meanwhile (and is announced behind this: there may be one D only)
        if (!wait(&s.done[pair][added_buffer], added_parity)) break;
        tmem_fence_after();
        const uint8_t* const st = s_mem + (size_t)added_stage * Z::kStage;
        const uint32_t at = my_tmem + Z::kBuffers * Z::kACols + (Z::kSums > 1 ? added_buffer * Z::kDCols : 0);
        const float scale = dev::half_bits_to_float(reinterpret_cast<const uint16_t*>(st + side * Z::kBlock)[scale_index(row)]);
        const dev::f32x2 scales = dev::f2_splat(scale);
        const ulonglong2* const undo = reinterpret_cast<const ulonglong2*>(st + Z::kUndo);  // of four rows each
        const ulonglong2* const less = reinterpret_cast<const ulonglong2*>(st + Z::kLess);
#pragma unroll
        for (int c = 0; c < N / 16; ++c) {
          uint32_t d[16];
          tmem_load16(at + 16 * c, d);
          tmem_loaded(d);
          if (BITS == 6) {
            uint32_t d2[16];
            tmem_load16(at + N + 16 * c, d2);
            tmem_loaded(d2);
#pragma unroll
            for (int j = 0; j < 16; ++j) d[j] = __float_as_uint(fmaf(16.0f, __uint_as_float(d2[j]), __uint_as_float(d[j])));
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const ulonglong2 u = undo[c * 2 + j], l = less[c * 2 + j];
            const dev::f32x2 us[2] = {u.x, u.y}, ls[2] = {l.x, l.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t* const v = d + 8 * j + 4 * i;
              const float t0 = fmaf(0.0625f, __uint_as_float(v[1]), __uint_as_float(v[0]));
              const float t1 = fmaf(0.0625f, __uint_as_float(v[3]), __uint_as_float(v[2]));
              dev::f32x2& to = acc[c * 4 + 2 * j + i];
              to = dev::f2_fma(dev::f2_mul(scales, us[i]), dev::f2_add(dev::f2_pack(__float_as_uint(t0), __float_as_uint(t1)), ls[i]), to);
            }
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&s.empty[added_stage]);
      }
      if (kLag > 0 && n < steps) announce();
      if (n < kLag) continue;
      if ((added_stage += 2) >= Z::kStages) added_stage -= Z::kStages;
      if (++added_buffer == Z::kBuffers) added_buffer = 0, added_parity ^= 1;
      g += 2;
      if (g < groups && n + 1 < steps + kLag) continue;

      // The pair's last step of the unit: the sums go to the finishers.
      if (!wait(&s.taken[unit_buffer][pair], unit_parity ^ 1u)) break;
      float* const to = s_unit + (unit_buffer * 2 + pair) * (Z::kRows * 256) + side * kTeamThreads + row;
#pragma unroll
      for (int t = 0; t < Z::kRows / 2; ++t) {
        to[t * 512] = __uint_as_float(dev::f2_lo(acc[t]));
        to[t * 512 + 256] = __uint_as_float(dev::f2_hi(acc[t]));
        acc[t] = 0;
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&s.given[unit_buffer][pair]);
      if (++unit_buffer == Z::kUnits) unit_buffer = 0, unit_parity ^= 1;
      while (g >= groups) g -= groups;
    }
    tmem_wait_stores();  // a step that was given up may have left some
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  // Every copy and product has been waited for by whoever takes what it gives, unless a wait ran out: nothing may be in flight when
  // the CTA ends, so then whoever issued them waits for the last ones (their loops may have ended before).
  if (s.fail) {
    if (warp == kProducer)
      for (int n = max(issued - Z::kStages, 0); n < issued; ++n) dev::mbar_wait_bounded(&s.weights[n % Z::kStages], (uint32_t)(n / Z::kStages) & 1u);
    // products end in order: with the newest, all have
    if (warp == kIssuer && last >= 0) dev::mbar_wait_bounded(&s.done[last >> 2][last >> 1 & 1], (uint32_t)last & 1u);
    __syncthreads();
  }
  if (warp == kIssuer) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}

template <int BITS, bool GATED, int N>
inline cudaError_t launch_product(const Experts& p, int sms, cudaStream_t s) {
  typedef Shape<BITS, N> Z;
  const cudaError_t e = cudaFuncSetAttribute(product_kernel<BITS, GATED, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::kBytes);
  if (e != cudaSuccess) return e;
  return kv8::launch(product_kernel<BITS, GATED, N>, dim3((unsigned)sms), kThreads, Z::kBytes, s, p);
}

}  // namespace experts
}  // namespace woq
