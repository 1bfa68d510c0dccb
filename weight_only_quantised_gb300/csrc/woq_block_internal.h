// Internal declarations of the parts of a block around its linears (include/woq_block.h): arguments of the kernels
// and their launchers, which return a cudaError_t.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

namespace woq {

struct BlockNorm {
  const void* u;
  const void* r;
  void* r_out;
  uint16_t* out;
  const uint16_t* post;
  const uint16_t* gate;
  const uint16_t* pre;
  int u_f32, r_f32;
  int rows, dim;
  int rows_per_gate;
  float alpha, beta, offset, eps, inv_dim;
};
cudaError_t launch_block_norm(const BlockNorm& p, cudaStream_t stream);

struct Route {
  const void* logits;
  const float* bias;
  const int32_t* live;
  int32_t* ids;
  float* weights;
  long long stride;
  int f32, softmax;
  int rows, experts, k;
  int groups, group_size, top_groups, group_best;
  int renormalise;
  float scale;
  int scratch, group_magic, group_share;  // set by the launcher
};
cudaError_t launch_route(const Route& p, cudaStream_t stream);

// Rows of one expert that are worked on together.
struct ExpertItem {
  int expert, first, rows, pad;  // entries order[first .. first + rows - 1]
};

struct Experts {
  const uint8_t* gate_up;
  const uint8_t* down;
  size_t gate_up_stride, down_stride;  // bytes from one expert's matrix to the next
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  uint16_t* y;
  int bits, experts, rows, k, hidden, inner;  // T, k, H, I
  int entries;                                // T k
  int item_rows;                              // most places of an item: 8, 16 or 32
  unsigned long long wait_ns;                 // bound of device waits
  int fault_cta;                              // a CTA that copies no weights (tests), -1: none
  // workspace
  uint32_t* status;   // word 0: WOQ_DEVERR_*; word 1: items; word 2: a wait ran out, and y is not written
  uint32_t* split_counts;  // [CTAs]: parts of a unit that have been written (zero between launches)
  float* split_sums;       // [CTAs][2][item rows][256]
  ExpertItem* item;
  int32_t* order;     // [entries]: places (t k + j) by expert
  uint8_t* x_halves;  // [rows][H / 128][256]: x in two e4m3 halves
  float2* x_meta;     // [rows][H / 128]: what undoes their factor, and what the codes' offset adds
  uint8_t* h_halves;  // [entries][I / 128][256]
  float2* h_meta;     // [entries][I / 128]
  float* parts;       // [entries][H]
};
constexpr int kLeastItemRows = 8;  // rows of an item, where they are fewest
constexpr int kMostCtas = 256;
constexpr int kMostEntries = 32768;
cudaError_t launch_experts(const Experts& p, cudaStream_t stream);

}  // namespace woq
