// Layout of the 8-bit key/value cache (include/woq_kv8.h) and the launchers of its kernels.
//
//   [256-byte header][lens][reserved][refs][map][moves][pairs][table][tails][pool]
//
// One page of the pool holds one block of 64 tokens of one sequence: a record for each (layer,
// kv head).  A record is one contiguous run, what a consumer warp of the attention reads in
// one bulk copy, in the order in which the tensor-core fragments take it:
//   64 D bytes of key codes, 8-row x 16-byte cores: row p, element d at
//     ((p / 8) (D / 16) + d / 16) 128 + (p % 8) 16 + d % 16,
//     row p holding token kv8_token_of_row(p);
//   64 D bytes of value codes, transposed, the same cores: element d, token j at
//     ((d / 8) 4 + j / 16) 128 + (d % 8) 16 + j % 16;
//   16 bytes: key scale, value scale, value scale times kUnit (fp32), zero.
// A lane (g = lane / 4, t = lane % 4) of the m16n8k16 pattern reads 16 bytes of row g of core
// t: the warp's 512 bytes are contiguous, so the reads are free of bank conflicts, and
// those 16 bytes are the lane's operands of four k-steps.  The token order of the key rows is the one
// that makes the transposed score fragments (movmatrix) the operand that meets 16 consecutive
// tokens of a value row.
//
// The tail of a (layer, sequence, head) is bf16: keys [72][D], then values transposed [D][72].
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "woq_kv8.h"

namespace woq {

constexpr int kKv8Block = WOQ_KV8_BLOCK;
constexpr int kKv8Tail = 72;  // 63 tokens and 8 draft rows, rounded up to whole 16-byte vectors
constexpr int kKv8MaxSeqs = 1024;
// The attention's weights are up to 2^14 in f16, which the value scale that they meet in fp32 takes off again: so the sums of
// weighted values never pass the sum of the values' magnitudes, as if weights were at most 1 (a power of two: exact, but for
// value scales below 2^-112, of which bits are lost under 2^-149).
constexpr float kUnit = 1.0f / 16384;
constexpr uint32_t kKv8Magic = 0x384B5657u;

#if defined(__CUDACC__)
#define WOQ_KV8_HD __host__ __device__
#else
#define WOQ_KV8_HD
#endif

// Token (0 .. 63) of key row p: with p = 16 i + r, tokens 16 t + 4 i + {0, 1} sit at r = 2 t + {0, 1}
// and tokens 16 t + 4 i + {2, 3} at r = 8 + 2 t + {0, 1}.
WOQ_KV8_HD inline int kv8_token_of_row(int p) {
  const int i = p >> 4, r = p & 15;
  return 16 * ((r & 7) >> 1) + 4 * i + (r & 1) + 2 * (r >> 3);
}

// Header words (uint32): 0 status, 1 magic, 2 config hash, 3 page limit
struct Kv8View {
  uint8_t* base;
  uint32_t hash;
  int fmt, layers, heads, dim, seqs, max_tokens, pages, blocks;  // blocks: row length of the table
  size_t lens, reserved, refs, map, moves, pairs, table, tails, pool, total;

  WOQ_KV8_HD size_t record_bytes() const { return (size_t)128 * dim + 16; }
  WOQ_KV8_HD size_t page_bytes() const { return record_bytes() * heads * layers; }
  WOQ_KV8_HD size_t tail_elems() const { return (size_t)2 * kKv8Tail * dim; }  // of one (layer, sequence, head)
  WOQ_KV8_HD uint32_t* status() const { return reinterpret_cast<uint32_t*>(base); }
  WOQ_KV8_HD int32_t* limit_p() const { return reinterpret_cast<int32_t*>(base) + 3; }
  WOQ_KV8_HD int32_t* lens_p() const { return reinterpret_cast<int32_t*>(base + lens); }
  WOQ_KV8_HD int32_t* reserved_p() const { return reinterpret_cast<int32_t*>(base + reserved); }
  WOQ_KV8_HD int32_t* refs_p() const { return reinterpret_cast<int32_t*>(base + refs); }
  WOQ_KV8_HD int32_t* map_p() const { return reinterpret_cast<int32_t*>(base + map); }
  WOQ_KV8_HD int4* moves_p() const { return reinterpret_cast<int4*>(base + moves); }
  WOQ_KV8_HD int32_t* pairs_p() const { return reinterpret_cast<int32_t*>(base + pairs); }
  WOQ_KV8_HD int32_t* table_row(int seq) const {
    return reinterpret_cast<int32_t*>(base + table) + (size_t)seq * blocks;
  }
  WOQ_KV8_HD uint16_t* tail(int layer, int seq, int head) const {
    return reinterpret_cast<uint16_t*>(base + tails) +
           (((size_t)layer * seqs + seq) * heads + head) * tail_elems();
  }
  WOQ_KV8_HD uint8_t* record(int page, int layer, int head) const {
    return base + pool + (((size_t)page * layers + layer) * heads + head) * record_bytes();
  }
};

// Rotary arguments as a kernel takes them.
struct Kv8Rope {
  const float* table;
  const int32_t* pos;
  int positions, half, interleaved, axes;  // half = rot_dim / 2; 0: no rotation
  uint8_t axis_of[128];
};

struct Kv8Append {
  Kv8View v;
  Kv8Rope rope;
  const int32_t* seqs;
  const void* qkv;
  uint16_t* q_out;
  long long row_stride;
  int layer, n, rows, q_heads, f32;  // append_rows: n entries of `rows`; prompt: n = sequence, rows = tokens
};

struct Kv8Attn {
  Kv8View v;
  const int32_t* seqs;
  const uint16_t* q;
  const uint32_t* vis;
  uint16_t* out;
  uint32_t* tickets;  // one word per CTA, that an item begins in and does not end in: zero between launches
  uint32_t* failed;   // not zero: a wait of a launch with this workspace ran out since it was zero-filled
  int2* joins;        // of each item: twice the first CTA with a part (+ 1: its second slot), number of parts
  float* parts;       // two parts per CTA of queries * (dim + 4) floats
  float scale_log2;
  int layer, n, rows, q_heads, group, window, sinks;
  int chunks, queries;  // parts that a kv head's rows * group queries are worked on in, and the queries of one
  int heads;         // items of an entry: kv heads * chunks, the chunks of one head next to each other
  int joined;        // 0: no item lies in several CTAs
  int team;          // 1: a team of four warps per block, 0: a warp
  int tiles;         // tiles of 8 queries of a team (a warp has one)
  int warps, query_groups, stages, ctas;
  int least_units;   // units a CTA takes at least (while there are more CTAs than that needs, they idle)
  int fault_cta;     // tests of the waits' bound: this CTA copies no records (-1: none)
  uint32_t wait_ns;  // bound of the waits in the ring
};

cudaError_t launch_kv8_init(const Kv8View& v, cudaStream_t s);
cudaError_t launch_rope_table(double theta, int half, int positions, float* table, cudaStream_t s);
cudaError_t launch_kv8_append_rows(const Kv8Append& p, cudaStream_t s);
cudaError_t launch_kv8_prompt(const Kv8Append& p, cudaStream_t s);
cudaError_t launch_kv8_accept_meta(const Kv8View& v, const int32_t* seqs, int n, const uint32_t* keep, cudaStream_t s);
cudaError_t launch_kv8_accept_rows(const Kv8View& v, int n, cudaStream_t s);  // what accept_meta decided
cudaError_t launch_kv8_extend(const Kv8View& v, int seq, int tokens, cudaStream_t s);
cudaError_t launch_kv8_fork(const Kv8View& v, const int32_t* src, const int32_t* dst, int n, cudaStream_t s);
cudaError_t launch_kv8_free(const Kv8View& v, const int32_t* seqs, int n, cudaStream_t s);
cudaError_t launch_kv8_copy(const Kv8View& src, const Kv8View& dst, const int32_t* src_seqs, const int32_t* dst_seqs,
                            int n, cudaStream_t s);
cudaError_t launch_kv8_compact(const Kv8View& v, int limit, cudaStream_t s);
cudaError_t launch_kv8_state(const Kv8View& v, int32_t* lens, int32_t* refs, int32_t* table, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8View& v, int layer, int layers, int seq, int first, int count, uint16_t* k,
                            uint16_t* vals, cudaStream_t s);

// Attention: fills in the launch shape for (dim, n, rows * group); returns the shared memory it takes,
// 0 if nothing fits.
int kv8_attn_plan(Kv8Attn* p, int smem_max);
cudaError_t launch_kv8_attn_int8(const Kv8Attn& p, int ctas, int smem, cudaStream_t s);
cudaError_t launch_kv8_attn_e4m3(const Kv8Attn& p, int ctas, int smem, cudaStream_t s);
cudaError_t launch_kv8_team_int8(const Kv8Attn& p, int ctas, int smem, cudaStream_t s);
cudaError_t launch_kv8_team_e4m3(const Kv8Attn& p, int ctas, int smem, cudaStream_t s);

}  // namespace woq
