// Attention over a cache of int8 codes: instances by head size and query tiles per warp.
#include "woq_kv8_attn.cuh"

namespace woq {

cudaError_t launch_kv8_attn_int8(const Kv8Attn& p, int ctas, int smem, cudaStream_t s) {
  switch (p.v.dim * 4 + p.tiles) {
    case 64 * 4 + 1: return kv8::launch_attn<WOQ_KV8_INT8, 64, 1>(p, ctas, smem, s);
    case 64 * 4 + 2: return kv8::launch_attn<WOQ_KV8_INT8, 64, 2>(p, ctas, smem, s);
    case 128 * 4 + 1: return kv8::launch_attn<WOQ_KV8_INT8, 128, 1>(p, ctas, smem, s);
    case 128 * 4 + 2: return kv8::launch_attn<WOQ_KV8_INT8, 128, 2>(p, ctas, smem, s);
    case 256 * 4 + 1: return kv8::launch_attn<WOQ_KV8_INT8, 256, 1>(p, ctas, smem, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace woq
