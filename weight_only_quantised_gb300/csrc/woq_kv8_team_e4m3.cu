// Attention over a cache of e4m3 codes, a team of warps per block.
#include "woq_kv8_attn.cuh"

namespace woq {

cudaError_t launch_kv8_team_e4m3(const Kv8Attn& p, int ctas, int smem, cudaStream_t s) {
  return kv8::launch_team_any<WOQ_KV8_E4M3>(p, ctas, smem, s);
}

}  // namespace woq
