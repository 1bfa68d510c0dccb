// Experts' products: the int4 kernels.
#include "woq_experts.cuh"

namespace woq {
namespace experts {

cudaError_t launch_products_w4(const Experts& p, bool gated, int sms, cudaStream_t s) {
  if (p.item_rows == 8) return gated ? launch_product<4, true, 16>(p, sms, s) : launch_product<4, false, 16>(p, sms, s);
  if (p.item_rows == 16) return gated ? launch_product<4, true, 32>(p, sms, s) : launch_product<4, false, 32>(p, sms, s);
  return gated ? launch_product<4, true, 64>(p, sms, s) : launch_product<4, false, 64>(p, sms, s);
}

}  // namespace experts
}  // namespace woq
