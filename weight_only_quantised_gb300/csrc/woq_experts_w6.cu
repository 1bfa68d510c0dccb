// Experts' products: the int6 kernels.
#include "woq_experts.cuh"

namespace woq {
namespace experts {

cudaError_t launch_products_w6(const Experts& p, bool gated, int sms, cudaStream_t s) {
  if (p.item_rows == 8) return gated ? launch_product<6, true, 16>(p, sms, s) : launch_product<6, false, 16>(p, sms, s);
  return gated ? launch_product<6, true, 32>(p, sms, s) : launch_product<6, false, 32>(p, sms, s);
}

}  // namespace experts
}  // namespace woq
