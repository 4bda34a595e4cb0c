// The distillation kernels for bfloat16 logits.
#define LOPT_DISTILL_KERNELS
#include "distill_rows.cuh"

namespace lopt {
namespace train {
cudaError_t distill_bf16(const Distill& a, uint64_t wait_ns, int sms, cudaStream_t s) {
  return distill_rows<__nv_bfloat16>(a, wait_ns, sms, s);
}
}  // namespace train
}  // namespace lopt
