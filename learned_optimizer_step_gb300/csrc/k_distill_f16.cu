// The distillation kernels for float16 logits.
#define LOPT_DISTILL_KERNELS
#include "distill_rows.cuh"

namespace lopt {
namespace train {
cudaError_t distill_f16(const Distill& a, uint64_t wait_ns, int sms, cudaStream_t s) {
  return distill_rows<__half>(a, wait_ns, sms, s);
}
}  // namespace train
}  // namespace lopt
