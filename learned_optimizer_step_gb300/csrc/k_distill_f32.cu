// The distillation kernels for float32 logits.
#define LOPT_DISTILL_KERNELS
#include "distill_rows.cuh"

namespace lopt {
namespace train {
cudaError_t distill_f32(const Distill& a, int sms, cudaStream_t s) { return distill_rows<float>(a, sms, s); }
}  // namespace train
}  // namespace lopt
