// The training operators' status word (see lopt_train.h): a variable of the
// module, so that it is zero before anything can run, and there for calls
// that are captured, of any thread, and for graphs that outlive their maker.
#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

__device__ int32_t g_status;

__global__ void k_status_clear(int32_t flags) { atomicAnd(&g_status, ~flags); }

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" {

int lopt_status_word(int32_t** word) {
  if (!word) return LOPT_E_ARG;
  // The first use of the module may load it, which a thread that captures a
  // stream may only do in this mode.  No stream is touched.
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return done(e);
  void* p = nullptr;
  e = cudaGetSymbolAddress(&p, g_status);
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  *word = static_cast<int32_t*>(p);
  return done(e != cudaSuccess ? e : back);
}

int lopt_status_take(int32_t* flags) {
  if (!flags) return LOPT_E_ARG;
  *flags = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return done(e);
  int32_t got = 0;
  if ((e = cudaMemcpyFromSymbol(&got, g_status, sizeof(got))) != cudaSuccess) return done(e);
  if (got) {   // those bits alone: another thread's call may have set one since
    if ((e = launch(k_status_clear, dim3(1), dim3(1), 0, nullptr, false, 1, got)) != cudaSuccess) return done(e);
    if ((e = cudaDeviceSynchronize()) != cudaSuccess) return done(e);
  }
  *flags = got;
  return LOPT_OK;
}

}  // extern "C"
