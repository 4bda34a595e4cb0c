// Entry of the distillation loss (see lopt_train.h): checks and dispatch.
#include "distill_rows.cuh"

using namespace lopt::train;

namespace {

constexpr uint64_t kWaitNs = 1000000000ull;   // 1 s

int distill(const void* logits, int type, int64_t rows, int64_t cols, int64_t logits_stride,
            const void* top_logits, int top_type, int64_t top_logits_stride, const void* top_index, int index_type,
            int64_t top_index_stride, int64_t top, float temperature, const float* row_weight, float* loss, void* grad,
            int64_t grad_stride, int32_t* status, uint64_t wait_ns, void* stream) {
  const int es = type_size(type), ts = type_size(top_type), is = index_size(index_type);
  if (!es || !ts || !is || (top_type != LOPT_F32 && top_type != type)) return LOPT_E_ARG;
  // log2(e) / T is finite.  Above, T^2 times the rounding of the logarithms (some
  // 1e-6) is larger than the loss of a list of all classes, which no longer
  // grows with T.
  if (!(temperature >= 1e-30f && temperature <= 1e3f)) return LOPT_E_ARG;
  if (rows < 0 || cols < 1 || rows >= kMaxRows || cols > kMaxCols || top < 1 || top > LOPT_MAX_TOP) return LOPT_E_SHAPE;
  if (rows == 0) return LOPT_OK;
  const Span mz{logits, rows, cols, logits_stride, es}, mt{top_logits, rows, top, top_logits_stride, ts};
  const Span mi{top_index, rows, top, top_index_stride, is}, mw{row_weight, 1, rows, rows, 4};
  const Span ml{loss, 1, rows, rows, 4}, mg{grad, rows, cols, grad_stride, es};
  int rc;
  if ((rc = check_matrix(mz, false)) || (rc = check_matrix(mt, false)) || (rc = check_matrix(mi, false)) ||
      (rc = check_matrix(ml, true)))
    return rc;
  if (grad && (rc = check_matrix(mg, true))) return rc;
  if (row_weight && (rc = check_matrix(mw, false))) return rc;
  if (status && (uintptr_t)status % 4) return LOPT_E_ALIGN;
  if (overlap(ml, mg) || (overlap(mg, mz) && !mg.same_place(mz))) return LOPT_E_ALIAS;
  for (const Span* in : {&mt, &mi, &mw})
    if (overlap(ml, *in) || overlap(mg, *in)) return LOPT_E_ALIAS;
  if (overlap(ml, mz)) return LOPT_E_ALIAS;
  const Distill a{logits, top_logits, top_index, row_weight, loss, grad, status, rows, cols, logits_stride,
                  top_logits_stride, top_index_stride, grad_stride, (int)top, top_type, index_type, temperature,
                  1.4426950408889634f / temperature};
  cudaStream_t s = (cudaStream_t)stream;
  const int sms = sm_count();
  switch (type) {
    case LOPT_F32: return done(distill_f32(a, wait_ns, sms, s));
    case LOPT_F16: return done(distill_f16(a, wait_ns, sms, s));
    default: return done(distill_bf16(a, wait_ns, sms, s));
  }
}

}  // namespace

extern "C" {

int lopt_distill(const void* logits, int type, int64_t rows, int64_t cols, int64_t logits_stride, const void* top_logits,
                 int top_type, int64_t top_logits_stride, const void* top_index, int index_type,
                 int64_t top_index_stride, int64_t top, float temperature, const float* row_weight, float* loss,
                 void* grad, int64_t grad_stride, int32_t* status, void* stream) {
  return distill(logits, type, rows, cols, logits_stride, top_logits, top_type, top_logits_stride, top_index, index_type,
                 top_index_stride, top, temperature, row_weight, loss, grad, grad_stride, status, kWaitNs, stream);
}

int lopt_selftest_distill(int64_t limit_ns, const void* logits, int type, int64_t rows, int64_t cols,
                          int64_t logits_stride, const void* top_logits, int top_type, int64_t top_logits_stride,
                          const void* top_index, int index_type, int64_t top_index_stride, int64_t top,
                          float temperature, const float* row_weight, float* loss, void* grad, int64_t grad_stride,
                          int32_t* status, void* stream) {
  if (limit_ns < 0 || limit_ns > (int64_t)kWaitNs) return LOPT_E_ARG;
  return distill(logits, type, rows, cols, logits_stride, top_logits, top_type, top_logits_stride, top_index, index_type,
                 top_index_stride, top, temperature, row_weight, loss, grad, grad_stride, status, (uint64_t)limit_ns, stream);
}

}  // extern "C"
