// C ABI entry points of the operators on rows of logits (include/dflash.h): argument checks.
#include <cmath>

#include "nvtx.h"
#include "rows.h"
#include "workspace.h"

namespace df {
namespace {

int rows_ok(const df_rows* x) {
  if (!x || x->rows < 0 || (x->dtype != DF_F32 && x->dtype != DF_BF16) || x->V < 1 || x->ld < x->V) return DF_ERR_ARG;
  if (x->V > 1 << 20 || x->rows > 1 << 27 || (x->rows && x->ld > ((int64_t)1 << 62) / x->rows)) return DF_ERR_SHAPE;
  if (x->rows == 0) return DF_OK;
  if (!x->data) return DF_ERR_ARG;
  return al16(x->data) ? DF_OK : DF_ERR_ALIGN;
}

// A gradient's array is the student's own or lies apart from it.
bool grad_ok(const df_rows* x, const void* grad, int64_t ld_grad) {
  if (!grad || x->rows == 0 || (grad == x->data && ld_grad == x->ld)) return true;
  const size_t es = x->dtype == DF_F32 ? 4 : 2;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x->data), b = reinterpret_cast<uintptr_t>(grad);
  const size_t na = ((size_t)(x->rows - 1) * x->ld + x->V) * es, nb = ((size_t)(x->rows - 1) * ld_grad + x->V) * es;
  return a + na <= b || b + nb <= a;
}

bool temperature_ok(float t) { return t >= 0x1p-100f && t <= 0x1p100f; }

int distill_ok(const df_rows* x, int K, int n_teacher, const int32_t* teacher_row, float temperature, int64_t ld_grad,
               const void* grad) {
  DF_TRY(rows_ok(x));
  if (K < 1 || n_teacher < 0 || !temperature_ok(temperature) || (!teacher_row && n_teacher < x->rows)) return DF_ERR_ARG;
  if (grad && ld_grad < x->V) return DF_ERR_ARG;
  if (K > 1024 || (grad && x->rows && ld_grad > ((int64_t)1 << 62) / x->rows)) return DF_ERR_SHAPE;
  if (!grad_ok(x, grad, ld_grad)) return DF_ERR_ARG;
  return grad && !al16(grad) ? DF_ERR_ALIGN : DF_OK;
}

}  // namespace
}  // namespace df

using namespace df;

extern "C" {

size_t dflash_sample_workspace_size(int rows, int V) {
  (void)V;
  Carver cv(nullptr);
  cv.take<SampleLeft>(rows > 0 ? (size_t)rows : 1);
  return cv.off;
}

int dflash_sample(const df_rows* x, int group, const float* temperature, const int32_t* top_k, const float* top_p,
                  const float* min_p, const float* u, int32_t* token, float* logprob, int32_t* n_kept, void* ws,
                  size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_sample");
  DF_TRY(rows_ok(x));
  if (group < 1 || x->rows % group) return DF_ERR_ARG;
  if (x->rows == 0) return DF_OK;
  if (!u || !token) return DF_ERR_ARG;
  if (!ws || ws_bytes < dflash_sample_workspace_size(x->rows, x->V)) return DF_ERR_WORKSPACE;
  SampleArgs a{};
  a.x = *x; a.group = group; a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p; a.u = u;
  a.token = token; a.logprob = logprob; a.n_kept = n_kept; a.status = status_of(ws);
  Carver cv(ws);
  a.left = cv.take<SampleLeft>((size_t)x->rows);
  return launch_sample(a, (cudaStream_t)stream);
}

size_t dflash_top_logits_workspace_size(int rows, int V) {
  (void)rows; (void)V;
  return kAlign;
}

int dflash_top_logits(const df_rows* x, int K, float temperature, int32_t* id, float* val, float* lse, void* ws,
                      size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_top_logits");
  DF_TRY(rows_ok(x));
  if (K < 1 || !temperature_ok(temperature)) return DF_ERR_ARG;
  if (K > 1024) return DF_ERR_SHAPE;
  if (x->rows == 0) return DF_OK;
  if (!id || !val) return DF_ERR_ARG;
  if (!ws || ws_bytes < dflash_top_logits_workspace_size(x->rows, x->V)) return DF_ERR_WORKSPACE;
  TopArgs a{};
  a.x = *x; a.K = K; a.temperature = temperature; a.id = id; a.val = val; a.lse = lse; a.status = status_of(ws);
  return launch_top_logits(a, (cudaStream_t)stream);
}

size_t dflash_distill_workspace_size(int rows, int V) {
  (void)rows; (void)V;
  return kAlign;
}

int dflash_distill(const df_rows* x, int K, int n_teacher, const int32_t* id, const float* val, const float* lse,
                   const int32_t* teacher_row, float temperature, const float* weight, float* loss, float* stats,
                   void* grad, int64_t ld_grad, void* ws, size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_distill");
  DF_TRY(distill_ok(x, K, n_teacher, teacher_row, temperature, ld_grad, grad));
  if (x->rows == 0) return DF_OK;
  if ((n_teacher && (!id || !val)) || !loss || !stats) return DF_ERR_ARG;
  if (!al16(stats)) return DF_ERR_ALIGN;
  if (!ws || ws_bytes < dflash_distill_workspace_size(x->rows, x->V)) return DF_ERR_WORKSPACE;
  DistillArgs a{};
  a.x = *x; a.K = K; a.n_teacher = n_teacher; a.id = id; a.val = val; a.lse = lse; a.teacher_row = teacher_row;
  a.temperature = temperature; a.weight = weight; a.loss = loss; a.stats = stats; a.grad = grad; a.ld_grad = ld_grad;
  a.status = status_of(ws);
  return launch_distill(a, (cudaStream_t)stream);
}

int dflash_distill_backward(const df_rows* x, int K, int n_teacher, const int32_t* id, const float* val,
                            const float* lse, const int32_t* teacher_row, float temperature, const float* weight,
                            const float* stats, const float* grad_loss, void* grad, int64_t ld_grad, void* ws,
                            size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_distill_backward");
  DF_TRY(distill_ok(x, K, n_teacher, teacher_row, temperature, ld_grad, grad));
  if (x->rows == 0) return DF_OK;
  if ((n_teacher && (!id || !val)) || !grad || !stats) return DF_ERR_ARG;
  if (!al16(stats)) return DF_ERR_ALIGN;
  if (!ws || ws_bytes < dflash_distill_workspace_size(x->rows, x->V)) return DF_ERR_WORKSPACE;
  DistillArgs a{};
  a.x = *x; a.K = K; a.n_teacher = n_teacher; a.id = id; a.val = val; a.lse = lse; a.teacher_row = teacher_row;
  a.temperature = temperature; a.weight = weight; a.stats = const_cast<float*>(stats); a.grad_loss = grad_loss;
  a.grad = grad; a.ld_grad = ld_grad; a.status = status_of(ws);
  return launch_distill_backward(a, (cudaStream_t)stream);
}

int dflash_path_rows(int b, int D, int n_tree, const int32_t* n_new, const int32_t* src_slot, int max_src,
                     const int32_t* cache_len, int32_t* teacher_row, df_stream stream) {
  DF_NVTX("dflash_path_rows");
  if (b < 0 || D < 1 || n_tree < 1 || max_src < 0 || max_src < D - 1) return DF_ERR_ARG;
  if ((long long)b * D > (1 << 27) || (long long)b * n_tree > 2147483647LL) return DF_ERR_SHAPE;
  if (b == 0) return DF_OK;
  if (!n_new || !cache_len || !teacher_row || (D > 1 && !src_slot)) return DF_ERR_ARG;
  return launch_path_rows(b, D, n_tree, n_new, src_slot, max_src, cache_len, teacher_row, (cudaStream_t)stream);
}

}  // extern "C"
