// block_api.cu -- extern "C" entry points of the operators around the layer
// (layer norm, router, 4-bit matrix-vector products): host-side argument checks
// (nothing is enqueued when one fails), then the launch.
#include <cmath>

#include "moe_internal.h"

namespace moe {

namespace {

moe_status finish(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  record_cuda_error(e);
  return MOE_ERR_CUDA;
}

int elem_bytes(int32_t dtype) {
  switch (dtype) {
    case MOE_ELEM_F32: return 4;
    case MOE_ELEM_BF16:
    case MOE_ELEM_F16: return 2;
  }
  return 0;
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool given(const moe_rows* m) { return m && m->data; }

// A row matrix of `rows` x `cols` elements: element-aligned, rows apart, of an
// extent that 64-bit sums of bytes hold.
bool rows_ok(const moe_rows* m, int64_t rows, int64_t cols, int bytes) {
  if (rows == 0) return m != nullptr;
  if (!given(m) || !aligned_to(m->data, (size_t)bytes)) return false;
  if (rows == 1) return true;
  return m->stride >= cols && m->stride <= (int64_t(1) << 40) && rows - 1 <= (int64_t(1) << 56) / m->stride;
}

// The same matrix: equal base, and equal strides where there is a second row.
bool same_rows(const moe_rows* a, const moe_rows* b, int64_t rows) {
  return given(a) && given(b) && a->data == b->data && (rows <= 1 || a->stride == b->stride);
}

// Whether the bytes the two matrices span overlap.
bool overlap(const moe_rows* a, int64_t acols, const moe_rows* b, int64_t bcols, int64_t rows, int bytes) {
  if (!given(a) || !given(b) || rows == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a->data), b0 = reinterpret_cast<uintptr_t>(b->data);
  const uintptr_t an = (uintptr_t)(((rows > 1 ? (rows - 1) * a->stride : 0) + acols) * bytes);
  const uintptr_t bn = (uintptr_t)(((rows > 1 ? (rows - 1) * b->stride : 0) + bcols) * bytes);
  if (!(a0 < b0 + bn && b0 < a0 + an)) return false;
  // column blocks of one wider matrix interleave without touching
  if (rows > 1 && a->stride == b->stride) {
    const uintptr_t s = (uintptr_t)a->stride * bytes;
    const uintptr_t d = a0 <= b0 ? (b0 - a0) % s : s - 1 - (a0 - b0 - 1) % s;
    if (d % s >= (uintptr_t)acols * bytes && d + (uintptr_t)bcols * bytes <= s) return false;
  }
  return true;
}

moe_status check_norm(const moe_norm* n) {
  if (!n || n->rows < 0 || n->rows > (int64_t(1) << 40) || n->H < 1 || n->H > (1 << 20)) return MOE_ERR_INVALID_ARG;
  if (!elem_bytes(n->dtype) || (n->param_dtype != n->dtype && n->param_dtype != MOE_ELEM_F32))
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(n->eps) || n->eps < 0.0f) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_router(const moe_router* r, int32_t format) {
  if (!r || r->T < 0 || r->E < 1 || r->E > 1024 || r->K < 1 || r->K > 128 || r->K > r->E) return MOE_ERR_INVALID_ARG;
  if (r->T >= (int64_t(1) << 40) / r->E) return MOE_ERR_INVALID_ARG;
  if (!elem_bytes(r->logits_dtype) || (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) ||
      !std::isfinite(r->scale))
    return MOE_ERR_INVALID_ARG;
  if (format != MOE_ROUTING_DENSE_I16 && format != MOE_ROUTING_SPARSE_BOOL) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_w4(const moe_w4* w) {
  if (!w || w->N < 1 || w->N > (1 << 24) || w->Kd < 32 || w->Kd > (1 << 20) || w->Kd % 32) return MOE_ERR_INVALID_ARG;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_ERR_INVALID_ARG;
  if (w->dtype != MOE_ELEM_BF16 && w->dtype != MOE_ELEM_F16) return MOE_ERR_INVALID_ARG;
  if (!w->codes || !aligned_to(w->codes, 16) || !w->scales || !aligned_to(w->scales, 16) ||
      !aligned_to(w->zeros, 16))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_w4_call(const moe_w4* w, int64_t rows, const moe_rows* x, int32_t activation, const moe_rows* y) {
  if (activation != MOE_W4_NONE && activation != MOE_W4_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (activation == MOE_W4_SWIGLU && w->N % 2) return MOE_ERR_INVALID_ARG;
  const int64_t n_out = activation == MOE_W4_SWIGLU ? w->N / 2 : w->N;
  if (!rows_ok(x, rows, w->Kd, 2) || !rows_ok(y, rows, n_out, 2)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!aligned_to(x->data, 16) || (rows > 1 && x->stride % 8))) return MOE_ERR_INVALID_ARG;
  if (overlap(x, w->Kd, y, n_out, rows, 2)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

#define MOE_TRY(expr)              \
  do {                             \
    moe_status _st = (expr);       \
    if (_st != MOE_OK) return _st; \
  } while (0)

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layer_norm(const moe_norm* norm, const moe_rows* x, const moe_rows* residual, const void* weight,
                          const void* bias, const moe_rows* y, const moe_rows* sum, float* mean, float* rstd,
                          void* stream) {
  MOE_TRY(check_norm(norm));
  const int b = elem_bytes(norm->dtype), pb = elem_bytes(norm->param_dtype);
  const int64_t rows = norm->rows, H = norm->H;
  if (!rows_ok(x, rows, H, b) || !rows_ok(y, rows, H, b)) return MOE_ERR_INVALID_ARG;
  if (given(residual) && !rows_ok(residual, rows, H, b)) return MOE_ERR_INVALID_ARG;
  if (given(sum) && (!given(residual) || !rows_ok(sum, rows, H, b))) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(weight, pb) || !aligned_to(bias, pb) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (overlap(y, H, x, H, rows, b) || overlap(y, H, residual, H, rows, b) || overlap(y, H, sum, H, rows, b))
    return MOE_ERR_INVALID_ARG;
  if ((overlap(sum, H, x, H, rows, b) && !same_rows(sum, x, rows)) ||
      (overlap(sum, H, residual, H, rows, b) && !same_rows(sum, residual, rows)))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  return finish(launch_layer_norm(*norm, *x, given(residual) ? residual : nullptr, weight, bias, *y,
                                  given(sum) ? sum : nullptr, mean, rstd, static_cast<cudaStream_t>(stream)));
}

moe_status moe_layer_norm_workspace_size(int64_t rows, int64_t H, size_t* bytes_out) {
  if (!bytes_out || rows < 0 || H < 1 || H > (1 << 20)) return MOE_ERR_INVALID_ARG;
  *bytes_out = layer_norm_workspace_bytes(rows, H);
  return MOE_OK;
}

moe_status moe_layer_norm_backward(const moe_norm* norm, const moe_rows* grad_y, const moe_rows* h, const void* weight,
                                   const float* mean, const float* rstd, const moe_rows* grad_sum,
                                   const moe_rows* grad_x, float* grad_weight, float* grad_bias, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  MOE_TRY(check_norm(norm));
  const int b = elem_bytes(norm->dtype), pb = elem_bytes(norm->param_dtype);
  const int64_t rows = norm->rows, H = norm->H;
  if (!rows_ok(grad_y, rows, H, b) || !rows_ok(h, rows, H, b) || !rows_ok(grad_x, rows, H, b))
    return MOE_ERR_INVALID_ARG;
  if (given(grad_sum) && !rows_ok(grad_sum, rows, H, b)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!mean || !rstd)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(weight, pb) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(grad_weight, 4) ||
      !aligned_to(grad_bias, 4))
    return MOE_ERR_INVALID_ARG;
  if (overlap(grad_x, H, h, H, rows, b) ||
      (overlap(grad_x, H, grad_y, H, rows, b) && !same_rows(grad_x, grad_y, rows)) ||
      (overlap(grad_x, H, grad_sum, H, rows, b) && !same_rows(grad_x, grad_sum, rows)))
    return MOE_ERR_INVALID_ARG;
  if (grad_weight || grad_bias) {
    if (!workspace || !aligned_to(workspace, 16)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < layer_norm_workspace_bytes(rows, H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  return finish(launch_layer_norm_backward(*norm, *grad_y, *h, weight, mean, rstd, given(grad_sum) ? grad_sum : nullptr,
                                           *grad_x, grad_weight, grad_bias, workspace,
                                           static_cast<cudaStream_t>(stream)));
}

moe_status moe_router_topk(const moe_router* router, const moe_rows* logits, const float* select_bias,
                           int32_t map_format, void* map, float* probs, int32_t* status, void* stream) {
  MOE_TRY(check_router(router, map_format));
  if (!rows_ok(logits, router->T, router->E, elem_bytes(router->logits_dtype))) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(select_bias, 4) || !aligned_to(status, 4)) return MOE_ERR_INVALID_ARG;
  if (router->T == 0) return MOE_OK;
  if (!map || !probs || !aligned_to(map, map_format == MOE_ROUTING_DENSE_I16 ? 2 : 1) || !aligned_to(probs, 4))
    return MOE_ERR_INVALID_ARG;
  return finish(launch_router_topk(*router, *logits, select_bias, map_format, map, probs, status,
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_router_topk_backward(const moe_router* router, const moe_rows* logits, int32_t map_format,
                                    const void* map, const float* grad_probs, const moe_rows* grad_logits,
                                    void* stream) {
  MOE_TRY(check_router(router, map_format));
  const int b = elem_bytes(router->logits_dtype);
  if (!rows_ok(logits, router->T, router->E, b) || !rows_ok(grad_logits, router->T, router->E, b))
    return MOE_ERR_INVALID_ARG;
  if (overlap(logits, router->E, grad_logits, router->E, router->T, b) &&
      !same_rows(logits, grad_logits, router->T))
    return MOE_ERR_INVALID_ARG;
  if (router->T == 0) return MOE_OK;
  if (!map || !grad_probs || !aligned_to(map, map_format == MOE_ROUTING_DENSE_I16 ? 2 : 1) ||
      !aligned_to(grad_probs, 4))
    return MOE_ERR_INVALID_ARG;
  return finish(launch_router_topk_backward(*router, *logits, map_format, map, grad_probs, *grad_logits,
                                            static_cast<cudaStream_t>(stream)));
}

moe_status moe_w4_matvec(const moe_w4* w, int64_t M, const moe_rows* x, int32_t activation, const moe_rows* addend,
                         const moe_rows* y, void* stream) {
  MOE_TRY(check_w4(w));
  if (M < 0 || M > (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_w4_call(w, M, x, activation, y));
  if (given(addend)) {
    if (activation != MOE_W4_NONE || !rows_ok(addend, M, w->N, 2)) return MOE_ERR_INVALID_ARG;
    if (overlap(addend, w->N, y, w->N, M, 2) && !same_rows(addend, y, M)) return MOE_ERR_INVALID_ARG;
  }
  if (M == 0) return MOE_OK;
  return finish(launch_w4_matvec(*w, M, *x, activation, given(addend) ? addend : nullptr, *y,
                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_grouped_w4_matvec(const moe_handle_dev* handle, const moe_shape* shape, const moe_layout* layout,
                                 const moe_w4* w, const moe_rows* x, int32_t activation, const moe_rows* y,
                                 void* stream) {
  if (!handle || !handle->tokens_per_expert || !handle->padded_offsets) return MOE_ERR_INVALID_ARG;
  if (!shape || shape->T < 0 || shape->E < 1 || shape->E > 1024 || shape->K < 1 || shape->K > 128 ||
      shape->K > shape->E || shape->T >= (int64_t(1) << 31) / shape->K)
    return MOE_ERR_INVALID_ARG;
  if (!layout || layout->capacity < 0 || layout->capacity >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_w4(w));
  MOE_TRY(check_w4_call(w, layout->capacity, x, activation, y));
  if (shape->T == 0 || layout->capacity == 0) return MOE_OK;
  return finish(launch_grouped_w4_matvec(*handle, *shape, *layout, *w, *x, activation, *y,
                                         static_cast<cudaStream_t>(stream)));
}

moe_status moe_quantize_w4_rows(const void* w, int64_t R, int64_t Kd, int32_t group, int32_t dtype, void* codes,
                                void* scales, void* zeros, void* stream) {
  if (R < 0 || R > (int64_t(1) << 40) || Kd < 32 || Kd > (1 << 20) || Kd % 32) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_ELEM_BF16 && dtype != MOE_ELEM_F16) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!w || !codes || !scales || !aligned_to(w, 2) || !aligned_to(scales, 2)) return MOE_ERR_INVALID_ARG;
  return finish(
      launch_quantize_w4_rows(w, R, Kd, group, dtype, codes, scales, zeros, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
