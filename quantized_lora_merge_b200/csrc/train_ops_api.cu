// C ABI of the operators around the adapted linears in a training step: layer
// norm, embedding, gradient norm and clipping. Host-side validation and the
// order of launches; see include/intlora.h for the contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <memory>
#include <new>

#include "elem.cuh"
#include "intlora.h"
#include "intlora_kernels.h"
#include "train_ops.h"

using namespace intlora;

static_assert(INTLORA_TYPE_F32 == kF32 && INTLORA_TYPE_BF16 == kBf16 && INTLORA_TYPE_F16 == kF16,
              "public and internal element types agree");

namespace {

constexpr int64_t kMaxElements = int64_t{1} << 40;
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

intlora_status fail(intlora_status st, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  set_last_error(text);
  return st;
}

// The error is reported here and now: calls that returned it (cudaLaunchKernelEx,
// cudaFuncSetAttribute) leave it as the runtime's last error too, where the next
// call's first launch would find it.
intlora_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(INTLORA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool valid_type(int32_t type) { return type == kF32 || type == kBf16 || type == kF16; }
bool type_aligned(const void* p, int32_t type) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elem_bytes(type)) == 0;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

intlora_status check_list(const void* jobs, int32_t count) {
  set_last_error("");
  if (count < 0 || (count > 0 && jobs == nullptr))
    return fail(INTLORA_ERR_INVALID_ARG, "jobs must be a non-NULL array, count >= 0");
  return INTLORA_OK;
}

intlora_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need > 0 && (ws == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0))
    return fail(INTLORA_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) required", need);
  return INTLORA_OK;
}

// rows x n with a row stride: the size of what a call may touch.
intlora_status check_rows(const char* what, int k, const char* name, int64_t rows, int64_t n, int64_t ld) {
  if (rows > 1 && ld < n) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: ld_%s must be >= n", what, k, name);
  if (ld < 0 || ld > kMaxElements || (rows > 0 && ld > 0 && rows > kMaxElements / ld))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: rows * ld_%s exceeds 2^40", what, k, name);
  return INTLORA_OK;
}

intlora_status check_size(const char* what, int k, int64_t tokens, int64_t n) {
  if (tokens < 0 || n < 1) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: tokens >= 0 and n >= 1 required", what, k);
  if (tokens > kMaxRows || n > kMaxRows)
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: tokens and n must be < 2^31", what, k);
  if (tokens > kMaxElements / n) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: tokens*n exceeds 2^40", what, k);
  return INTLORA_OK;
}

// ------------------------------------------------------------------------
// layer norm
// ------------------------------------------------------------------------
intlora_status check_ln(const intlora_layer_norm_job& j, int k) {
  static const char* what = "layer norm";
  intlora_status s = check_size(what, k, j.tokens, j.n);
  if (s != INTLORA_OK) return s;
  if (!valid_type(j.x_type) || !valid_type(j.param_type) || !valid_type(j.y_type))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: types must be INTLORA_TYPE_*", what, k);
  if (!(j.eps >= 0.0f) || !std::isfinite(j.eps))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: eps must be finite and >= 0", what, k);
  if ((s = check_rows(what, k, "x", j.tokens, j.n, j.ld_x)) != INTLORA_OK) return s;
  if ((s = check_rows(what, k, "y", j.tokens, j.n, j.ld_y)) != INTLORA_OK) return s;
  if (j.tokens == 0) return INTLORA_OK;
  if (j.x == nullptr || j.y == nullptr) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: x and y are required", what, k);
  if (!type_aligned(j.x, j.x_type) || !type_aligned(j.y, j.y_type) || !type_aligned(j.weight, j.param_type) ||
      !type_aligned(j.bias, j.param_type) || !aligned4(j.mean) || !aligned4(j.rstd))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: a pointer is not aligned to its elements", what, k);
  return INTLORA_OK;
}

intlora_status check_lnb(const intlora_layer_norm_backward_job& j, int k) {
  static const char* what = "layer-norm-backward";
  intlora_status s = check_size(what, k, j.tokens, j.n);
  if (s != INTLORA_OK) return s;
  if (!valid_type(j.x_type) || !valid_type(j.param_type) || !valid_type(j.dy_type) || !valid_type(j.dx_type))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: types must be INTLORA_TYPE_*", what, k);
  if ((s = check_rows(what, k, "dy", j.tokens, j.n, j.ld_dy)) != INTLORA_OK) return s;
  if ((s = check_rows(what, k, "x", j.tokens, j.n, j.ld_x)) != INTLORA_OK) return s;
  if (j.dx != nullptr && (s = check_rows(what, k, "dx", j.tokens, j.n, j.ld_dx)) != INTLORA_OK) return s;
  if (j.tokens > 0 && (j.dy == nullptr || j.x == nullptr || j.mean == nullptr || j.rstd == nullptr))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: dy, x, mean and rstd are required", what, k);
  if (!type_aligned(j.dy, j.dy_type) || !type_aligned(j.x, j.x_type) || !type_aligned(j.weight, j.param_type) ||
      !type_aligned(j.dx, j.dx_type) || !aligned4(j.mean) || !aligned4(j.rstd) || !aligned4(j.dweight) ||
      !aligned4(j.dbias))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: a pointer is not aligned to its elements", what, k);
  return INTLORA_OK;
}

bool lnb_sums(const intlora_layer_norm_backward_job& j) { return j.dweight != nullptr || j.dbias != nullptr; }

// ------------------------------------------------------------------------
// embedding
// ------------------------------------------------------------------------
intlora_status check_emb(const intlora_embedding_job& j, int k) {
  static const char* what = "embedding";
  intlora_status s = check_size(what, k, j.tokens, j.n);
  if (s != INTLORA_OK) return s;
  if (j.vocab < 1 || j.vocab > kMaxRows)
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: vocab must be in [1, 2^31)", what, k);
  if (!valid_type(j.table_type) || !valid_type(j.y_type))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: types must be INTLORA_TYPE_*", what, k);
  if (j.id_bytes != 4 && j.id_bytes != 8)
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: id_bytes must be 4 or 8", what, k);
  if (!std::isfinite(j.scale)) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: scale must be finite", what, k);
  if ((s = check_rows(what, k, "table", j.vocab, j.n, j.ld_table)) != INTLORA_OK) return s;
  if ((s = check_rows(what, k, "y", j.tokens, j.n, j.ld_y)) != INTLORA_OK) return s;
  if (j.tokens == 0) return INTLORA_OK;
  if (j.table == nullptr || j.ids == nullptr || j.y == nullptr)
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: table, ids and y are required", what, k);
  if (!type_aligned(j.table, j.table_type) || !type_aligned(j.y, j.y_type) ||
      reinterpret_cast<uintptr_t>(j.ids) % static_cast<uintptr_t>(j.id_bytes) != 0 || !aligned4(j.invalid))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: a pointer is not aligned to its elements", what, k);
  return INTLORA_OK;
}

intlora_status check_embb(const intlora_embedding_backward_job& j, int k) {
  static const char* what = "embedding-backward";
  intlora_status s = check_size(what, k, j.tokens, j.n);
  if (s != INTLORA_OK) return s;
  if (j.vocab < 1 || j.vocab > kMaxRows)
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: vocab must be in [1, 2^31)", what, k);
  if (!valid_type(j.dy_type) || !valid_type(j.dtable_type))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: types must be INTLORA_TYPE_*", what, k);
  if (j.id_bytes != 4 && j.id_bytes != 8)
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: id_bytes must be 4 or 8", what, k);
  if (!std::isfinite(j.scale)) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: scale must be finite", what, k);
  if ((s = check_rows(what, k, "dtable", j.vocab, j.n, j.ld_dtable)) != INTLORA_OK) return s;
  if ((s = check_rows(what, k, "dy", j.tokens, j.n, j.ld_dy)) != INTLORA_OK) return s;
  if (j.dtable == nullptr) return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: dtable is required", what, k);
  if (j.tokens > 0 && (j.dy == nullptr || j.ids == nullptr))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: dy and ids are required", what, k);
  if (!type_aligned(j.dy, j.dy_type) || !type_aligned(j.dtable, j.dtable_type) ||
      reinterpret_cast<uintptr_t>(j.ids) % static_cast<uintptr_t>(j.id_bytes) != 0 || !aligned4(j.invalid))
    return fail(INTLORA_ERR_INVALID_ARG, "%s job %d: a pointer is not aligned to its elements", what, k);
  return INTLORA_OK;
}

// ------------------------------------------------------------------------
// gradient norm and clipping
// ------------------------------------------------------------------------
intlora_status check_grads(const intlora_grad_job* jobs, int32_t count) {
  intlora_status s = check_list(jobs, count);
  if (s != INTLORA_OK) return s;
  int64_t total = 0;
  for (int32_t k = 0; k < count; ++k) {
    const intlora_grad_job& j = jobs[k];
    if (j.count < 0) return fail(INTLORA_ERR_INVALID_ARG, "gradient job %d: count must be >= 0", k);
    if (!valid_type(j.type)) return fail(INTLORA_ERR_INVALID_ARG, "gradient job %d: type must be INTLORA_TYPE_*", k);
    if (j.count > kMaxElements - total)
      return fail(INTLORA_ERR_INVALID_ARG, "gradient job %d: the tensors' elements exceed 2^40", k);
    total += j.count;
    if (j.count == 0) continue;
    if (j.g == nullptr) return fail(INTLORA_ERR_INVALID_ARG, "gradient job %d: g is NULL", k);
    if (!type_aligned(j.g, j.type))
      return fail(INTLORA_ERR_INVALID_ARG, "gradient job %d: g is not aligned to its elements", k);
  }
  return INTLORA_OK;
}

// A tensor that is listed twice, or overlaps another, would be scaled twice.
struct Extent {
  uintptr_t begin, end;
  int32_t job;
};
Extent extent_of(const intlora_grad_job* jobs, int32_t k) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(jobs[k].g);
  return Extent{b, b + static_cast<uintptr_t>(jobs[k].count) * static_cast<uintptr_t>(elem_bytes(jobs[k].type)), k};
}
intlora_status check_disjoint(const intlora_grad_job* jobs, int32_t count) {
  // tensors in the order of their addresses, as an arena has them, need no sort
  bool ascending = true;
  uintptr_t end = 0;
  for (int32_t k = 0; k < count && ascending; ++k) {
    if (jobs[k].count == 0) continue;
    const Extent e = extent_of(jobs, k);
    ascending = e.begin >= end;
    end = e.end;
  }
  if (ascending) return INTLORA_OK;
  std::unique_ptr<Extent[]> all(new (std::nothrow) Extent[static_cast<size_t>(count)]);
  if (!all) return fail(INTLORA_ERR_UNSUPPORTED, "out of host memory for %d gradient jobs", count);
  int32_t n = 0;
  for (int32_t k = 0; k < count; ++k)
    if (jobs[k].count > 0) all[n++] = extent_of(jobs, k);
  std::sort(all.get(), all.get() + n, [](const Extent& a, const Extent& b) { return a.begin < b.begin; });
  for (int32_t k = 1; k < n; ++k)
    if (all[k].begin < all[k - 1].end)
      return fail(INTLORA_ERR_INVALID_ARG, "gradient jobs %d and %d overlap", std::min(all[k - 1].job, all[k].job),
                  std::max(all[k - 1].job, all[k].job));
  return INTLORA_OK;
}

size_t partial_bytes(int64_t partials) { return (static_cast<size_t>(partials) * sizeof(double) + 255) / 256 * 256; }

intlora_status check_max_norm(float max_norm) {
  if (!(max_norm >= 0.0f) || !std::isfinite(max_norm))
    return fail(INTLORA_ERR_INVALID_ARG, "max_norm must be finite and >= 0");
  return INTLORA_OK;
}

intlora_status check_norm(const float* norm) {
  if (norm == nullptr || !aligned4(norm))
    return fail(INTLORA_ERR_INVALID_ARG, "norm is required, aligned to 4 bytes");
  return INTLORA_OK;
}

}  // namespace

extern "C" {

intlora_status intlora_layer_norm_batched(const intlora_layer_norm_job* jobs, int32_t count, void* stream) {
  intlora_status s = check_list(jobs, count);
  for (int32_t k = 0; s == INTLORA_OK && k < count; ++k) s = check_ln(jobs[k], k);
  if (s != INTLORA_OK) return s;
  for (int32_t k = 0; k < count; ++k) {
    const intlora_layer_norm_job& j = jobs[k];
    if (j.tokens == 0) continue;
    const cudaError_t e = launch_layer_norm(
        LayerNormJob{j.x, j.weight, j.bias, j.y, j.mean, j.rstd, j.tokens, j.n, j.ld_x, j.ld_y, j.x_type, j.param_type,
                     j.y_type, j.eps},
        static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "layer norm launch");
  }
  return INTLORA_OK;
}

size_t intlora_layer_norm_backward_workspace_size(const intlora_layer_norm_backward_job* jobs, int32_t count) {
  size_t total = 0;
  for (int32_t k = 0; k < count && jobs != nullptr; ++k)
    if (lnb_sums(jobs[k]) && check_lnb(jobs[k], k) == INTLORA_OK)
      total += layer_norm_backward_ws(jobs[k].tokens, jobs[k].n);
  return total;
}

intlora_status intlora_layer_norm_backward_batched(const intlora_layer_norm_backward_job* jobs, int32_t count, void* ws,
                                                   size_t ws_bytes, void* stream) {
  intlora_status s = check_list(jobs, count);
  for (int32_t k = 0; s == INTLORA_OK && k < count; ++k) s = check_lnb(jobs[k], k);
  if (s != INTLORA_OK) return s;
  if ((s = check_ws(ws, ws_bytes, intlora_layer_norm_backward_workspace_size(jobs, count))) != INTLORA_OK) return s;
  char* w = static_cast<char*>(ws);
  for (int32_t k = 0; k < count; ++k) {
    const intlora_layer_norm_backward_job& j = jobs[k];
    const cudaError_t e = launch_layer_norm_backward(
        LayerNormBackwardJob{j.dy, j.x, j.weight, j.mean, j.rstd, j.dx, j.dweight, j.dbias, j.tokens, j.n, j.ld_dy,
                             j.ld_x, j.ld_dx, j.dy_type, j.x_type, j.param_type, j.dx_type, j.accumulate != 0},
        w, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "layer norm backward launch");
    if (lnb_sums(j)) w += layer_norm_backward_ws(j.tokens, j.n);
  }
  return INTLORA_OK;
}

intlora_status intlora_embedding_batched(const intlora_embedding_job* jobs, int32_t count, void* stream) {
  intlora_status s = check_list(jobs, count);
  for (int32_t k = 0; s == INTLORA_OK && k < count; ++k) s = check_emb(jobs[k], k);
  if (s != INTLORA_OK) return s;
  for (int32_t k = 0; k < count; ++k) {
    const intlora_embedding_job& j = jobs[k];
    if (j.tokens == 0) continue;
    const cudaError_t e = launch_embedding(
        EmbeddingJob{j.table, j.ids, j.y, j.invalid, j.vocab, j.n, j.tokens, j.ld_table, j.ld_y, j.table_type,
                     j.y_type, j.id_bytes, j.scale},
        static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "embedding launch");
  }
  return INTLORA_OK;
}

size_t intlora_embedding_backward_workspace_size(const intlora_embedding_backward_job* jobs, int32_t count) {
  size_t total = 0;
  for (int32_t k = 0; k < count && jobs != nullptr; ++k)
    if (check_embb(jobs[k], k) == INTLORA_OK) total += embedding_backward_ws(jobs[k].tokens, jobs[k].n);
  return total;
}

intlora_status intlora_embedding_backward_batched(const intlora_embedding_backward_job* jobs, int32_t count, void* ws,
                                                  size_t ws_bytes, void* stream) {
  intlora_status s = check_list(jobs, count);
  for (int32_t k = 0; s == INTLORA_OK && k < count; ++k) s = check_embb(jobs[k], k);
  if (s != INTLORA_OK) return s;
  if ((s = check_ws(ws, ws_bytes, intlora_embedding_backward_workspace_size(jobs, count))) != INTLORA_OK) return s;
  char* w = static_cast<char*>(ws);
  for (int32_t k = 0; k < count; ++k) {
    const intlora_embedding_backward_job& j = jobs[k];
    const cudaError_t e = launch_embedding_backward(
        EmbeddingBackwardJob{j.dy, j.ids, j.dtable, j.invalid, j.vocab, j.n, j.tokens, j.padding_id, j.ld_dy,
                             j.ld_dtable, j.dy_type, j.dtable_type, j.id_bytes, j.accumulate != 0, j.scale},
        w, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "embedding backward launch");
    w += embedding_backward_ws(j.tokens, j.n);
  }
  return INTLORA_OK;
}

size_t intlora_grad_norm_workspace_size(const intlora_grad_job* jobs, int32_t count) {
  if (jobs == nullptr || count <= 0 || check_grads(jobs, count) != INTLORA_OK) return 0;
  return partial_bytes(grad_norm_partials(jobs, count));
}

intlora_status intlora_grad_norm_batched(const intlora_grad_job* jobs, int32_t count, float* norm, void* ws,
                                         size_t ws_bytes, void* stream) {
  intlora_status s = check_grads(jobs, count);
  if (s != INTLORA_OK || (s = check_norm(norm)) != INTLORA_OK) return s;
  const int64_t partials = grad_norm_partials(jobs, count);
  if ((s = check_ws(ws, ws_bytes, partial_bytes(partials))) != INTLORA_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_grad_squares(jobs, count, ws, st);
  if (e == cudaSuccess) e = launch_grad_norm_finish(partials, ws, norm, st);
  return e == cudaSuccess ? INTLORA_OK : cuda_fail(e, "gradient norm launch");
}

intlora_status intlora_grad_clip_batched(const intlora_grad_job* jobs, int32_t count, float max_norm, const float* norm,
                                         void* stream) {
  intlora_status s = check_grads(jobs, count);
  if (s != INTLORA_OK || (s = check_max_norm(max_norm)) != INTLORA_OK || (s = check_norm(norm)) != INTLORA_OK ||
      (s = check_disjoint(jobs, count)) != INTLORA_OK)
    return s;
  const cudaError_t e = launch_grad_clip(jobs, count, max_norm, nullptr, 0, const_cast<float*>(norm),
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? INTLORA_OK : cuda_fail(e, "gradient clipping launch");
}

intlora_status intlora_clip_grad_norm_batched(const intlora_grad_job* jobs, int32_t count, float max_norm, float* norm,
                                              void* ws, size_t ws_bytes, void* stream) {
  intlora_status s = check_grads(jobs, count);
  if (s != INTLORA_OK || (s = check_max_norm(max_norm)) != INTLORA_OK || (s = check_norm(norm)) != INTLORA_OK ||
      (s = check_disjoint(jobs, count)) != INTLORA_OK)
    return s;
  const int64_t partials = grad_norm_partials(jobs, count);
  if ((s = check_ws(ws, ws_bytes, partial_bytes(partials))) != INTLORA_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = count == 0 ? launch_grad_norm_finish(0, ws, norm, st)
                                   : launch_clip_grad_norm(jobs, count, max_norm, ws, partials, norm, st);
  return e == cudaSuccess ? INTLORA_OK : cuda_fail(e, "gradient clipping launch");
}

}  // extern "C"
