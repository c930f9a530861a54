// Launchers of the operators around the adapted linears in a training step:
// layer norm, embedding, gradient norm and clipping. The C ABI
// (train_ops_api.cu) validates the public descriptors and calls these.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "intlora.h"

namespace intlora {

// Layer norm (layer_norm_kernels.cu).
struct LayerNormJob {
  const void* x;
  const void* weight;        // may be nullptr: 1
  const void* bias;          // may be nullptr: 0
  void* y;
  float* mean;               // may be nullptr
  float* rstd;               // may be nullptr
  int64_t tokens, n;
  int64_t ld_x, ld_y;        // elements between rows
  int32_t x_type, param_type, y_type;
  float eps;
};
struct LayerNormBackwardJob {
  const void* dy;
  const void* x;
  const void* weight;        // may be nullptr
  const float* mean;
  const float* rstd;
  void* dx;                  // may be nullptr
  float* dweight;            // may be nullptr
  float* dbias;              // may be nullptr
  int64_t tokens, n;
  int64_t ld_dy, ld_x, ld_dx;
  int32_t dy_type, x_type, param_type, dx_type;
  int32_t accumulate;
};
cudaError_t launch_layer_norm(const LayerNormJob& j, cudaStream_t s);
size_t layer_norm_backward_ws(int64_t tokens, int64_t n);
cudaError_t launch_layer_norm_backward(const LayerNormBackwardJob& j, void* ws, cudaStream_t s);

// Embedding (embedding_kernels.cu).
struct EmbeddingJob {
  const void* table;
  const void* ids;
  void* y;
  int32_t* invalid;          // may be nullptr
  int64_t vocab, n, tokens;
  int64_t ld_table, ld_y;
  int32_t table_type, y_type, id_bytes;
  float scale;
};
struct EmbeddingBackwardJob {
  const void* dy;
  const void* ids;
  void* dtable;
  int32_t* invalid;          // may be nullptr
  int64_t vocab, n, tokens, padding_id;
  int64_t ld_dy, ld_dtable;
  int32_t dy_type, dtable_type, id_bytes, accumulate;
  float scale;
};
cudaError_t launch_embedding(const EmbeddingJob& j, cudaStream_t s);
size_t embedding_backward_ws(int64_t tokens, int64_t n);
cudaError_t launch_embedding_backward(const EmbeddingBackwardJob& j, void* ws, cudaStream_t s);

// Gradient norm and clipping (grad_norm_kernels.cu).
// Partial sums, of 8 bytes each in ws.
int64_t grad_norm_partials(const intlora_grad_job* jobs, int32_t count);
// Sum of squares over all tensors, as partial sums in ws.
cudaError_t launch_grad_squares(const intlora_grad_job* jobs, int32_t count, void* ws, cudaStream_t s);
// *norm = root of the partial sums' total.
cudaError_t launch_grad_norm_finish(int64_t partials, const void* ws, float* norm, cudaStream_t s);
// g *= min(1, max_norm / (norm + 1e-6)). ws not nullptr: the norm comes from
// the partial sums and is written to *norm; else it is read from *norm.
cudaError_t launch_grad_clip(const intlora_grad_job* jobs, int32_t count, float max_norm, const void* ws,
                             int64_t partials, float* norm, cudaStream_t s);
// launch_grad_squares and launch_grad_clip; count >= 1.
cudaError_t launch_clip_grad_norm(const intlora_grad_job* jobs, int32_t count, float max_norm, void* ws,
                                  int64_t partials, float* norm, cudaStream_t s);

}  // namespace intlora
