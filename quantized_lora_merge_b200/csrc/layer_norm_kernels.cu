// Layer norm over the rows of a tokens x n activation, and its gradients.
//
//   forward   m = mean_j x_j, v = mean_j (x_j - m)^2, rstd = (v + eps)^-1/2,
//             y_j = (x_j - m) rstd w_j + b_j
//   backward  xh_j = (x_j - m) rstd, g_j = dy_j w_j,
//             dx_j = rstd (g_j - mean g - xh_j mean(g xh)),
//             dw_j = sum_t dy_tj xh_tj, db_j = sum_t dy_tj
//
// Both are bound by memory: 8 and 14 operations an element against 4 to 12
// bytes. Every row is read once and stays in registers: T threads share a
// row, thread t holding V chunks of 8 elements (elem.cuh), so the mean and the
// centred squares are summed from registers (two passes over the values, one
// over memory). Rows of up to 32 threads' slices live inside one warp and never
// wait for the rest of the block; wider rows take a whole block each.
// Statistics, sums and products are fp32; y and dx are rounded once.
#include <algorithm>

#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "intlora_kernels.h"
#include "train_ops.h"

namespace intlora {

namespace {

constexpr int kSms = 148;
constexpr int kRowBlock = 256;                 // threads of a block whose rows are inside warps
constexpr int kFwdMaxV = 5, kBwdMaxV = 5;
constexpr int kFwdMaxT = 1024, kBwdMaxT = 512;
constexpr int kBwdBlockMaxV = 2;               // accumulators and both rows within 128 registers
constexpr int kWideThreads = 1024;
constexpr int kColThreads = 256;               // column sums of wide rows: columns per block
constexpr int kReduceWarps = 16;

// Sums over the T threads of a row. Inside a warp: T a power of two up to 32.
template <bool BLOCK, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int T, float* scratch) {
  const int w = BLOCK ? 32 : T;
#pragma unroll
  for (int i = 0; i < N; ++i)
    for (int o = w >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (BLOCK) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) scratch[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = lane < warps ? scratch[i * 32 + lane] : 0.0f;
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[i] = s;
    }
  }
}

template <int V, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kFwdMaxT : kRowBlock)
    layer_norm_kernel(const __grid_constant__ LayerNormJob j, int T) {
  __shared__ float scratch[2][32];             // one per sum: no wait between a row's reads and the next writes
  const int t = BLOCK ? threadIdx.x : threadIdx.x % T;
  const int group = BLOCK ? 0 : threadIdx.x / T;
  const int groups = BLOCK ? 1 : blockDim.x / T;
  const int n = static_cast<int>(j.n);
  const float inv_n = 1.0f / static_cast<float>(n);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < j.tokens;
       base += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t row = base + group;
    const bool live = row < j.tokens;          // the whole warp walks on: the sums below are warp-wide
    RawSlice<V> raw;
    load_slice<V, VEC>(raw, row_ptr(j.x, live ? row : base, j.ld_x, j.x_type), j.x_type, n, t, T);
    float x[8 * V];
#pragma unroll
    for (int k = 0; k < V; ++k) slice_chunk<V, VEC>(raw, j.x_type, k, x + 8 * k);
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < 8 * V; ++i) s[0] += x[i];
    row_sum<BLOCK, 1>(s, T, scratch[0]);
    const float mean = s[0] * inv_n;
    s[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& v = x[8 * k + e];
        v = slice_col<VEC>(k, e, t, T) < n ? v - mean : 0.0f;
        s[0] = fmaf(v, v, s[0]);
      }
    row_sum<BLOCK, 1>(s, T, scratch[1]);
    const float rstd = 1.0f / sqrtf(s[0] * inv_n + j.eps);
    if (!live) continue;
    if (t == 0) {
      if (j.mean != nullptr) j.mean[row] = mean;
      if (j.rstd != nullptr) j.rstd[row] = rstd;
    }
    void* y = row_ptr(j.y, row, j.ld_y, j.y_type);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float o[8], p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = x[8 * k + e] * rstd;
      if (VEC) {
        const int c = slice_col<VEC>(k, 0, t, T);
        if (c >= n) continue;
        if (j.weight != nullptr) {
          load8(j.weight, c, j.param_type, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] *= p[e];
        }
        if (j.bias != nullptr) {
          load8(j.bias, c, j.param_type, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += p[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = slice_col<VEC>(k, e, t, T);
          if (c >= n) continue;
          if (j.weight != nullptr) o[e] *= load_elem(j.weight, c, j.param_type);
          if (j.bias != nullptr) o[e] += load_elem(j.bias, c, j.param_type);
        }
      }
      store_chunk<VEC>(y, j.y_type, n, t, T, k, o);
    }
  }
}

// Rows too wide for registers: a block per row, three walks over it (the later
// ones served by L1 and L2).
__global__ void __launch_bounds__(kWideThreads) layer_norm_wide_kernel(const __grid_constant__ LayerNormJob j) {
  __shared__ float scratch[2][32];
  for (int64_t row = blockIdx.x; row < j.tokens; row += gridDim.x) {
    const void* x = row_ptr(j.x, row, j.ld_x, j.x_type);
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) s[0] += load_elem(x, c, j.x_type);
    row_sum<true, 1>(s, 0, scratch[0]);
    const float mean = s[0] / static_cast<float>(j.n);
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float v = load_elem(x, c, j.x_type) - mean;
      s[0] = fmaf(v, v, s[0]);
    }
    row_sum<true, 1>(s, 0, scratch[1]);
    const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(j.n) + j.eps);
    if (threadIdx.x == 0) {
      if (j.mean != nullptr) j.mean[row] = mean;
      if (j.rstd != nullptr) j.rstd[row] = rstd;
    }
    void* y = row_ptr(j.y, row, j.ld_y, j.y_type);
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      float o = (load_elem(x, c, j.x_type) - mean) * rstd;
      if (j.weight != nullptr) o *= load_elem(j.weight, c, j.param_type);
      if (j.bias != nullptr) o += load_elem(j.bias, c, j.param_type);
      store_elem(y, c, j.y_type, o);
    }
  }
}

// Backward: a block walks over rows with a grid stride; every thread keeps the
// sums of its columns of dy xh and dy in registers over all its rows, and the
// block writes them once, as row blockIdx.x of partial ([blocks][2][n]).
template <int V, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kBwdMaxT : kRowBlock)
    layer_norm_backward_kernel(const __grid_constant__ LayerNormBackwardJob j, int T, float* partial) {
  __shared__ float scratch[2][2 * 32];
  __shared__ __align__(16) float cols[BLOCK ? 1 : 2 * 32 * 8 * V];
  const int t = BLOCK ? threadIdx.x : threadIdx.x % T;
  const int group = BLOCK ? 0 : threadIdx.x / T;
  const int groups = BLOCK ? 1 : blockDim.x / T;
  const int n = static_cast<int>(j.n);
  const float inv_n = 1.0f / static_cast<float>(n);
  float w[8 * V], dw[8 * V], db[8 * V];
  {
    RawSlice<V> raw;
    if (j.weight != nullptr) load_slice<V, VEC>(raw, j.weight, j.param_type, n, t, T);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (j.weight != nullptr) {
        slice_chunk<V, VEC>(raw, j.param_type, k, w + 8 * k);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * k + e] = 1.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[8 * k + e] = db[8 * k + e] = 0.0f;
    }
  }
  int flip = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < j.tokens;
       base += static_cast<int64_t>(gridDim.x) * groups) {
    const bool live = base + group < j.tokens;
    const int64_t row = live ? base + group : base;
    RawSlice<V> rx, rdy;
    load_slice<V, VEC>(rx, row_ptr(j.x, row, j.ld_x, j.x_type), j.x_type, n, t, T);
    load_slice<V, VEC>(rdy, row_ptr(j.dy, row, j.ld_dy, j.dy_type), j.dy_type, n, t, T);
    const float mean = j.mean[row], rstd = j.rstd[row];
    float xh[8 * V], dy[8 * V], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < V; ++k) {
      slice_chunk<V, VEC>(rx, j.x_type, k, xh + 8 * k);
      slice_chunk<V, VEC>(rdy, j.dy_type, k, dy + 8 * k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 8 * k + e;
        // columns past n hold dy = 0 and take no part in any sum
        xh[i] = slice_col<VEC>(k, e, t, T) < n ? (xh[i] - mean) * rstd : 0.0f;
        const float g = dy[i] * w[i];
        s[0] += g;
        s[1] = fmaf(g, xh[i], s[1]);
        if (live) {
          dw[i] = fmaf(dy[i], xh[i], dw[i]);
          db[i] += dy[i];
        }
      }
    }
    if (j.dx == nullptr) continue;             // uniform over the grid
    row_sum<BLOCK, 2>(s, T, scratch[flip]);
    flip ^= 1;
    if (!live) continue;
    const float c1 = s[0] * inv_n, c2 = s[1] * inv_n;
    void* dx = row_ptr(j.dx, row, j.ld_dx, j.dx_type);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 8 * k + e;
        o[e] = rstd * (fmaf(dy[i], w[i], -c1) - xh[i] * c2);
      }
      store_chunk<VEC>(dx, j.dx_type, n, t, T, k, o);
    }
  }
  if (partial == nullptr) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * n;
  if (BLOCK) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      store_chunk<VEC>(out, kF32, n, t, T, k, dw + 8 * k);
      store_chunk<VEC>(out + n, kF32, n, t, T, k, db + 8 * k);
    }
  } else {
    // groups of one warp, then the warps in turn: a fixed order
#pragma unroll
    for (int i = 0; i < 8 * V; ++i)
      for (int o = T; o < 32; o <<= 1) {
        dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
        db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
      }
    float* cw = cols;
    float* cb = cols + 32 * 8 * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int turn = 0; turn < static_cast<int>(blockDim.x >> 5); ++turn) {
      if (warp == turn && lane < T) {
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) {
          const int at = i * T + lane;
          cw[at] = (turn == 0 ? 0.0f : cw[at]) + dw[i];
          cb[at] = (turn == 0 ? 0.0f : cb[at]) + db[i];
        }
      }
      __syncthreads();
    }
    for (int at = threadIdx.x; at < T * 8 * V; at += blockDim.x) {
      const int i = at / T, tt = at % T;
      const int c = slice_col<VEC>(i >> 3, i & 7, tt, T);
      if (c < n) {
        out[c] = cw[at];
        out[n + c] = cb[at];
      }
    }
  }
}

// dx of rows too wide for registers.
__global__ void __launch_bounds__(kWideThreads)
    layer_norm_backward_wide_kernel(const __grid_constant__ LayerNormBackwardJob j) {
  __shared__ float scratch[2][2 * 32];
  int flip = 0;
  for (int64_t row = blockIdx.x; row < j.tokens; row += gridDim.x) {
    const void* x = row_ptr(j.x, row, j.ld_x, j.x_type);
    const void* dy = row_ptr(j.dy, row, j.ld_dy, j.dy_type);
    const float mean = j.mean[row], rstd = j.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float w = j.weight != nullptr ? load_elem(j.weight, c, j.param_type) : 1.0f;
      const float g = load_elem(dy, c, j.dy_type) * w;
      s[0] += g;
      s[1] = fmaf(g, (load_elem(x, c, j.x_type) - mean) * rstd, s[1]);
    }
    row_sum<true, 2>(s, 0, scratch[flip]);
    flip ^= 1;
    const float c1 = s[0] / static_cast<float>(j.n), c2 = s[1] / static_cast<float>(j.n);
    void* dx = row_ptr(j.dx, row, j.ld_dx, j.dx_type);
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float w = j.weight != nullptr ? load_elem(j.weight, c, j.param_type) : 1.0f;
      const float xh = (load_elem(x, c, j.x_type) - mean) * rstd;
      store_elem(dx, c, j.dx_type, rstd * (fmaf(load_elem(dy, c, j.dy_type), w, -c1) - xh * c2));
    }
  }
}

// Column sums of dy xh and dy for wide rows: a thread owns a column over the
// rows of its split.
__global__ void __launch_bounds__(kColThreads)
    layer_norm_columns_kernel(const __grid_constant__ LayerNormBackwardJob j, float* partial) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (c >= j.n) return;
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < j.tokens; row += gridDim.y) {
    const float dy = load_elem(row_ptr(j.dy, row, j.ld_dy, j.dy_type), c, j.dy_type);
    const float x = load_elem(row_ptr(j.x, row, j.ld_x, j.x_type), c, j.x_type);
    dw = fmaf(dy, (x - j.mean[row]) * j.rstd[row], dw);
    db += dy;
  }
  float* out = partial + static_cast<int64_t>(blockIdx.y) * 2 * j.n;
  out[c] = dw;
  out[j.n + c] = db;
}

// dweight and dbias from the blocks' partial sums, added in block order.
__global__ void __launch_bounds__(32 * kReduceWarps)
    layer_norm_reduce_kernel(const float* partial, int64_t blocks, int64_t n, float* dweight, float* dbias,
                             int accumulate) {
  __shared__ float part[kReduceWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < 2 * n) {
#pragma unroll 8
    for (int64_t p = warp; p < blocks; p += kReduceWarps) s += partial[p * 2 * n + c];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= 2 * n) return;
  s = part[0][lane];
#pragma unroll
  for (int k = 1; k < kReduceWarps; ++k) s += part[k][lane];
  float* out = c < n ? dweight : dbias;
  if (out == nullptr) return;
  const int64_t at = c < n ? c : c - n;
  out[at] = accumulate ? out[at] + s : s;
}

bool row_aligned(const void* p, int64_t ld, int type) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elem_bytes(type)) % 16 == 0;
}

// Threads T and chunks V of a row of n columns: the least idle slots first,
// then the most chunks a thread (fewer threads to join) up to max_v; T a power
// of two inside a warp, else whole warps. False: the row does not fit.
bool row_shape(int64_t n, int min_v, int max_v, int block_max_v, int max_t, int* T_out, int* V_out) {
  const int64_t chunks = (n + 7) / 8;
  int64_t best = INT64_MAX;
  for (int v = min_v; v <= max_v; ++v) {
    int64_t t = 1;
    while (t < 32 && t * v < chunks) t *= 2;
    if (t * v < chunks) {
      if (v > block_max_v) continue;
      t = ((chunks + v - 1) / v + 31) / 32 * 32;
      if (t > max_t) continue;
    }
    if (t * v <= best) {
      best = t * v;
      *T_out = static_cast<int>(t);
      *V_out = v;
    }
  }
  return best != INT64_MAX;
}

unsigned grid_of(int64_t blocks, int64_t cap) { return static_cast<unsigned>(std::max<int64_t>(1, std::min(blocks, cap))); }

}  // namespace

cudaError_t launch_layer_norm(const LayerNormJob& j, cudaStream_t s) {
  const bool vec = j.n % 8 == 0 && row_aligned(j.x, j.ld_x, j.x_type) && row_aligned(j.y, j.ld_y, j.y_type) &&
                   (reinterpret_cast<uintptr_t>(j.weight) & 15u) == 0 && (reinterpret_cast<uintptr_t>(j.bias) & 15u) == 0;
  int T = 0, V = 0;
  // Few rows: the narrowest slices, so that a row's time is one load deep.
  const int max_v = j.tokens <= kSms ? 1 : kFwdMaxV;
  if (!row_shape(j.n, 1, max_v, max_v, kFwdMaxT, &T, &V) && !row_shape(j.n, 1, kFwdMaxV, 4, kFwdMaxT, &T, &V)) {
    layer_norm_wide_kernel<<<grid_of(j.tokens, 1 << 20), kWideThreads, 0, s>>>(j);
    return counted(cudaGetLastError());
  }
  const bool block = T > 32;
  const int threads = block ? T : kRowBlock;
  const unsigned grid = grid_of((j.tokens + (block ? 0 : kRowBlock / T - 1)) / (block ? 1 : kRowBlock / T), int64_t{1} << 30);
#define LN_LAUNCH(v)                                                                                       \
  case v:                                                                                                  \
    if (vec && block) layer_norm_kernel<v, true, true><<<grid, threads, 0, s>>>(j, T);                     \
    else if (vec) layer_norm_kernel<v, true, false><<<grid, threads, 0, s>>>(j, T);                        \
    else if (block) layer_norm_kernel<v, false, true><<<grid, threads, 0, s>>>(j, T);                      \
    else layer_norm_kernel<v, false, false><<<grid, threads, 0, s>>>(j, T);                                \
    break;
  switch (V) {
    LN_LAUNCH(1)
    LN_LAUNCH(2)
    LN_LAUNCH(3)
    LN_LAUNCH(4)
    LN_LAUNCH(5)
  }
#undef LN_LAUNCH
  return counted(cudaGetLastError());
}

namespace {
// Blocks of the backward kernel, which is also the number of partial sums.
struct BackwardShape {
  int T = 0, V = 0;
  bool wide = false;
  int64_t blocks = 0;
};
BackwardShape backward_shape(int64_t tokens, int64_t n) {
  BackwardShape b;
  if (!row_shape(n, 1, kBwdMaxV, kBwdBlockMaxV, kBwdMaxT, &b.T, &b.V)) {
    b.wide = true;
    const int64_t strips = (n + kColThreads - 1) / kColThreads;
    b.blocks = std::min<int64_t>(std::max<int64_t>(1, kSms * 8 / strips), std::max<int64_t>(1, tokens / 8));
    return b;
  }
  const int64_t per = b.T > 32 ? 1 : kRowBlock / b.T;
  b.blocks = std::max<int64_t>(1, std::min<int64_t>(kSms * 2, (tokens + per - 1) / per));
  return b;
}
}  // namespace

size_t layer_norm_backward_ws(int64_t tokens, int64_t n) {
  const BackwardShape b = backward_shape(tokens, n);
  return (static_cast<size_t>(b.blocks) * 2 * static_cast<size_t>(n) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardJob& j, void* ws, cudaStream_t s) {
  const BackwardShape b = backward_shape(j.tokens, j.n);
  const bool sums = j.dweight != nullptr || j.dbias != nullptr;
  float* partial = sums ? static_cast<float*>(ws) : nullptr;
  if (b.wide) {
    if (j.dx != nullptr && j.tokens > 0) {
      layer_norm_backward_wide_kernel<<<grid_of(j.tokens, 1 << 20), kWideThreads, 0, s>>>(j);
      const cudaError_t e = counted(cudaGetLastError());
      if (e != cudaSuccess) return e;
    }
    if (sums) {
      const dim3 grid(static_cast<unsigned>((j.n + kColThreads - 1) / kColThreads), static_cast<unsigned>(b.blocks));
      layer_norm_columns_kernel<<<grid, kColThreads, 0, s>>>(j, partial);
      const cudaError_t e = counted(cudaGetLastError());
      if (e != cudaSuccess) return e;
    }
  } else {
    const bool vec = j.n % 8 == 0 && row_aligned(j.x, j.ld_x, j.x_type) && row_aligned(j.dy, j.ld_dy, j.dy_type) &&
                     (j.dx == nullptr || row_aligned(j.dx, j.ld_dx, j.dx_type)) &&
                     (reinterpret_cast<uintptr_t>(j.weight) & 15u) == 0;
    const bool block = b.T > 32;
    const int threads = block ? b.T : kRowBlock;
    const unsigned grid = static_cast<unsigned>(b.blocks);
#define LN_LAUNCH(v)                                                                                             \
  case v:                                                                                                        \
    if (vec) layer_norm_backward_kernel<v, true, false><<<grid, threads, 0, s>>>(j, b.T, partial);               \
    else layer_norm_backward_kernel<v, false, false><<<grid, threads, 0, s>>>(j, b.T, partial);                  \
    break;
#define LN_LAUNCH_BLOCK(v)                                                                                       \
  case v:                                                                                                        \
    if (vec) layer_norm_backward_kernel<v, true, true><<<grid, threads, 0, s>>>(j, b.T, partial);                \
    else layer_norm_backward_kernel<v, false, true><<<grid, threads, 0, s>>>(j, b.T, partial);                   \
    break;
    if (block) {
      switch (b.V) {
        LN_LAUNCH_BLOCK(1)
        LN_LAUNCH_BLOCK(2)
      }
    } else {
      switch (b.V) {
        LN_LAUNCH(1)
        LN_LAUNCH(2)
        LN_LAUNCH(3)
        LN_LAUNCH(4)
        LN_LAUNCH(5)
      }
    }
#undef LN_LAUNCH
#undef LN_LAUNCH_BLOCK
    const cudaError_t e = counted(cudaGetLastError());
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  layer_norm_reduce_kernel<<<static_cast<unsigned>((2 * j.n + 31) / 32), 32 * kReduceWarps, 0, s>>>(
      partial, b.blocks, j.n, j.dweight, j.dbias, j.accumulate);
  return counted(cudaGetLastError());
}

}  // namespace intlora
