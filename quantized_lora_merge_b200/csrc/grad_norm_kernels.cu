// Global norm over the gradients of many tensors, and clipping in place.
//
//   norm = sqrt(sum over all tensors of g^2),   g <- g min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: one read for the norm and one read and write for the
// clipping, which needs the whole norm first. The tensors are cut into chunks
// of kChunk elements (a chunk never spans two tensors), and every block owns a
// contiguous stretch of chunks, walked forwards for the norm and backwards for
// the clipping, so that what was read last, and is still in L2, is used first.
// Each block leaves one fp64 partial sum, and every reader adds the partial
// sums in the same order: the norm has the same bits on every run.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "intlora.h"
#include "intlora_kernels.h"
#include "train_ops.h"

namespace intlora {

namespace {

constexpr int kSms = 148;
constexpr int kThreads = 256;
constexpr int kPerThread = 32;                 // elements of a chunk a thread holds
constexpr int64_t kChunk = kThreads * kPerThread;
constexpr int kMaxBlocks = kSms * 4;
constexpr int kMaxSpans = 512, kMidSpans = 256, kFewSpans = 64;   // tensors per launch

// Tensors of one launch, by value: no table in device memory. 14 bytes each, since
// a launch copies them: what a chunk needs beside its tensor's first element is
// the length of the last chunk and the type.
template <int N>
struct Spans {
  void* g[N];
  uint32_t begin[N + 1];                       // first chunk of each tensor
  uint16_t last[N];                            // (elements of the last chunk - 1) | type << 14
  int32_t spans;
  uint32_t chunks;
};
static_assert(kChunk <= (1 << 14), "a chunk's length fits beside the type");

// Sum of squares of a thread's values. Squares of fp32 and bf16 values above
// 2^64 or below 2^-63 leave the range of fp32, so a sum that is not well inside
// it is formed again in fp64; where it is inside, what underflow drops is below
// 2^-30 of it.
__device__ __forceinline__ double square_sum(const float (&v)[kPerThread]) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
  const float f = (s[0] + s[1]) + (s[2] + s[3]);
  if (f > 0x1p-90f && f < 0x1p126f) return f;
  if (f == 0.0f) {                             // nothing but zeros (a factor's first step), or squares too small
    uint32_t any = 0u;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) any |= __float_as_uint(v[i]) << 1;
    if (any == 0u) return 0.0;
  }
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) d = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), d);
  return d;
}

// A thread's part of a chunk of a tensor: 4 groups of 8 elements where the
// tensor starts at a multiple of 8 elements, else single elements.
struct Piece {
  void* g;
  int64_t first;                               // element of the chunk's begin
  int len;                                     // elements of the chunk
  int type;
  bool vec;
};
template <int N>
__device__ __forceinline__ Piece piece_of(const Spans<N>& b, int span, uint32_t chunk) {
  Piece p;
  p.g = b.g[span];
  p.first = static_cast<int64_t>(chunk - b.begin[span]) * kChunk;
  p.len = chunk + 1 < b.begin[span + 1] ? static_cast<int>(kChunk) : (b.last[span] & 0x3fff) + 1;
  p.type = b.last[span] >> 14;
  p.vec = reinterpret_cast<uintptr_t>(p.g) % (8 * elem_bytes(p.type)) == 0;
  return p;
}
__device__ __forceinline__ void load_piece(const Piece& p, float (&v)[kPerThread]) {
  if (p.vec && p.len == kChunk) {
#pragma unroll
    for (int k = 0; k < kPerThread / 8; ++k)
      load8(p.g, p.first + (k * kThreads + static_cast<int>(threadIdx.x)) * 8, p.type, v + 8 * k);
  } else {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int at = i * kThreads + static_cast<int>(threadIdx.x);
      v[i] = at < p.len ? load_elem(p.g, p.first + at, p.type) : 0.0f;
    }
  }
}
__device__ __forceinline__ void store_piece(const Piece& p, const float (&v)[kPerThread]) {
  if (p.vec && p.len == kChunk) {
#pragma unroll
    for (int k = 0; k < kPerThread / 8; ++k)
      store8(p.g, p.first + (k * kThreads + static_cast<int>(threadIdx.x)) * 8, p.type, v + 8 * k);
  } else {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int at = i * kThreads + static_cast<int>(threadIdx.x);
      if (at < p.len) store_elem(p.g, p.first + at, p.type, v[i]);
    }
  }
}

// Tensor of a chunk.
template <int N>
__device__ __forceinline__ int span_of(const Spans<N>& b, uint32_t chunk) {
  int lo = 0, hi = b.spans - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.begin[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ uint32_t stretch(uint32_t chunks, uint32_t block) {
  return static_cast<uint32_t>(static_cast<uint64_t>(chunks) * block / gridDim.x);
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int k = 1; k < kThreads / 32; ++k) v += part[k];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ Spans<N> b, double* partial) {
  const uint32_t end = stretch(b.chunks, blockIdx.x + 1);
  uint32_t chunk = stretch(b.chunks, blockIdx.x);
  int span = chunk < end ? span_of(b, chunk) : 0;
  double sum = 0.0;
  for (; chunk < end; ++chunk) {
    while (chunk >= b.begin[span + 1]) ++span;
    float v[kPerThread];
    load_piece(piece_of(b, span, chunk), v);
    sum += square_sum(v);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from all partial sums, the same in every block.
__device__ __forceinline__ float total_norm(const double* partial, int64_t count) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) s += partial[i];
  return static_cast<float>(sqrt(block_sum(s)));
}

__global__ void __launch_bounds__(kThreads) grad_norm_finish_kernel(const double* partial, int64_t count, float* norm) {
  wait_for_previous();
  const float v = total_norm(partial, count);
  if (threadIdx.x == 0) *norm = v;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_clip_kernel(const __grid_constant__ Spans<N> b, const double* partial, int64_t partials, float max_norm,
                     float* norm, int write_norm) {
  float v_norm;
  wait_for_previous();
  if (partial != nullptr) {
    v_norm = total_norm(partial, partials);
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v_norm;
  } else {
    v_norm = *norm;
  }
  // a NaN norm gives a NaN factor, an infinite one the factor 0
  const float scale = static_cast<float>(static_cast<double>(max_norm) / (static_cast<double>(v_norm) + 1e-6));
  if (scale >= 1.0f) return;
  const uint32_t begin = stretch(b.chunks, blockIdx.x);
  uint32_t chunk = stretch(b.chunks, blockIdx.x + 1);
  if (chunk == begin) return;
  int span = span_of(b, chunk - 1);
  while (chunk-- > begin) {
    while (chunk < b.begin[span]) --span;
    const Piece p = piece_of(b, span, chunk);
    float v[kPerThread];
    load_piece(p, v);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) v[i] *= scale;
    store_piece(p, v);
  }
}

int64_t blocks_of(int64_t chunks) { return std::max<int64_t>(1, std::min<int64_t>(chunks, kMaxBlocks)); }

// Fills one launch from jobs[k0 ..), tensors without elements left out;
// returns the index of the first job not taken.
template <int N>
int32_t fill(const intlora_grad_job* jobs, int32_t k0, int32_t count, Spans<N>* b) {
  int32_t n = 0, k = k0;
  uint32_t chunks = 0;
  for (; k < count && n < N; ++k) {
    const uint64_t c = static_cast<uint64_t>(jobs[k].count);
    if (c == 0) continue;
    b->g[n] = jobs[k].g;
    b->begin[n] = chunks;
    b->last[n] = static_cast<uint16_t>(((c - 1) % kChunk) | (static_cast<uint64_t>(jobs[k].type) << 14));
    chunks += static_cast<uint32_t>((c + kChunk - 1) / kChunk);
    ++n;
  }
  b->begin[n] = chunks;
  b->spans = n;
  b->chunks = chunks;
  return k;
}

// Calls f(table, blocks) for launch after launch over the jobs. Few tensors get
// a smaller table, since it is part of the launch: both launches over 256 tensors
// take the host 9.7 us with a table of 256, 10.2 with one of 512.
template <int N, typename F>
cudaError_t each_launch(const intlora_grad_job* jobs, int32_t count, F f) {
  static thread_local Spans<N> b;
  for (int32_t k = 0; k < count;) {
    k = fill(jobs, k, count, &b);
    const cudaError_t e = f(b, blocks_of(b.chunks));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <int N>
cudaError_t clip_after(const Spans<N>& b, int64_t blocks, const void* ws, int64_t partials, float max_norm, float* norm,
                       int write, cudaStream_t s) {
  return counted(launch_after(grad_clip_kernel<N>, static_cast<unsigned>(blocks), kThreads, 0, s, b,
                              static_cast<const double*>(ws), partials, max_norm, norm, write));
}
template <typename F>
cudaError_t each_launch(const intlora_grad_job* jobs, int32_t count, F f) {
  if (count <= kFewSpans) return each_launch<kFewSpans>(jobs, count, f);
  return count <= kMidSpans ? each_launch<kMidSpans>(jobs, count, f) : each_launch<kMaxSpans>(jobs, count, f);
}

}  // namespace

// One fp64 partial sum per block of every launch, in launch order.
int64_t grad_norm_partials(const intlora_grad_job* jobs, int32_t count) {
  int64_t total = 0;
  for (int32_t k = 0; k < count;) {
    int64_t chunks = 0;
    for (int32_t n = 0; k < count && n < kMaxSpans; ++k) {
      if (jobs[k].count == 0) continue;
      chunks += (jobs[k].count + kChunk - 1) / kChunk;
      ++n;
    }
    total += blocks_of(chunks);
  }
  return total;
}

cudaError_t launch_grad_squares(const intlora_grad_job* jobs, int32_t count, void* ws, cudaStream_t s) {
  double* partial = static_cast<double*>(ws);
  return each_launch(jobs, count, [&](const auto& b, int64_t blocks) {
    grad_squares_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(b, partial);
    partial += blocks;
    return counted(cudaGetLastError());
  });
}

cudaError_t launch_grad_norm_finish(int64_t partials, const void* ws, float* norm, cudaStream_t s) {
  return counted(launch_after(grad_norm_finish_kernel, 1, kThreads, 0, s, static_cast<const double*>(ws), partials, norm));
}

cudaError_t launch_grad_clip(const intlora_grad_job* jobs, int32_t count, float max_norm, const void* ws,
                             int64_t partials, float* norm, cudaStream_t s) {
  int write = 1;                               // the first launch writes the norm
  return each_launch(jobs, count, [&](const auto& b, int64_t blocks) {
    const cudaError_t launched = clip_after(b, blocks, ws, partials, max_norm, norm, write, s);
    write = 0;
    return launched;
  });
}

cudaError_t launch_clip_grad_norm(const intlora_grad_job* jobs, int32_t count, float max_norm, void* ws,
                                  int64_t partials, float* norm, cudaStream_t s) {
  if (count > kMaxSpans) {                     // the whole norm comes before the first clipping
    const cudaError_t e = launch_grad_squares(jobs, count, ws, s);
    return e != cudaSuccess ? e : launch_grad_clip(jobs, count, max_norm, ws, partials, norm, s);
  }
  return each_launch(jobs, count, [&](const auto& b, int64_t blocks) {   // one table for both
    grad_squares_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(b, static_cast<double*>(ws));
    const cudaError_t e = counted(cudaGetLastError());
    if (e != cudaSuccess) return e;
    return clip_after(b, blocks, ws, partials, max_norm, norm, 1, s);
  });
}

}  // namespace intlora
