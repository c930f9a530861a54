// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   y_t = scale E[id_t]
//   backward  dE_v = scale sum_{t: id_t = v, v != padding} dy_t
//
// Both are bound by memory. The forward gathers rows with 16-byte accesses.
// The backward first sorts the token positions by id, so that every table row
// has one owner that adds its tokens in a fixed order: no atomics on floats,
// the same bits on every run, and each row of dE is written once, untouched
// rows as zeros in the same pass. A word that fills whole aligned chunks of the
// sorted list has those summed side by side by other blocks first, so that one
// frequent word does not become one long serial sum.
//
// Sort: runs of 256 ids are ranked by comparing all pairs of a run; groups of
// 64 sorted runs are then joined by ranks (an element's place is its place in
// its own run plus, by binary search, the number of elements before it in each
// other run), level by level. Ids of equal value keep their order. Ids outside
// the table, and the padding id, get the key `vocab` and sort behind
// everything; nothing reads or writes a row for them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "intlora_kernels.h"
#include "train_ops.h"

namespace intlora {

namespace {

constexpr int kSms = 148;
constexpr int kThreads = 256;
constexpr int kRun = 256;                      // ids ranked at once
constexpr int kFan = 64;                       // runs joined per level
constexpr int kChunk = 32;                     // sorted positions summed by one block of the chunk pass

__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i, int id_bytes) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// A block is tx threads across the chunks of a row times kThreads / tx rows.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    embedding_kernel(const __grid_constant__ EmbeddingJob j, int tx_log2, int rows_per_thread) {
  constexpr int W = VEC ? 8 : 1;
  const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
  const int rows = kThreads >> tx_log2;
  const int64_t c = ((static_cast<int64_t>(blockIdx.y) << tx_log2) + tx) * W;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows * rows_per_thread + ty;
#pragma unroll 4
  for (int k = 0; k < rows_per_thread; ++k) {
    const int64_t t = row0 + static_cast<int64_t>(k) * rows;
    if (t >= j.tokens) break;
    const int64_t id = load_id(j.ids, t, j.id_bytes);
    const bool ok = id >= 0 && id < j.vocab;
    if (!ok && c == 0 && j.invalid != nullptr) atomicAdd(j.invalid, 1);
    if (c >= j.n) continue;
    float v[W];
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = 0.0f;
    if (ok) {
      const void* src = row_ptr(j.table, id, j.ld_table, j.table_type);
      if (VEC) load8(src, c, j.table_type, v);
      else v[0] = load_elem(src, c, j.table_type);
    }
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] *= j.scale;
    void* dst = row_ptr(j.y, t, j.ld_y, j.y_type);
    if (VEC) store8(dst, c, j.y_type, v);
    else store_elem(dst, c, j.y_type, v[0]);
  }
}

// First level of the sort: ranks within a run of kRun ids.
__global__ void __launch_bounds__(kRun)
    embedding_sort_runs_kernel(const __grid_constant__ EmbeddingBackwardJob j, uint32_t* key, uint32_t* pos) {
  __shared__ __align__(16) uint32_t k[kRun];
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * kRun;
  const int64_t at = begin + threadIdx.x;
  const int len = static_cast<int>(min(static_cast<int64_t>(kRun), j.tokens - begin));
  uint32_t mine = 0xffffffffu;                 // behind the run's end: after every id
  if (at < j.tokens) {
    const int64_t id = load_id(j.ids, at, j.id_bytes);
    const bool ok = id >= 0 && id < j.vocab;
    if (!ok && j.invalid != nullptr) atomicAdd(j.invalid, 1);
    mine = static_cast<uint32_t>(ok && id != j.padding_id ? id : j.vocab);
  }
  k[threadIdx.x] = mine;
  __syncthreads();
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < kRun; i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(&k[i]);
    const int t = threadIdx.x;
    rank += (o.x < mine || (o.x == mine && i < t)) + (o.y < mine || (o.y == mine && i + 1 < t)) +
            (o.z < mine || (o.z == mine && i + 2 < t)) + (o.w < mine || (o.w == mine && i + 3 < t));
  }
  if (static_cast<int>(threadIdx.x) < len) {
    key[begin + rank] = mine;
    pos[begin + rank] = static_cast<uint32_t>(at);
  }
}

// Number of elements of run[0 .. len) that come before x: those below x, or
// those up to x for a run that stands earlier in the list.
__device__ __forceinline__ int64_t run_rank(const uint32_t* run, int64_t len, uint32_t x, bool earlier) {
  int64_t lo = 0, hi = len;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (run[mid] < x || (earlier && run[mid] == x)) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Joins groups of kFan sorted runs of `run` elements: `lanes` (a power of two
// up to 32) lanes search the runs of a group for one element and add up.
__global__ void __launch_bounds__(kThreads)
    embedding_join_runs_kernel(const uint32_t* key, const uint32_t* pos, uint32_t* key_out, uint32_t* pos_out,
                               int64_t tokens, int64_t run, int lanes) {
  const int64_t items = kThreads / lanes;
  const int lane = threadIdx.x & (lanes - 1);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * items; base < tokens;
       base += static_cast<int64_t>(gridDim.x) * items) {
    const int64_t e = base + threadIdx.x / lanes;
    const bool live = e < tokens;
    int64_t rank = 0, group = 0;
    if (live) {
      group = e / (run * kFan) * (run * kFan);
      const int64_t own = e / run * run;
      const uint32_t x = key[e];
      for (int64_t b = group + lane * run; b < tokens && b < group + run * kFan; b += lanes * run) {
        if (b == own) rank += e - own;
        else rank += run_rank(key + b, min(run, tokens - b), x, b < own);
      }
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (live && lane == 0) {
      key_out[group + rank] = key[e];
      pos_out[group + rank] = pos[e];
    }
  }
}

// Sum of dy rows pos[a .. b) at columns c .. c + W.
template <bool VEC>
__device__ __forceinline__ void add_rows(const EmbeddingBackwardJob& j, const uint32_t* pos, int64_t a, int64_t b,
                                         int64_t c, float* v) {
  constexpr int W = VEC ? 8 : 1;
#pragma unroll 4
  for (int64_t p = a; p < b; ++p) {
    const void* src = row_ptr(j.dy, static_cast<int64_t>(pos[p]), j.ld_dy, j.dy_type);
    if (VEC) {
      float d[8];
      load8(src, c, j.dy_type, d);
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] += d[e];
    } else {
      v[0] += load_elem(src, c, j.dy_type);
    }
  }
}

// Chunks of kChunk sorted positions that hold one word only: their sum goes to
// row (chunk) of partial.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    embedding_chunks_kernel(const __grid_constant__ EmbeddingBackwardJob j, const uint32_t* key, const uint32_t* pos,
                            float* partial) {
  constexpr int W = VEC ? 8 : 1;
  const int64_t chunk = blockIdx.x;
  const int64_t a = chunk * kChunk, b = a + kChunk;      // the grid covers whole chunks only
  if (key[a] != key[b - 1] || key[a] >= j.vocab) return;
  for (int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * W; c < j.n;
       c += static_cast<int64_t>(gridDim.y) * blockDim.x * W) {
    float v[W];
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = 0.0f;
    add_rows<VEC>(j, pos, a, b, c, v);
    float* out = partial + chunk * j.n + c;
    if (VEC) store8(out, 0, kF32, v);
    else out[0] = v[0];
  }
}

// One table row's gradient at columns c .. c + W from the sorted positions
// [a, b): loose rows, whole chunks, loose rows.
template <bool VEC>
__device__ __forceinline__ void table_row(const EmbeddingBackwardJob& j, const uint32_t* pos, const float* partial,
                                          int64_t row, int64_t a, int64_t b, int64_t c) {
  constexpr int W = VEC ? 8 : 1;
  float v[W];
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = 0.0f;
  const int64_t lo = (a + kChunk - 1) / kChunk, hi = b / kChunk;
  if (lo < hi) {
    add_rows<VEC>(j, pos, a, lo * kChunk, c, v);
#pragma unroll 4
    for (int64_t k = lo; k < hi; ++k) {
      float d[W];
      if (VEC) load8(partial + k * j.n, c, kF32, d);
      else d[0] = partial[k * j.n + c];
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] += d[e];
    }
    add_rows<VEC>(j, pos, hi * kChunk, b, c, v);
  } else {
    add_rows<VEC>(j, pos, a, b, c, v);
  }
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] *= j.scale;
  void* dst = row_ptr(j.dtable, row, j.ld_dtable, j.dtable_type);
  if (j.accumulate) {
    float d[W];
    if (VEC) load8(dst, c, j.dtable_type, d);
    else d[0] = load_elem(dst, c, j.dtable_type);
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] += d[e];
  }
  if (VEC) store8(dst, c, j.dtable_type, v);
  else store_elem(dst, c, j.dtable_type, v[0]);
}

// The whole table: a block owns `rows` (up to kThreads - 1) consecutive rows
// and finds their stretches of the sorted list by binary search.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    embedding_table_kernel(const __grid_constant__ EmbeddingBackwardJob j, const uint32_t* key, const uint32_t* pos,
                           const float* partial, int rows) {
  constexpr int W = VEC ? 8 : 1;
  __shared__ int64_t first[kThreads];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * rows;
  const int live = static_cast<int>(min(static_cast<int64_t>(rows), j.vocab - v0));
  if (static_cast<int>(threadIdx.x) <= live)
    first[threadIdx.x] = run_rank(key, j.tokens, static_cast<uint32_t>(v0 + threadIdx.x), false);
  __syncthreads();
  for (int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * W; c < j.n;
       c += static_cast<int64_t>(gridDim.y) * blockDim.x * W)
    for (int r = 0; r < live; ++r) table_row<VEC>(j, pos, partial, v0 + r, first[r], first[r + 1], c);
}

// Touched rows only: a block looks at `span` sorted positions and owns the
// words that begin there.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    embedding_touched_kernel(const __grid_constant__ EmbeddingBackwardJob j, const uint32_t* key, const uint32_t* pos,
                             const float* partial, int span) {
  constexpr int W = VEC ? 8 : 1;
  __shared__ int64_t end[kThreads];            // 0: no word begins here
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * span;
  if (static_cast<int>(threadIdx.x) < span) {
    const int64_t p = p0 + threadIdx.x;
    int64_t e = 0;
    if (p < j.tokens && key[p] < j.vocab && (p == 0 || key[p - 1] != key[p]))
      e = p + run_rank(key + p, j.tokens - p, key[p], true);
    end[threadIdx.x] = e;
  }
  __syncthreads();
  for (int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * W; c < j.n;
       c += static_cast<int64_t>(gridDim.y) * blockDim.x * W)
    for (int r = 0; r < span; ++r)
      if (end[r] != 0) table_row<VEC>(j, pos, partial, key[p0 + r], p0 + r, end[r], c);
}

bool row_aligned(const void* p, int64_t ld, int type) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elem_bytes(type)) % 16 == 0;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

cudaError_t launch_embedding(const EmbeddingJob& j, cudaStream_t s) {
  const bool vec = j.n % 8 == 0 && row_aligned(j.table, j.ld_table, j.table_type) && row_aligned(j.y, j.ld_y, j.y_type);
  const int64_t units = vec ? j.n / 8 : j.n;
  int tx_log2 = 0;
  while (tx_log2 < 8 && (int64_t{1} << tx_log2) < units) ++tx_log2;
  const int64_t strips = ceil_div(units, int64_t{1} << tx_log2);
  const int64_t rows = kThreads >> tx_log2;
  // four loads in flight a thread once there are rows enough to fill the GPU
  const int per = ceil_div(j.tokens, rows) * strips >= kSms * 8 * 4 ? 4 : 1;
  const int64_t gx = ceil_div(j.tokens, rows * per);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(strips));
  if (vec) embedding_kernel<true><<<grid, kThreads, 0, s>>>(j, tx_log2, per);
  else embedding_kernel<false><<<grid, kThreads, 0, s>>>(j, tx_log2, per);
  return counted(cudaGetLastError());
}

// Two buffers of keys and positions, and a row of partial sums per whole chunk.
size_t embedding_backward_ws(int64_t tokens, int64_t n) {
  return 4 * round256(static_cast<size_t>(tokens) * 4) +
         round256(static_cast<size_t>(tokens / kChunk) * static_cast<size_t>(n) * sizeof(float));
}

cudaError_t launch_embedding_backward(const EmbeddingBackwardJob& j, void* ws, cudaStream_t s) {
  const size_t list = round256(static_cast<size_t>(j.tokens) * 4);
  char* w = static_cast<char*>(ws);
  uint32_t* key = reinterpret_cast<uint32_t*>(w);
  uint32_t* pos = reinterpret_cast<uint32_t*>(w + list);
  uint32_t* key2 = reinterpret_cast<uint32_t*>(w + 2 * list);
  uint32_t* pos2 = reinterpret_cast<uint32_t*>(w + 3 * list);
  float* partial = reinterpret_cast<float*>(w + 4 * list);
  const bool vec = j.n % 8 == 0 && row_aligned(j.dy, j.ld_dy, j.dy_type) &&
                   row_aligned(j.dtable, j.ld_dtable, j.dtable_type);
  const int64_t units = vec ? j.n / 8 : j.n;
  const int threads = static_cast<int>(std::min<int64_t>(kThreads, ceil_div(units, 32) * 32));
  const unsigned strips = static_cast<unsigned>(std::min<int64_t>(ceil_div(units, threads), 32768));
  cudaError_t e = cudaSuccess;
  if (j.tokens > 0) {
    embedding_sort_runs_kernel<<<static_cast<unsigned>(ceil_div(j.tokens, kRun)), kRun, 0, s>>>(j, key, pos);
    if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
    for (int64_t run = kRun; run < j.tokens; run *= kFan) {
      int lanes = 1;
      while (lanes < 32 && lanes < ceil_div(j.tokens, run)) lanes *= 2;
      const int64_t blocks = std::min<int64_t>(ceil_div(j.tokens, kThreads / lanes), kSms * 32);
      embedding_join_runs_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(key, pos, key2, pos2, j.tokens, run,
                                                                                   lanes);
      if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
      std::swap(key, key2);
      std::swap(pos, pos2);
    }
    if (j.tokens >= kChunk) {
      const dim3 grid(static_cast<unsigned>(j.tokens / kChunk), strips);
      if (vec) embedding_chunks_kernel<true><<<grid, threads, 0, s>>>(j, key, pos, partial);
      else embedding_chunks_kernel<false><<<grid, threads, 0, s>>>(j, key, pos, partial);
      if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
    }
  }
  if (j.accumulate) {
    if (j.tokens == 0) return cudaSuccess;
    const int span = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, j.tokens * strips / (kSms * 8))));
    const dim3 grid(static_cast<unsigned>(ceil_div(j.tokens, span)), strips);
    if (vec) embedding_touched_kernel<true><<<grid, threads, 0, s>>>(j, key, pos, partial, span);
    else embedding_touched_kernel<false><<<grid, threads, 0, s>>>(j, key, pos, partial, span);
  } else {
    const int rows = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, j.vocab * strips / (kSms * 8))));
    const dim3 grid(static_cast<unsigned>(ceil_div(j.vocab, rows)), strips);
    if (vec) embedding_table_kernel<true><<<grid, threads, 0, s>>>(j, key, pos, partial, rows);
    else embedding_table_kernel<false><<<grid, threads, 0, s>>>(j, key, pos, partial, rows);
  }
  return counted(cudaGetLastError());
}

}  // namespace intlora
