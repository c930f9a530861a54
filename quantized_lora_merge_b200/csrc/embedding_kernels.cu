// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   y_t = scale E[id_t]
//   backward  dE_v = scale sum_{t: id_t = v, v != padding} dy_t
//
// Both are bound by memory. The forward gathers rows with 16- or 32-byte
// accesses, a thread's next rows in flight while it writes the last ones.
//
// The backward sorts the token positions by id, so that every table row has one
// owner that adds its tokens in a fixed order: no atomics on floats, the same
// bits on every run, and each row of dE is written once, untouched rows as zeros
// in the same pass. A warp owns one strip of a row's columns, so that a row
// whose tokens have to be fetched holds up no other. A word that fills whole
// aligned chunks of the sorted list has those summed side by side by other
// warps first, so that one frequent word does not become one long serial sum.
//
// Sort: runs of 256 ids are ranked by comparing all pairs of a run; groups of
// 64 sorted runs are then joined by ranks (an element's place is its place in
// its own run plus, by binary search, the number of elements before it in each
// other run), level by level. Ids of equal value keep their order. Ids outside
// the table, and the padding id, get the key `vocab` and sort behind
// everything; nothing reads or writes a row for them.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "elem.cuh"
#include "intlora_kernels.h"
#include "train_ops.h"

namespace intlora {

namespace {

constexpr int kSms = 148;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 256;                      // ids ranked at once
constexpr int kFan = 64;                       // runs joined per level
constexpr int kJoinThreads = 512;
constexpr int kRunPitch = kRun + 1;            // words between runs in shared memory: searches that start in
                                               // the middle of every run fall into different banks
constexpr int kChunk = 32;                     // sorted positions summed by one warp of the chunk pass
constexpr int kMaxRows = 32;                   // table rows, or sorted positions, of a block
constexpr int kLookupBlocks = 3;               // of the lookup, an SM: 60 us for 32768 x 4096, with 2 68, with 4 66

// A row of a matrix. Row numbers are below 2^32 everywhere, so that the product
// with the row's bytes is one of 32 by 64 bits.
__device__ __forceinline__ const char* row_at(const void* p, uint32_t row, int64_t row_bytes) {
  return static_cast<const char*>(p) + static_cast<uint64_t>(row) * static_cast<uint64_t>(row_bytes);
}
__device__ __forceinline__ char* row_at(void* p, uint32_t row, int64_t row_bytes) {
  return static_cast<char*>(p) + static_cast<uint64_t>(row) * static_cast<uint64_t>(row_bytes);
}

__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i, int id_bytes) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// A block is tx threads across the 8-column units (VEC) or columns of a row
// times kThreads / tx rows; blocks walk over tiles of R rows a thread, U units
// of each, with a grid stride. The ids of a tile are read two tiles ahead and
// its rows one tile ahead, so that neither read is waited for.
constexpr uint32_t kNoRow = 0xffffffffu;
template <int TYPE, int TO, bool VEC, int R, int U>
__global__ void __launch_bounds__(kThreads)
    embedding_kernel(const __grid_constant__ EmbeddingJob j, int tx_log2, unsigned strips) {
  constexpr int kWords = VEC ? (TYPE == kF32 ? 8 : 4) : 1;
  const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
  const uint32_t rows = kThreads >> tx_log2;
  const unsigned strip = blockIdx.x % strips, block = blockIdx.x / strips, blocks = gridDim.x / strips;
  const int64_t c = ((static_cast<int64_t>(strip) << tx_log2) * U + tx) * (VEC ? 8 : 1);
  const int64_t hop = static_cast<int64_t>(VEC ? 8 : 1) << tx_log2;      // columns between a thread's units
  const uint32_t tokens = static_cast<uint32_t>(j.tokens);
  const uint32_t tile = rows * R, step = tile * blocks;
  const int64_t table_row = j.ld_table * elem_bytes(TYPE), y_row = j.ld_y * elem_bytes(TO);
  uint32_t t0 = block * tile + ty;
  uint32_t id[R];                              // kNoRow: outside the table, or no token
  uint32_t next[R][U][kWords];
  const auto read_ids = [&](uint32_t t) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      id[k] = kNoRow;
      if (t + k * rows >= tokens) continue;
      const uint64_t v = static_cast<uint64_t>(load_id(j.ids, t + k * rows, j.id_bytes));
      if (v < static_cast<uint64_t>(j.vocab)) id[k] = static_cast<uint32_t>(v);
      else if (c == 0 && j.invalid != nullptr) atomicAdd(j.invalid, 1);
    }
  };
  const auto read_rows = [&]() {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const char* src = row_at(j.table, id[k], table_row) + c * elem_bytes(TYPE);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t* w = next[k][u];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
        if (id[k] == kNoRow || c + u * hop >= j.n) continue;
        const char* p = src + u * hop * elem_bytes(TYPE);
        if constexpr (!VEC) {
          w[0] = TYPE == kF32 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : __ldg(reinterpret_cast<const uint16_t*>(p));
        } else if constexpr (TYPE == kF32) {
          load32(p, w);
        } else {
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
          w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        }
      }
    }
  };
  read_ids(t0);
  read_rows();
  read_ids(t0 + step);
  for (; t0 < tokens; t0 += step) {
    uint32_t w[R][U][kWords];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[k][u][i] = next[k][u][i];
    read_rows();
    read_ids(t0 + 2 * step);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (t0 + k * rows >= tokens) break;
      char* y = row_at(j.y, t0 + k * rows, y_row);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c + u * hop >= j.n) break;
        if constexpr (VEC) {
          float v[8];
          if constexpr (TYPE == kF32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[k][u][e]);
          } else {
            unpack8(w[k][u], TYPE, v);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= j.scale;
          store8(y, c + u * hop, TO, v);
        } else {
          store_elem(y, c + u * hop, TO, elem_from_bits(w[k][u][0], TYPE) * j.scale);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
// The sort key of token `at`; ids outside the table are counted when `count`.
__device__ __forceinline__ uint32_t token_key(const EmbeddingBackwardJob& j, int64_t at, bool count) {
  const int64_t id = load_id(j.ids, at, j.id_bytes);
  const bool ok = id >= 0 && id < j.vocab;
  if (!ok && count && j.invalid != nullptr) atomicAdd(j.invalid, 1);
  return static_cast<uint32_t>(ok && id != j.padding_id ? id : j.vocab);
}

// First level: ranks within a run of kRun ids.
__global__ void __launch_bounds__(kRun)
    embedding_sort_runs_kernel(const __grid_constant__ EmbeddingBackwardJob j, uint32_t* key, uint32_t* pos) {
  __shared__ __align__(16) uint32_t k[kRun];
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * kRun;
  const int64_t at = begin + threadIdx.x;
  // behind the run's end: after every id
  const uint32_t mine = at < j.tokens ? token_key(j, at, true) : 0xffffffffu;
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
  if (at < j.tokens) {
    key[begin + rank] = mine;
    pos[begin + rank] = static_cast<uint32_t>(at);
  }
}

// Number of elements of run[0 .. len) that come before x: those below x, or
// those up to x for a run that stands earlier in the list.
template <typename I>
__device__ __forceinline__ I run_rank(const uint32_t* run, I len, uint32_t x, bool earlier) {
  I lo = 0, hi = len;
  while (lo < hi) {
    const I mid = (lo + hi) >> 1;
    const uint32_t k = run[mid];
    if (k < x || (earlier && k == x)) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Joins a group of up to kFan runs of kRun elements, whose keys lie in shared
// memory (missing ones as the largest): a warp ranks one element, every lane
// searching two runs in step, without branches. Blocks blockIdx.x of gridDim.x
// share the group blockIdx.y. (Searching in global memory instead took 29 us for
// 16384 tokens.)
__global__ void __launch_bounds__(kJoinThreads)
    embedding_join_first_kernel(const uint32_t* key, const uint32_t* pos, uint32_t* key_out, uint32_t* pos_out,
                                int64_t tokens) {
  static_assert(kFan == 64, "two runs a lane");
  extern __shared__ uint32_t runs[];           // kFan x kRunPitch
  const int64_t group = static_cast<int64_t>(blockIdx.y) * (kRun * kFan);
  const int count = static_cast<int>(min(static_cast<int64_t>(kRun * kFan), tokens - group));
  const int nruns = (count + kRun - 1) / kRun;
  wait_for_previous();
#pragma unroll 8
  for (int i = threadIdx.x; i < nruns * (kRun / 4); i += kJoinThreads) {
    uint4 k = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
    if (i * 4 + 4 <= count) {                  // the lists start at 256-byte boundaries
      k = *(reinterpret_cast<const uint4*>(key + group) + i);
    } else {
      if (i * 4 < count) k.x = key[group + i * 4];
      if (i * 4 + 1 < count) k.y = key[group + i * 4 + 1];
      if (i * 4 + 2 < count) k.z = key[group + i * 4 + 2];
    }
    uint32_t* to = runs + i * 4 / kRun * kRunPitch + i * 4 % kRun;
    to[0] = k.x;
    to[1] = k.y;
    to[2] = k.z;
    to[3] = k.w;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t* run_a = runs + lane * kRunPitch;
  const uint32_t* run_b = runs + (lane + 32) * kRunPitch;
  const bool has_a = lane < nruns, has_b = lane + 32 < nruns;
  for (int e = blockIdx.x * (kJoinThreads / 32) + warp; e < count; e += gridDim.x * (kJoinThreads / 32)) {
    const int own = e / kRun;
    const uint32_t x = runs[own * kRunPitch + e % kRun];
    // elements of a run before x: below it, or up to it in earlier runs (x < 2^31)
    const uint32_t xa = x + (lane < own), xb = x + (lane + 32 < own);
    int a = 0, b = 0;
#pragma unroll
    for (int step = kRun / 2; step > 0; step >>= 1) {
      if (has_a && run_a[a + step - 1] < xa) a += step;
      if (has_b && run_b[b + step - 1] < xb) b += step;
    }
    if (has_a && run_a[a] < xa) ++a;           // a < kRun: the last of the run
    if (has_b && run_b[b] < xb) ++b;
    if (lane == own) a = e % kRun;
    if (lane + 32 == own) b = e % kRun;
    int rank = a + b;
    for (int o = 16; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (lane == 0) {
      key_out[group + rank] = x;
      pos_out[group + rank] = pos[group + e];
    }
  }
}

// The levels above: `lanes` (a power of two up to 32) lanes search the runs of a
// group in memory for one element and add up.
__global__ void __launch_bounds__(kThreads)
    embedding_join_runs_kernel(const uint32_t* key, const uint32_t* pos, uint32_t* key_out, uint32_t* pos_out,
                               int64_t tokens, int64_t run, int lanes) {
  const int64_t items = kThreads / lanes;
  const int lane = threadIdx.x & (lanes - 1);
  wait_for_previous();
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

// First place in key[0 .. count) that is not below x, by a whole warp: 33-fold
// in every step.
__device__ __forceinline__ int64_t warp_lower_bound(const uint32_t* key, int64_t count, uint32_t x) {
  int64_t lo = 0, hi = count;
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int64_t step = (hi - lo + 32) / 33;
    const int64_t at = lo + (lane + 1) * step - 1;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && key[at] < x);
    const int passed = __popc(below);          // key is sorted: the lower lanes
    if (passed < 32) hi = min(hi, lo + (passed + 1) * step - 1);
    lo += passed * step;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// sums of token rows
// ---------------------------------------------------------------------------
// A warp's strip of columns: lane l has, for chunk k of kStrip, the 8 columns
// from (32 k + l) 8 on (VEC), or single columns 32 k + l.
constexpr int kVecChunks = 1, kScalarChunks = 4;
constexpr int strip_columns(bool vec) { return vec ? 32 * 8 * kVecChunks : 32 * kScalarChunks; }

template <bool VEC>
struct Strip {
  static constexpr int C = VEC ? kVecChunks : kScalarChunks;
  static constexpr int W = VEC ? 8 : 1;
  float v[C * W];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < C * W; ++i) v[i] = 0.0f;
  }
};

// Raw words of one row's strip; columns at or past n are zero.
template <int TYPE, bool VEC>
struct RawStrip {
  using S = Strip<VEC>;
  static constexpr int kWords = VEC ? (TYPE == kF32 ? 8 : 4) : 1;
  uint32_t w[S::C * kWords];
  __device__ __forceinline__ void load(const void* row, int64_t c0, int64_t n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < S::C; ++k) {
      const int64_t c = c0 + (32 * k + lane) * S::W;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[k * kWords + i] = 0u;
      if (c >= n) continue;
      if constexpr (!VEC) {
        if constexpr (TYPE == kF32) w[k] = static_cast<const uint32_t*>(row)[c];     // dy, or the chunks' sums
        else w[k] = __ldg(static_cast<const uint16_t*>(row) + c);
      } else {
        const char* p = static_cast<const char*>(row) + c * elem_bytes(TYPE);
        if constexpr (TYPE == kF32) {
          load32(p, w + k * kWords);
        } else {
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
          w[k * kWords] = a.x; w[k * kWords + 1] = a.y; w[k * kWords + 2] = a.z; w[k * kWords + 3] = a.w;
        }
      }
    }
  }
  __device__ __forceinline__ void add_to(S& s) const {
#pragma unroll
    for (int k = 0; k < S::C; ++k) {
      if constexpr (VEC && TYPE != kF32) {
        float d[8];
        unpack8(&w[k * kWords], TYPE, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[8 * k + e] += d[e];
      } else {
#pragma unroll
        for (int e = 0; e < S::W; ++e) s.v[S::W * k + e] += elem_from_bits(w[k * kWords + (VEC ? e : 0)], TYPE);
      }
    }
  }
};

// Adds `count` rows in order. at(i) is the number of row i; every lane looks up
// one of the next 32 numbers, and the warp hands them round.
template <int TYPE, bool VEC, int U, typename F>
__device__ __forceinline__ void add_rows(Strip<VEC>& s, const void* base, int64_t ld, int64_t count, int64_t c0, int64_t n,
                                         F at) {
  const int lane = threadIdx.x & 31;
  for (int64_t i0 = 0; i0 < count; i0 += 32) {
    const uint32_t mine = i0 + lane < count ? at(i0 + lane) : 0u;
    const int here = static_cast<int>(min(int64_t{32}, count - i0));
    for (int i = 0; i < here; i += U) {
      RawStrip<TYPE, VEC> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // behind the last row: that row again, so that no branch parts the loads
        const uint32_t row = __shfl_sync(0xffffffffu, mine, min(i + u, here - 1));
        r[u].load(row_at(base, row, ld * elem_bytes(TYPE)), c0, n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < here) r[u].add_to(s);
    }
  }
}

// Rows in flight where many warps share an SM.
template <int TYPE>
constexpr int kRowsAhead = TYPE == kF32 ? 2 : 4;

// A strip of row v as it is (accumulate), read ahead of the token rows.
template <bool VEC>
struct OldStrip {
  using S = Strip<VEC>;
  float d[S::C * S::W];
  __device__ __forceinline__ void load(const EmbeddingBackwardJob& j, uint32_t v, int64_t c0) {
    const char* src = row_at(j.dtable, v, j.ld_dtable * elem_bytes(j.dtable_type));
#pragma unroll
    for (int k = 0; k < S::C; ++k) {
      const int64_t c = c0 + (32 * k + (threadIdx.x & 31)) * S::W;
#pragma unroll
      for (int e = 0; e < S::W; ++e) d[k * S::W + e] = 0.0f;
      if (!j.accumulate || c >= j.n) continue;
      if constexpr (VEC) load8(src, c, j.dtable_type, d + k * S::W);
      else d[k] = load_elem(src, c, j.dtable_type);
    }
  }
};
// Scales a strip, adds what was there, and writes it to row v of the table.
template <bool VEC>
__device__ __forceinline__ void finish_row(Strip<VEC>& s, const OldStrip<VEC>& old, const EmbeddingBackwardJob& j,
                                           uint32_t v, int64_t c0) {
  using S = Strip<VEC>;
  char* dst = row_at(j.dtable, v, j.ld_dtable * elem_bytes(j.dtable_type));
#pragma unroll
  for (int k = 0; k < S::C; ++k) {
    const int64_t c = c0 + (32 * k + (threadIdx.x & 31)) * S::W;
    if (c >= j.n) continue;
    float* p = s.v + k * S::W;
#pragma unroll
    for (int e = 0; e < S::W; ++e) {
      p[e] *= j.scale;
      if (j.accumulate) p[e] += old.d[k * S::W + e];   // keeps a sum of -0 as it is otherwise
    }
    if constexpr (VEC) store8(dst, c, j.dtable_type, p);
    else store_elem(dst, c, j.dtable_type, p[0]);
  }
}

// Zeros in a table row, by a whole block.
template <bool VEC>
__device__ __forceinline__ void zero_row(const EmbeddingBackwardJob& j, uint32_t v) {
  const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  const int es = elem_bytes(j.dtable_type);
  char* dst = row_at(j.dtable, v, j.ld_dtable * es);
  if (VEC) {
    const int64_t bytes = j.n * es;
    if (es == 4) {
      for (int64_t b = threadIdx.x * 32; b < bytes; b += kThreads * 32) store32(dst + b, zero);
    } else {
      for (int64_t b = threadIdx.x * 16; b < bytes; b += kThreads * 16)
        *reinterpret_cast<uint4*>(dst + b) = make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    for (int64_t c = threadIdx.x; c < j.n; c += kThreads) store_elem(dst, c, j.dtable_type, 0.0f);
  }
}

// What does not wait for the rows' owners. The first chunk_blocks blocks: chunks
// of kChunk sorted positions that hold one word only, a warp a strip of a chunk;
// their sum goes to row (chunk) of partial. The others, where the whole table is
// written: zeros in the untouched ones of `rows` table rows a block. (One after
// the other these took 24 us and 60 us for 16384 tokens, 32000 x 4096.)
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(kThreads, 4)
    embedding_chunks_kernel(const __grid_constant__ EmbeddingBackwardJob j, const uint32_t* key, const uint32_t* pos,
                            float* partial, int strips, unsigned chunk_blocks, int rows) {
  wait_for_previous();
  if (blockIdx.x >= chunk_blocks) {
    __shared__ int64_t stretch[2];
    __shared__ int has[kMaxRows];
    const int64_t v0 = static_cast<int64_t>(blockIdx.x - chunk_blocks) * rows;
    const int live = static_cast<int>(min(static_cast<int64_t>(rows), j.vocab - v0));
    if (threadIdx.x < kMaxRows) has[threadIdx.x] = 0;
    if (threadIdx.x < 64) {
      const int64_t p = warp_lower_bound(key, j.tokens, static_cast<uint32_t>(v0 + (threadIdx.x < 32 ? 0 : live)));
      if ((threadIdx.x & 31) == 0) stretch[threadIdx.x >> 5] = p;
    }
    __syncthreads();
    for (int64_t p = stretch[0] + threadIdx.x; p < stretch[1]; p += kThreads) has[key[p] - v0] = 1;
    __syncthreads();
    for (int r = 0; r < live; ++r)
      if (!has[r]) zero_row<VEC>(j, static_cast<uint32_t>(v0 + r));
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t chunk = item / strips;
  if (chunk >= j.tokens / kChunk) return;
  const int64_t a = chunk * kChunk, b = a + kChunk;
  if (key[a] != key[b - 1] || key[a] >= j.vocab) return;
  const int64_t c0 = (item - chunk * strips) * strip_columns(VEC);
  Strip<VEC> s;
  s.clear();
  add_rows<TYPE, VEC, TYPE == kF32 && VEC ? 4 : 8>(s, j.dy, j.ld_dy, kChunk, c0, j.n,
                                                   [&](int64_t i) { return pos[a + i]; });
  float* out = partial + chunk * j.n;
#pragma unroll
  for (int k = 0; k < Strip<VEC>::C; ++k) {
    const int64_t c = c0 + (32 * k + (threadIdx.x & 31)) * Strip<VEC>::W;
    if (c >= j.n) continue;
    if constexpr (VEC) store8(out, c, kF32, s.v + 8 * k);
    else out[c] = s.v[k];
  }
}

// A strip that the block's warps have summed in parts: added in the order of the
// warps, scaled, and written. part: [kWarps][strip].
template <bool VEC>
__device__ __forceinline__ void join_parts(float (*part)[strip_columns(VEC)], const Strip<VEC>& s,
                                           const EmbeddingBackwardJob& j, uint32_t v, int64_t c0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < Strip<VEC>::C; ++k)
#pragma unroll
    for (int e = 0; e < Strip<VEC>::W; ++e)
      part[warp][(32 * k + lane) * Strip<VEC>::W + e] = s.v[k * Strip<VEC>::W + e];
  __syncthreads();
  for (int c = threadIdx.x; c < strip_columns(VEC) && c0 + c < j.n; c += kThreads) {
    float x = part[0][c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x += part[w][c];
    char* dst = row_at(j.dtable, v, j.ld_dtable * elem_bytes(j.dtable_type));
    x *= j.scale;
    if (j.accumulate) x += load_elem(dst, c0 + c, j.dtable_type);
    store_elem(dst, c0 + c, j.dtable_type, x);
  }
  __syncthreads();
}

// Up to kSmall tokens: one launch, no sort. Every block has all keys in shared
// memory; of its `per` (up to kMaxRows) table rows, or tokens, a warp collects
// the positions of one word in order and adds their rows, a strip at a time.
// A word with more than kManyTokens tokens is shared by the block's warps
// instead: contiguous parts of its list, added in the order of the warps.
constexpr int kSmall = 512, kManyTokens = 48;
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(kThreads)
    embedding_small_kernel(const __grid_constant__ EmbeddingBackwardJob j, int per, int strips) {
  __shared__ uint32_t key[kSmall];
  __shared__ uint16_t list[kWarps][kSmall];
  __shared__ uint32_t word[kMaxRows];
  __shared__ int has[kMaxRows], heavy[kMaxRows];
  __shared__ float part[kWarps][strip_columns(VEC)];
  __shared__ int words, heavies;
  const int tokens = static_cast<int>(j.tokens), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSmall; i += kThreads) key[i] = i < tokens ? token_key(j, i, blockIdx.x == 0) : kNoRow;
  if (threadIdx.x < kMaxRows) has[threadIdx.x] = 0;
  if (threadIdx.x == 0) heavies = 0;
  __syncthreads();
  const int64_t l0 = static_cast<int64_t>(blockIdx.x) * per;
  if (j.accumulate) {                          // a word belongs to its first token
    for (int p = static_cast<int>(l0) + warp; p < min(static_cast<int>(l0) + per, tokens); p += kWarps) {
      const uint32_t x = key[p];
      bool before = x >= j.vocab;
      for (int q = lane; q < p; q += 32) before |= key[q] == x;
      if (!__any_sync(0xffffffffu, before) && lane == 0) has[p - l0] = 1;
    }
  } else {
    for (int i = threadIdx.x; i < tokens; i += kThreads)
      if (key[i] >= l0 && key[i] < min(l0 + per, j.vocab)) has[key[i] - l0] = 1;
  }
  __syncthreads();
  if (warp == 0) {
    const bool mine = has[lane] != 0;
    const unsigned all = __ballot_sync(0xffffffffu, mine);
    if (mine) word[__popc(all & ((1u << lane) - 1u))] = j.accumulate ? key[l0 + lane] : static_cast<uint32_t>(l0 + lane);
    if (lane == 0) words = __popc(all);
  }
  if (!j.accumulate)
    for (int r = 0; r < per && l0 + r < j.vocab; ++r)
      if (!has[r]) zero_row<VEC>(j, static_cast<uint32_t>(l0 + r));
  __syncthreads();
  // positions of a word, in order, in the warp's list
  const auto collect = [&](uint32_t x) {
    int count = 0;
    __syncwarp();
    for (int q = 0; q < tokens; q += 32) {
      const bool hit = key[q + lane] == x;     // kSmall keys, no word behind the tokens
      const unsigned all = __ballot_sync(0xffffffffu, hit);
      if (hit) list[warp][count + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(q + lane);
      count += __popc(all);
    }
    __syncwarp();
    return count;
  };
  uint32_t known = kNoRow;
  int count = 0;
  for (int item = warp; item < words * strips; item += kWarps) {
    const int r = item / strips;
    if (word[r] != known) {
      known = word[r];
      count = collect(known);
    }
    if (count > kManyTokens) {
      if (item == r * strips && lane == 0) heavy[atomicAdd(&heavies, 1)] = r;
      continue;
    }
    const int64_t c0 = static_cast<int64_t>(item - r * strips) * strip_columns(VEC);
    OldStrip<VEC> old;
    old.load(j, known, c0);
    Strip<VEC> s;
    s.clear();
    add_rows<TYPE, VEC, 4>(s, j.dy, j.ld_dy, count, c0, j.n, [&](int64_t i) { return uint32_t{list[warp][i]}; });
    finish_row<VEC>(s, old, j, known, c0);
  }
  __syncthreads();
  for (int h = 0; h < heavies; ++h) {          // in any order: their rows are disjoint
    const uint32_t x = word[heavy[h]];
    count = collect(x);
    const int from = count * warp / kWarps, to = count * (warp + 1) / kWarps;
    for (int strip = 0; strip < strips; ++strip) {
      const int64_t c0 = static_cast<int64_t>(strip) * strip_columns(VEC);
      Strip<VEC> s;
      s.clear();
      add_rows<TYPE, VEC, 4>(s, j.dy, j.ld_dy, to - from, c0, j.n, [&](int64_t i) { return uint32_t{list[warp][from + i]}; });
      join_parts<VEC>(part, s, j, x, c0);
    }
  }
}

// Words of up to kFewTokens tokens, the most of a text: no chunk, positions in
// shared memory, 32-bit arithmetic, two strips at once, up to four token rows in
// flight. (By the general way below, 50 instructions an
// element, the touched rows of 16384 tokens of different words took 133 us.)
constexpr int kFewTokens = 8;
template <int TYPE, bool VEC, bool ACC, bool OUT32>
__device__ __forceinline__ void few_tokens(const EmbeddingBackwardJob& j, const uint32_t* pos, int count, uint32_t v,
                                           int64_t c0) {
  constexpr int W = VEC ? 8 : 1, C = VEC ? 2 : 4, U = TYPE == kF32 && VEC ? 2 : 4;
  constexpr int kWords = VEC ? (TYPE == kF32 ? 8 : 4) : 1;
  const int to = OUT32 ? kF32 : j.dtable_type;
  const int lane = threadIdx.x & 31;
  const int64_t c = c0 + lane * W;
  const int64_t dy_row = j.ld_dy * elem_bytes(TYPE);
  char* dst = row_at(j.dtable, v, j.ld_dtable * elem_bytes(to));
  float s[C][W], old[C][W];
#pragma unroll
  for (int k = 0; k < C; ++k) {
#pragma unroll
    for (int e = 0; e < W; ++e) s[k][e] = old[k][e] = 0.0f;
    if (!ACC || c + 32 * W * k >= j.n) continue;
    if constexpr (VEC) load8(dst, c + 32 * W * k, to, old[k]);
    else old[k][0] = load_elem(dst, c + 32 * W * k, to);
  }
#pragma unroll
  for (int i = 0; i < kFewTokens; i += U) {
    if (i >= count) break;
    uint32_t w[U][C][kWords];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const char* src = row_at(j.dy, pos[min(i + u, count - 1)], dy_row) + c * elem_bytes(TYPE);
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int q = 0; q < kWords; ++q) w[u][k][q] = 0u;
        if (c + 32 * W * k >= j.n) continue;
        const char* p = src + 32 * W * k * elem_bytes(TYPE);
        if constexpr (!VEC) {
          w[u][k][0] = TYPE == kF32 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : __ldg(reinterpret_cast<const uint16_t*>(p));
        } else if constexpr (TYPE == kF32) {
          load32(p, w[u][k]);
        } else {
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
          w[u][k][0] = a.x; w[u][k][1] = a.y; w[u][k][2] = a.z; w[u][k][3] = a.w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= count) break;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float d[8];
        if constexpr (VEC && TYPE != kF32) unpack8(w[u][k], TYPE, d);
#pragma unroll
        for (int e = 0; e < W; ++e) s[k][e] += VEC && TYPE != kF32 ? d[e] : elem_from_bits(w[u][k][e], TYPE);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < C; ++k) {
    if (c + 32 * W * k >= j.n) continue;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      s[k][e] *= j.scale;
      if (ACC) s[k][e] += old[k][e];
    }
    if constexpr (VEC) store8(dst, c + 32 * W * k, to, s[k]);
    else store_elem(dst, c + 32 * W * k, to, s[k][0]);
  }
}

// Sorted positions that a block of the touched pass keeps in shared memory, and
// the words that begin among the first `span` of them.
constexpr int kPositions = 128;
struct Words {
  int64_t first[kPositions], last[kPositions]; // sorted positions of a word
  uint32_t word[kPositions];
  uint32_t pos[kPositions], key[kPositions + 1];   // key[i + 1]: position p0 + i
  int count;
};
// Words with at least `least` tokens, in no particular order.
__device__ __forceinline__ void find_words(Words& w, const EmbeddingBackwardJob& j, const uint32_t* key,
                                           const uint32_t* pos, int64_t p0, int span, int least) {
  static_assert(kThreads == 2 * kPositions, "a thread an entry");
  const int t = threadIdx.x;
  const int near = static_cast<int>(min(static_cast<int64_t>(kPositions), j.tokens - p0));
  if (t < kPositions) {
    if (t < near) w.key[t + 1] = key[p0 + t];
    if (t == 0) {
      w.key[0] = p0 > 0 ? key[p0 - 1] : kNoRow;
      w.count = 0;
    }
  } else if (t - kPositions < near) {
    w.pos[t - kPositions] = pos[p0 + t - kPositions];
  }
  __syncthreads();
  if (t < span && t < near) {
    const uint32_t x = w.key[t + 1];
    if (x < j.vocab && w.key[t] != x) {
      int end = t + 1;
      while (end < near && w.key[end + 1] == x) ++end;
      int64_t e = p0 + end;
      if (end == near && e < j.tokens)         // it goes on behind what is here
        e += run_rank<int64_t>(key + e, j.tokens - e, x, true);
      if (e - (p0 + t) >= least) {
        const int at = atomicAdd(&w.count, 1);
        w.first[at] = p0 + t;
        w.last[at] = e;
        w.word[at] = x;
      }
    }
  }
  __syncthreads();
}

// The rows that make up a word's sum: the tokens before and behind whole chunks,
// then the whole chunks' sums.
struct WordRows {
  int64_t a, head, loose, skip, lo, count;
  __device__ __forceinline__ WordRows(int64_t first, int64_t last) {
    const int64_t hi = last / kChunk;
    a = first;
    lo = (first + kChunk - 1) / kChunk;
    const bool whole = lo < hi;
    head = whole ? lo * kChunk - first : last - first;
    loose = whole ? head + last - hi * kChunk : head;
    skip = whole ? hi * kChunk - head : first;             // from there on the positions behind the chunks
    count = loose + (whole ? hi - lo : 0);
  }
};
template <int TYPE, bool VEC>
__device__ __forceinline__ void add_word(Strip<VEC>& s, const EmbeddingBackwardJob& j, const Words& words,
                                         const uint32_t* pos, int64_t p0, const float* partial, const WordRows& w,
                                         int64_t from, int64_t to, int64_t c0) {
  add_rows<TYPE, VEC, kRowsAhead<TYPE>>(s, j.dy, j.ld_dy, min(to, w.loose) - from, c0, j.n, [&](int64_t i) {
    const int64_t p = (from + i < w.head ? w.a : w.skip) + from + i;
    return p - p0 < kPositions ? words.pos[p - p0] : pos[p];
  });
  const int64_t begin = max(from, w.loose);
  add_rows<kF32, VEC, kRowsAhead<kF32>>(s, partial, j.n, to - begin, c0, j.n,
                                        [&](int64_t i) { return static_cast<uint32_t>(w.lo + (begin - w.loose) + i); });
}

// The touched rows. The first heavy_blocks blocks each look at kPositions sorted
// positions and one strip of columns, for words of more than kManyRows rows that
// begin there: the block's warps add contiguous parts. (One warp alone took 80 us
// for a word with 1500 of 16384 tokens, while all others waited; a block for 8
// strips of it 40 us.) The others look at `span` (up to kMaxRows) positions and
// kBlockStrips strips: words of up to kFewTokens tokens, a warp two strips at
// once, and those between, a warp a strip.
constexpr int kBlockStrips = 8, kManyRows = 16;
template <int TYPE, bool VEC, bool ACC, bool OUT32>
__global__ void __launch_bounds__(kThreads, 4)
    embedding_touched_kernel(const __grid_constant__ EmbeddingBackwardJob j, const uint32_t* key, const uint32_t* pos,
                             const float* partial, int span, int strips, unsigned groups, unsigned heavy_blocks) {
  __shared__ Words words;
  __shared__ float part[kWarps][strip_columns(VEC)];
  const int warp = threadIdx.x >> 5;
  wait_for_previous();
  if (blockIdx.x < heavy_blocks) {
    const int64_t p0 = static_cast<int64_t>(blockIdx.x / strips) * kPositions;
    find_words(words, j, key, pos, p0, kPositions, kManyRows + 1);
    const int64_t c0 = static_cast<int64_t>(blockIdx.x % strips) * strip_columns(VEC);
    for (int r = 0; r < words.count; ++r) {    // in any order: their rows are disjoint
      const WordRows w(words.first[r], words.last[r]);
      if (w.count <= kManyRows) continue;      // the same in all threads
      Strip<VEC> s;
      s.clear();
      add_word<TYPE, VEC>(s, j, words, pos, p0, partial, w, w.count * warp / kWarps, w.count * (warp + 1) / kWarps, c0);
      join_parts<VEC>(part, s, j, words.word[r], c0);
    }
    return;
  }
  const unsigned block = blockIdx.x - heavy_blocks;
  const int64_t p0 = static_cast<int64_t>(block / groups) * span;
  find_words(words, j, key, pos, p0, span, 1);
  const int strip0 = static_cast<int>(block % groups) * kBlockStrips, here = min(kBlockStrips, strips - strip0);
  const int64_t c_begin = static_cast<int64_t>(strip0) * strip_columns(VEC);
  constexpr int kFewColumns = VEC ? 512 : 128;
  const int64_t columns = min(static_cast<int64_t>(here) * strip_columns(VEC), j.n - c_begin);
  const int parts = static_cast<int>((columns + kFewColumns - 1) / kFewColumns);
  const int count = words.count;
  for (int item = warp; item < count * parts; item += kWarps) {
    const int r = item / parts;
    const int64_t tokens = words.last[r] - words.first[r];
    if (tokens <= kFewTokens)
      few_tokens<TYPE, VEC, ACC, OUT32>(j, words.pos + (words.first[r] - p0), static_cast<int>(tokens), words.word[r],
                                        c_begin + (item - r * parts) * kFewColumns);
  }
  for (int item = warp; item < count * here; item += kWarps) {
    const int r = item / here;
    if (words.last[r] - words.first[r] <= kFewTokens) continue;
    const WordRows w(words.first[r], words.last[r]);
    if (w.count > kManyRows) continue;
    const int64_t c0 = c_begin + static_cast<int64_t>(item - r * here) * strip_columns(VEC);
    OldStrip<VEC> old;
    old.load(j, words.word[r], c0);
    Strip<VEC> s;
    s.clear();
    add_word<TYPE, VEC>(s, j, words, pos, p0, partial, w, 0, w.count, c0);
    finish_row<VEC>(s, old, j, words.word[r], c0);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// The sums over the sorted list: chunk pass and table pass.
template <int TYPE, bool VEC>
cudaError_t launch_sums(const EmbeddingBackwardJob& j, const uint32_t* key, const uint32_t* pos, float* partial,
                        cudaStream_t s) {
  const int64_t strips = ceil_div(j.n, strip_columns(VEC));
  if (j.tokens <= kSmall) {
    const int64_t lines = j.accumulate ? j.tokens : j.vocab;
    const int64_t per = std::max<int64_t>(1, std::min<int64_t>(kMaxRows, lines / (kSms * 4)));
    embedding_small_kernel<TYPE, VEC><<<static_cast<unsigned>(ceil_div(lines, per)), kThreads, 0, s>>>(
        j, static_cast<int>(per), static_cast<int>(strips));
    return counted(cudaGetLastError());
  }
  const int64_t chunk_blocks = ceil_div(j.tokens / kChunk * strips, kWarps);
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(kMaxRows, j.vocab / (kSms * 8)));
  const int64_t zero_blocks = j.accumulate ? 0 : ceil_div(j.vocab, rows);
  const cudaError_t e = counted(launch_after(embedding_chunks_kernel<TYPE, VEC>,
                                             static_cast<unsigned>(chunk_blocks + zero_blocks), kThreads, 0, s, j, key, pos,
                                             partial, static_cast<int>(strips), static_cast<unsigned>(chunk_blocks),
                                             static_cast<int>(rows)));
  if (e != cudaSuccess) return e;
  const int64_t groups = ceil_div(strips, kBlockStrips);
  const int64_t span = std::max<int64_t>(1, std::min<int64_t>(kMaxRows / 2, j.tokens * groups / (kSms * 8)));
  const unsigned heavy = static_cast<unsigned>(ceil_div(j.tokens, kPositions) * strips);
  const unsigned grid = heavy + static_cast<unsigned>(ceil_div(j.tokens, span) * groups);
  const int sp = static_cast<int>(span), st = static_cast<int>(strips);
  const unsigned gr = static_cast<unsigned>(groups);
  const bool out32 = j.dtable_type == kF32;
  const auto launch = [&](auto kernel) {
    return counted(launch_after(kernel, grid, kThreads, 0, s, j, key, pos, partial, sp, st, gr, heavy));
  };
  if (j.accumulate && out32) return launch(embedding_touched_kernel<TYPE, VEC, true, true>);
  if (j.accumulate) return launch(embedding_touched_kernel<TYPE, VEC, true, false>);
  if (out32) return launch(embedding_touched_kernel<TYPE, VEC, false, true>);
  return launch(embedding_touched_kernel<TYPE, VEC, false, false>);
}

// The join's shared memory is asked for once per device.
cudaError_t allow_join_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(embedding_join_first_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int TYPE, int TO>
void lookup(const EmbeddingJob& j, bool vec, bool many, unsigned grid, int tx_log2, unsigned strips, cudaStream_t s) {
  if (vec && many) embedding_kernel<TYPE, TO, true, 2, 2><<<grid, kThreads, 0, s>>>(j, tx_log2, strips);
  else if (vec) embedding_kernel<TYPE, TO, true, 1, 1><<<grid, kThreads, 0, s>>>(j, tx_log2, strips);
  else if (many) embedding_kernel<TYPE, TO, false, 2, 4><<<grid, kThreads, 0, s>>>(j, tx_log2, strips);
  else embedding_kernel<TYPE, TO, false, 1, 1><<<grid, kThreads, 0, s>>>(j, tx_log2, strips);
}
template <int TYPE>
void lookup_to(const EmbeddingJob& j, bool vec, bool many, unsigned grid, int tx_log2, unsigned strips, cudaStream_t s) {
  if (j.y_type == kF32) lookup<TYPE, kF32>(j, vec, many, grid, tx_log2, strips, s);
  else if (j.y_type == kBf16) lookup<TYPE, kBf16>(j, vec, many, grid, tx_log2, strips, s);
  else lookup<TYPE, kF16>(j, vec, many, grid, tx_log2, strips, s);
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingJob& j, cudaStream_t s) {
  const bool vec = j.n % 8 == 0 && rows_by_8(j.table, j.ld_table, j.table_type) && rows_by_8(j.y, j.ld_y, j.y_type);
  const int64_t units = vec ? j.n / 8 : j.n;
  // a thread has several units of several rows once that still fills the GPU
  const int most = vec ? 2 : 4;
  bool many = true;
  int tx_log2 = 0;
  unsigned grid = 0, strips = 0;
  for (;;) {
    const int64_t per = many ? most : 1;       // units a thread
    tx_log2 = 0;
    while (tx_log2 < 8 && (per << tx_log2) < units) ++tx_log2;
    const int64_t across = ceil_div(units, per << tx_log2);
    const int64_t tiles = ceil_div(j.tokens, (kThreads >> tx_log2) * (many ? 2 : 1));
    strips = static_cast<unsigned>(across);
    grid = static_cast<unsigned>(across * (many ? std::min(tiles, ceil_div(kSms * kLookupBlocks, across)) : tiles));
    if (!many || tiles * across >= kSms * kLookupBlocks) break;
    many = false;
  }
  if (j.table_type == kF32) lookup_to<kF32>(j, vec, many, grid, tx_log2, strips, s);
  else if (j.table_type == kBf16) lookup_to<kBf16>(j, vec, many, grid, tx_log2, strips, s);
  else lookup_to<kF16>(j, vec, many, grid, tx_log2, strips, s);
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
  cudaError_t e = cudaSuccess;
  if (j.tokens == 0 && j.accumulate) return cudaSuccess;
  if (j.tokens > kSmall) {
    embedding_sort_runs_kernel<<<static_cast<unsigned>(ceil_div(j.tokens, kRun)), kRun, 0, s>>>(j, key, pos);
    if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
    for (int64_t run = kRun; run < j.tokens; run *= kFan) {
      if (run == kRun) {
        constexpr int bytes = kFan * kRunPitch * static_cast<int>(sizeof(uint32_t));
        if ((e = allow_join_smem(bytes)) != cudaSuccess) return e;
        const int64_t groups = ceil_div(j.tokens, kRun * kFan);
        const int64_t warps = std::min<int64_t>(j.tokens, kRun * kFan);
        const int64_t blocks = std::max<int64_t>(1, std::min(ceil_div(warps, kJoinThreads / 32), ceil_div(2 * kSms, groups)));
        // the grid's second dimension ends at 65535: 2^30 tokens a launch
        for (int64_t g = 0; g < groups; g += 65535) {
          const int64_t skip = g * kRun * kFan;
          const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(std::min<int64_t>(65535, groups - g)));
          e = counted(launch_after(embedding_join_first_kernel, grid, kJoinThreads, bytes, s, key + skip, pos + skip,
                                   key2 + skip, pos2 + skip, j.tokens - skip));
          if (e != cudaSuccess) return e;
        }
      } else {
        int lanes = 1;
        while (lanes < 32 && lanes < ceil_div(j.tokens, run)) lanes *= 2;
        const int64_t blocks = std::min<int64_t>(ceil_div(j.tokens, kThreads / lanes), kSms * 32);
        e = counted(launch_after(embedding_join_runs_kernel, static_cast<unsigned>(blocks), kThreads, 0, s, key, pos, key2,
                                 pos2, j.tokens, run, lanes));
        if (e != cudaSuccess) return e;
      }
      std::swap(key, key2);
      std::swap(pos, pos2);
    }
  }
  const bool vec = j.n % 8 == 0 && rows_by_8(j.dy, j.ld_dy, j.dy_type) &&
                   rows_by_8(j.dtable, j.ld_dtable, j.dtable_type);
  if (vec) {
    if (j.dy_type == kF32) return launch_sums<kF32, true>(j, key, pos, partial, s);
    if (j.dy_type == kBf16) return launch_sums<kBf16, true>(j, key, pos, partial, s);
    return launch_sums<kF16, true>(j, key, pos, partial, s);
  }
  if (j.dy_type == kF32) return launch_sums<kF32, false>(j, key, pos, partial, s);
  if (j.dy_type == kBf16) return launch_sums<kBf16, false>(j, key, pos, partial, s);
  return launch_sums<kF16, false>(j, key, pos, partial, s);
}

}  // namespace intlora
