// Layer norm over the rows of a tokens x n activation, and its gradients.
//
//   forward   m = mean_j x_j, v = mean_j (x_j - m)^2, rstd = (v + eps)^-1/2,
//             y_j = (x_j - m) rstd w_j + b_j
//   backward  xh_j = (x_j - m) rstd, g_j = dy_j w_j,
//             dx_j = rstd (g_j - mean g - xh_j mean(g xh)),
//             dw_j = sum_t dy_tj xh_tj, db_j = sum_t dy_tj
//
// Both are bound by memory as long as the instructions an element takes stay
// few: at 6.5 TB/s an SM has 22 issue slots for an element of the bf16 forward
// and 33 of the bf16 backward. So: every row is read from memory once; blocks
// are persistent, and their teams of T threads walk over the rows with a grid
// stride, copying the rows that come next into a ring in shared memory
// (cp.async: no registers, no wait that could fail to end) while they work on
// the present one; a warp of a team holds V x 128 neighbouring columns, so that
// its addresses are one base and constants; sums and products are done two at a
// time (f32x2); types are compile-time in the loops; the parameters are turned
// into fp32 in shared memory once per block. Teams of up to 32 threads never
// leave their warp; wider ones join their row sums through shared memory and a
// named barrier of their own, so that no team waits for another. Statistics,
// sums and products are fp32; y and dx are rounded once.
//
// Two ways through the ring:
//   VEC   rows start at 16-byte boundaries and fill whole 16-byte granules: a
//         warp copies its own columns; a thread works on chunks of 4 of them
//   else  the team copies the row's granules, wherever the row starts in the
//         first one, and a thread works on single columns, 32 apart. A granule
//         that begins before the tensor is fetched element by element and one
//         that ends behind the row is cut short: nothing outside [first
//         element, last element] of the tensor is read.
#include <algorithm>
#include <atomic>

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "intlora_kernels.h"
#include "train_ops.h"

namespace intlora {

namespace {

constexpr int kSms = 148;
constexpr int kChunk = 4;                      // elements of a chunk
constexpr int kWarpCols = 32 * kChunk;         // columns of one chunk of a warp
constexpr int kBlock = 512;                    // threads of a block's teams together; one block per SM
constexpr int kMaxRowT = 1024;                 // threads of a team that has a block to itself
constexpr int kFwdMaxV = 16, kBwdMaxV = 8;     // chunks a thread: 64 values, or 64 accumulators
constexpr int kHoldV = 4;                      // backward: a row stays in registers up to here
constexpr int kMaxStages = 4;
constexpr int64_t kSmemPerSm = 222 * 1024;
constexpr int kWideThreads = 1024;
constexpr int kColThreads = 256;               // column sums of wide rows: columns per block
constexpr int kReduceWarps = 16;

// How rows are spread over a block.
struct RowShape {
  int T = 0, V = 0;                            // threads of a team, chunks of a thread
  int teams = 0, stages = 0;                   // teams of a block, rows of a team's ring
  int stage_bytes = 0;                         // one row of all tensors
  int second = 0;                              // offset of the second tensor in a stage
  int params = 0;                              // offset of the fp32 parameters behind the rings
  int threads() const { return (T * teams + 31) / 32 * 32; }
};

// ---------------------------------------------------------------------------
// two floats at a time
// ---------------------------------------------------------------------------
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float both(F2 a) {
  const float2 s = split(a);
  return s.x + s.y;
}

// ---------------------------------------------------------------------------
// element types at compile time. kAny16: bf16 or fp16, told apart at run time by
// selecting between both conversions; no branch stands in the loops over a row,
// so that the loads of a whole row are in flight together. (With a branch on
// the type around every two chunks the backward of 8192 x 4096 took 73 us
// instead of 63.)
// ---------------------------------------------------------------------------
constexpr int kAny16 = 3;
template <int TYPE>
constexpr int kBytes = TYPE == kF32 ? 4 : 2;

// The block's dynamic shared memory; rows and parameters are addressed by their
// offsets in it.
__device__ __forceinline__ char* smem() {
  extern __shared__ __align__(16) char ring[];
  return ring;
}

template <int TYPE>
__device__ __forceinline__ void unpack4(uint2 w, int type, F2& a, F2& b) {
  float v[4];
  if (TYPE != kF16) {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  if (TYPE != kBf16) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    const bool half = TYPE == kF16 || type == kF16;
    v[0] = half ? x.x : v[0];
    v[1] = half ? x.y : v[1];
    v[2] = half ? y.x : v[2];
    v[3] = half ? y.y : v[3];
  }
  a = f2(v[0], v[1]);
  b = f2(v[2], v[3]);
}
// Four elements at a 16-byte (fp32) or 8-byte boundary.
template <int TYPE>
__device__ __forceinline__ void get4(const char* p, int type, F2& a, F2& b) {
  if (TYPE == kF32) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(p);
    a.v = w.x;
    b.v = w.y;
  } else {
    unpack4<TYPE>(*reinterpret_cast<const uint2*>(p), type, a, b);
  }
}
template <int TYPE>
__device__ __forceinline__ void put4(char* p, int type, bool in, F2 a, F2 b) {
  if (TYPE == kF32) {
    if (in) *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(a.v, b.v);
  } else {
    const float2 x = split(a), y = split(b);
    uint2 w;
    if (TYPE != kF16) {
      const __nv_bfloat162 g = __floats2bfloat162_rn(x.x, x.y), h = __floats2bfloat162_rn(y.x, y.y);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&g), *reinterpret_cast<const uint32_t*>(&h));
    }
    if (TYPE != kBf16) {
      const __half2 g = __floats2half2_rn(x.x, x.y), h = __floats2half2_rn(y.x, y.y);
      const bool half = TYPE == kF16 || type == kF16;
      w.x = half ? *reinterpret_cast<const uint32_t*>(&g) : w.x;
      w.y = half ? *reinterpret_cast<const uint32_t*>(&h) : w.y;
    }
    if (in) *reinterpret_cast<uint2*>(p) = w;
  }
}
// One element.
template <int TYPE>
__device__ __forceinline__ float get1(const char* p, int type) {
  if (TYPE == kF32) return *reinterpret_cast<const float*>(p);
  return elem_from_bits(*reinterpret_cast<const uint16_t*>(p), TYPE == kAny16 ? type : TYPE);
}
template <int TYPE>
__device__ __forceinline__ void put1(char* p, int type, float v) {
  if (TYPE == kF32) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(elem_to_bits(v, TYPE == kAny16 ? type : TYPE));
}

// ---------------------------------------------------------------------------
// columns of a thread. VEC: chunk k begins at first + k kWarpCols; else its
// element e is at first + (4 k + e) 32.
// ---------------------------------------------------------------------------
template <int V, bool VEC>
struct Columns {
  int first;
  int count;                                   // of chunks (VEC) or elements below n
  __device__ __forceinline__ Columns(int t, int n) {
    const int lane = t & 31, warp = t >> 5;
    first = warp * V * kWarpCols + (VEC ? lane * kChunk : lane);
    count = VEC ? max(0, (n - first + kWarpCols - 1) / kWarpCols) : max(0, (n - first + 31) / 32);
  }
  __device__ __forceinline__ bool has(int k, int e) const { return VEC ? k < count : k * kChunk + e < count; }
  __device__ __forceinline__ bool full() const { return count >= (VEC ? V : V * kChunk); }
};

// Chunk k of a row in shared memory as floats; what lies behind the n columns
// there is zero.
template <int TYPE, int V, bool VEC>
__device__ __forceinline__ void read_chunk(uint32_t row, int type, const Columns<V, VEC>& c, int k, F2& a, F2& b) {
  constexpr int es = kBytes<TYPE>;
  const char* p = smem() + (row + c.first * es) + k * kWarpCols * es;
  if (VEC) {
    get4<TYPE>(p, type, a, b);
  } else {
    a = f2(get1<TYPE>(p, type), get1<TYPE>(p + 32 * es, type));
    b = f2(get1<TYPE>(p + 64 * es, type), get1<TYPE>(p + 96 * es, type));
  }
}
// A thread's part of a row in memory, as raw words: what several tensors' loads
// need is in flight before the first is converted. Nothing at or past n is read.
template <int V, bool VEC>
struct RawRow {
  uint32_t w[V * kChunk];
  __device__ __forceinline__ void load(const void* row, int type, const Columns<V, VEC>& c) {
    const int es = elem_bytes(type);
    const char* p = static_cast<const char*>(row) + c.first * es;
#pragma unroll
    for (int i = 0; i < V * kChunk; ++i) w[i] = 0u;
    if (row == nullptr) return;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (VEC) {
        if (!c.has(k, 0)) continue;
        if (type == kF32) {
          const uint4 a = *reinterpret_cast<const uint4*>(p + k * kWarpCols * 4);
          w[4 * k] = a.x; w[4 * k + 1] = a.y; w[4 * k + 2] = a.z; w[4 * k + 3] = a.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(p + k * kWarpCols * 2);
          w[4 * k] = a.x; w[4 * k + 1] = a.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          if (!c.has(k, e)) continue;
          if (type == kF32) w[4 * k + e] = *reinterpret_cast<const uint32_t*>(p + (k * kChunk + e) * 128);
          else w[4 * k + e] = *reinterpret_cast<const uint16_t*>(p + (k * kChunk + e) * 64);
        }
      }
    }
  }
  __device__ __forceinline__ void convert(int type, F2* x) const {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (VEC && type != kF32) {
        float v[8];
        unpack8(&w[4 * k], type, v);           // the second half is not used
        x[2 * k] = f2(v[0], v[1]);
        x[2 * k + 1] = f2(v[2], v[3]);
      } else {
        x[2 * k] = f2(elem_from_bits(w[4 * k], type), elem_from_bits(w[4 * k + 1], type));
        x[2 * k + 1] = f2(elem_from_bits(w[4 * k + 2], type), elem_from_bits(w[4 * k + 3], type));
      }
    }
  }
};

// Writes chunk k; columns at or past n are left alone. Single elements: FULL,
// where the thread has all of its columns, saves a comparison for each.
template <int TYPE, int V, bool VEC, bool FULL>
__device__ __forceinline__ void write_chunk(char* row, int type, const Columns<V, VEC>& c, int k, F2 a, F2 b) {
  constexpr int es = kBytes<TYPE>;
  char* to = row + c.first * es + k * kWarpCols * es;
  if (VEC) {
    put4<TYPE>(to, type, c.has(k, 0), a, b);
  } else {
    const float2 p = split(a), q = split(b);
    if (FULL || c.has(k, 0)) put1<TYPE>(to, type, p.x);
    if (FULL || c.has(k, 1)) put1<TYPE>(to + 32 * es, type, p.y);
    if (FULL || c.has(k, 2)) put1<TYPE>(to + 64 * es, type, q.x);
    if (FULL || c.has(k, 3)) put1<TYPE>(to + 96 * es, type, q.y);
  }
}
template <int TYPE, int V, bool VEC>
__device__ __forceinline__ void write_typed(char* row, int type, const Columns<V, VEC>& c, const F2* x) {
  if (!VEC && c.full()) {
#pragma unroll
    for (int k = 0; k < V; ++k) write_chunk<TYPE, V, VEC, true>(row, type, c, k, x[2 * k], x[2 * k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) write_chunk<TYPE, V, VEC, false>(row, type, c, k, x[2 * k], x[2 * k + 1]);
  }
}
// Writes a thread's part of a row.
template <int V, bool VEC>
__device__ __forceinline__ void write_row(char* row, int type, const Columns<V, VEC>& c, const F2* x) {
  if (type == kF32) write_typed<kF32, V, VEC>(row, type, c, x);
  else if (type == kBf16) write_typed<kBf16, V, VEC>(row, type, c, x);
  else write_typed<kF16, V, VEC>(row, type, c, x);
}

// Parameters as fp32 in shared memory, zeros from n to `width`.
template <bool VEC>
__device__ __forceinline__ void stage_params(float* to, const void* p, int type, int n, int width, float fill) {
  if (VEC) {
    for (int i = threadIdx.x * kChunk; i < width; i += blockDim.x * kChunk) {
      F2 a = f2(i < n ? fill : 0.0f), b = a;
      if (p != nullptr && i < n) {
        const char* from = static_cast<const char*>(p) + i * elem_bytes(type);
        if (type == kF32) get4<kF32>(from, type, a, b);
        else get4<kAny16>(from, type, a, b);
      }
      *reinterpret_cast<ulonglong2*>(to + i) = make_ulonglong2(a.v, b.v);
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < width; i += blockDim.x)
      to[i] = i >= n ? 0.0f : p != nullptr ? load_elem(p, i, type) : fill;
  }
}
template <int V, bool VEC>
__device__ __forceinline__ void param_chunk(uint32_t p, const Columns<V, VEC>& c, int k, F2& a, F2& b) {
  read_chunk<kF32, V, VEC>(p, kF32, c, k, a, b);
}

// ---------------------------------------------------------------------------
// teams
// ---------------------------------------------------------------------------
__device__ __forceinline__ void team_sync(int T, int team) {
  if (T <= 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(T) : "memory");
}

// Sums over a team's threads. T: a power of two up to 32, or a multiple of 32
// (then scratch holds a float per value and warp of the block).
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int T, int team, float* scratch) {
  const int w = T < 32 ? T : 32;
#pragma unroll
  for (int i = 0; i < N; ++i)
    for (int o = w >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (T > 32) {
    const int warps = T >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) scratch[i * 32 + (threadIdx.x >> 5)] = v[i];
    }
    team_sync(T, team);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float* s = scratch + i * 32 + team * warps;
      v[i] = s[0];
      for (int k = 1; k < warps; ++k) v[i] += s[k];
    }
  }
}

// ---------------------------------------------------------------------------
// the ring
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(uint32_t offset) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(smem())) + offset;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_cut(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `newer` of this thread's groups have arrived.
__device__ __forceinline__ void copy_wait(int newer) {
  switch (newer) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// Starts the copy of a row that begins at src into its place in the ring.
// first_row: nothing before src belongs to the tensor.
template <int ES, int V, bool VEC>
__device__ __forceinline__ void fetch_row(uint32_t stage, const char* src, bool first_row, int n, int t, int T) {
  constexpr int es = ES;
  if (VEC) {
    const int at = (t >> 5) * V * kWarpCols * es + (t & 31) * 16;
    const int end = min(n * es, ((t >> 5) + 1) * V * kWarpCols * es) - at;
#pragma unroll
    for (int i = 0; i < (es == 4 ? V : (V + 1) / 2); ++i)
      if (i * 512 < end) copy16(stage + at + i * 512, src + at + i * 512);
  } else {
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15u);
    const int end = shift + n * es;            // of the row, from its first granule on
    const char* from = src - shift;
    const bool cut = first_row && shift != 0;  // the first granule begins before the tensor
    const int whole = end / 16 * 16;
#pragma unroll 1
    for (int g = (t == 0 && cut ? T : t) * 16; g < whole; g += T * 16) copy16(stage + g, from + g);
    if (t == 0 && cut) {
      for (int b = shift; b < min(end, 16); b += es) {
        if (es == 4)
          *reinterpret_cast<uint32_t*>(smem() + stage + b) = *reinterpret_cast<const uint32_t*>(from + b);
        else
          *reinterpret_cast<uint16_t*>(smem() + stage + b) = *reinterpret_cast<const uint16_t*>(from + b);
      }
    }
    // the granule in which the row ends, filled up with zeros, and one of zeros
    // over what a row that started later in its first granule left there
    if (t == T - 1) {
      const bool open = end > whole && !(cut && whole == 0);
      if (open) copy16_cut(stage + whole, from + whole, end - whole);
      copy16_cut(stage + (end + 15) / 16 * 16, from, 0);
    }
  }
}
// Zeros from byte `used` to byte `width` of every row of a ring (whole granules).
__device__ __forceinline__ void clear_tails(char* rows, int row_count, int stage_bytes, int used, int width) {
  const int words = (width - used) / 16;
  for (int i = threadIdx.x; i < row_count * words; i += blockDim.x)
    *reinterpret_cast<uint4*>(rows + static_cast<size_t>(i / words) * stage_bytes + used + i % words * 16) =
        make_uint4(0u, 0u, 0u, 0u);
}
// Between the arrival of a row and its first read: VEC rows are copied and read
// by the same warp.
template <bool VEC>
__device__ __forceinline__ void arrive_sync(int T, int team) {
  if (VEC) __syncwarp();
  else team_sync(T, team);
}
__device__ __forceinline__ int granule_shift(const void* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Mean and rstd of a row held in registers; x becomes x - mean.
template <int V, bool VEC>
__device__ __forceinline__ void row_stats(F2 (&x)[2 * V], const Columns<V, VEC>& c, float inv_n, float eps, int T,
                                          int team, float* scratch, float* mean_out, float* rstd_out) {
  F2 a = x[0], b = x[1];
#pragma unroll
  for (int k = 1; k < V; ++k) {
    a = a + x[2 * k];
    b = b + x[2 * k + 1];
  }
  float s[1] = {both(a + b)};
  team_sum<1>(s, T, team, scratch);
  const float mean = s[0] * inv_n;
  a = b = f2(0.0f);
  if (!VEC && c.full()) {
    const F2 m = f2(-mean);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x[2 * k] = x[2 * k] + m;
      x[2 * k + 1] = x[2 * k + 1] + m;
      a = fma2(x[2 * k], x[2 * k], a);
      b = fma2(x[2 * k + 1], x[2 * k + 1], b);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {              // zeros behind n stay zeros
      F2 mp, mq;
      if (VEC) {
        mp = mq = f2(c.has(k, 0) ? -mean : 0.0f);
      } else {
        mp = f2(c.has(k, 0) ? -mean : 0.0f, c.has(k, 1) ? -mean : 0.0f);
        mq = f2(c.has(k, 2) ? -mean : 0.0f, c.has(k, 3) ? -mean : 0.0f);
      }
      x[2 * k] = x[2 * k] + mp;
      x[2 * k + 1] = x[2 * k + 1] + mq;
      a = fma2(x[2 * k], x[2 * k], a);
      b = fma2(x[2 * k + 1], x[2 * k + 1], b);
    }
  }
  s[0] = both(a + b);
  team_sum<1>(s, T, team, scratch + 32);       // another part: no barrier between the reads and these writes
  *mean_out = mean;
  *rstd_out = rsqrtf(s[0] * inv_n + eps);      // within 2 units in the last place
}

template <int TX, int V, bool VEC>
__global__ void __launch_bounds__(kBlock, 1)
    layer_norm_kernel(const __grid_constant__ LayerNormJob j, const __grid_constant__ RowShape r) {
  char* ring = smem();
  __shared__ float scratch[2 * 32];
  const int T = r.T, team = threadIdx.x / T, t = threadIdx.x - team * T;
  const int n = static_cast<int>(j.n);
  const float inv_n = 1.0f / static_cast<float>(n);
  const bool idle = team >= r.teams;           // threads behind the last whole team: touch nothing
  float* weight = reinterpret_cast<float*>(ring + r.params);
  const int width = max(T, 32) / 32 * V * kWarpCols;     // columns of a team's slots
  float* bias = weight + width;
  const uint32_t mine = static_cast<uint32_t>(min(team, r.teams - 1) * r.stages * r.stage_bytes);
  const Columns<V, VEC> c(t, n);
  const int64_t step = static_cast<int64_t>(gridDim.x) * r.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * r.teams + team;
  const int64_t ahead = step * (r.stages - 1);
  const int64_t x_step = step * j.ld_x * elem_bytes(j.x_type), y_step = step * j.ld_y * elem_bytes(j.y_type);
  const char* next = static_cast<const char*>(row_ptr(j.x, row, j.ld_x, j.x_type));
  const char* here = next;
  char* y = static_cast<char*>(row_ptr(j.y, row, j.ld_y, j.y_type));
  const auto fetch = [&](int slot, int64_t which) {
    if (which < j.tokens && !idle) fetch_row<kBytes<TX>, V, VEC>(mine + slot * r.stage_bytes, next, which == 0, n, t, T);
    copy_commit();
    next += x_step;
  };
  clear_tails(ring, r.teams * r.stages, r.stage_bytes, n * elem_bytes(j.x_type) / 16 * 16, r.stage_bytes);
  if (!VEC) __syncthreads();                   // copies write there too, later
  for (int s = 0; s + 1 < r.stages; ++s) fetch(s, row + s * step);
  stage_params<VEC>(weight, j.weight, j.param_type, n, width, 1.0f);
  stage_params<VEC>(bias, j.bias, j.param_type, n, width, 0.0f);
  __syncthreads();
  if (T > 32 && idle) return;
  int slot = 0;
  // threads of one warp leave together: the block's first team decides
  for (int64_t base = row - team; base < j.tokens; base += step, row += step, here += x_step, y += y_step) {
    const bool live = row < j.tokens && !idle;
    fetch(slot == 0 ? r.stages - 1 : slot - 1, row + ahead);
    copy_wait(r.stages - 1);
    arrive_sync<VEC>(T, team);
    F2 x[2 * V];
    if (live) {
      const uint32_t stage = mine + slot * r.stage_bytes + (VEC ? 0 : granule_shift(here));
#pragma unroll
      for (int k = 0; k < V; ++k) read_chunk<TX, V, VEC>(stage, j.x_type, c, k, x[2 * k], x[2 * k + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) x[i] = f2(0.0f);
    }
    slot = slot + 1 == r.stages ? 0 : slot + 1;
    float mean, rstd;
    row_stats<V, VEC>(x, c, inv_n, j.eps, T, team, scratch, &mean, &rstd);
    if (T <= 32) __syncwarp();                 // every lane has read the slot that the next copy may take
    if (!live) continue;
    if (t == 0) {
      if (j.mean != nullptr) j.mean[row] = mean;
      if (j.rstd != nullptr) j.rstd[row] = rstd;
    }
    const F2 scale = f2(rstd);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      F2 wa, wb, ba, bb;
      param_chunk<V, VEC>(r.params, c, k, wa, wb);
      param_chunk<V, VEC>(r.params + width * 4, c, k, ba, bb);
      x[2 * k] = fma2(x[2 * k] * scale, wa, ba);
      x[2 * k + 1] = fma2(x[2 * k + 1] * scale, wb, bb);
    }
    write_row<V, VEC>(y, j.y_type, c, x);
  }
}

// One row a team and few rows: straight from memory, no ring, no parameters in
// shared memory. What counts is the depth of dependent loads: one.
template <int V, bool VEC>
__global__ void __launch_bounds__(kMaxRowT)
    layer_norm_row_kernel(const __grid_constant__ LayerNormJob j, const __grid_constant__ RowShape r) {
  __shared__ float scratch[2 * 32];
  const int T = r.T, team = threadIdx.x / T, t = threadIdx.x - team * T;
  const int n = static_cast<int>(j.n);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * r.teams + team;
  const bool live = team < r.teams && row < j.tokens;
  if (T > 32 && !live) return;
  const Columns<V, VEC> c(t, live ? n : 0);
  RawRow<V, VEC> rx, rw, rb;
  rx.load(row_ptr(j.x, live ? row : 0, j.ld_x, j.x_type), j.x_type, c);
  rw.load(j.weight, j.param_type, c);
  rb.load(j.bias, j.param_type, c);
  F2 x[2 * V], p[2 * V];
  rx.convert(j.x_type, x);
  float mean, rstd;
  row_stats<V, VEC>(x, c, 1.0f / static_cast<float>(n), j.eps, T, team, scratch, &mean, &rstd);
  if (!live) return;
  if (t == 0) {
    if (j.mean != nullptr) j.mean[row] = mean;
    if (j.rstd != nullptr) j.rstd[row] = rstd;
  }
  const F2 scale = f2(rstd);
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) x[i] = x[i] * scale;
  if (j.weight != nullptr) {
    rw.convert(j.param_type, p);
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) x[i] = x[i] * p[i];
  }
  if (j.bias != nullptr) {
    rb.convert(j.param_type, p);
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) x[i] = x[i] + p[i];
  }
  write_row<V, VEC>(static_cast<char*>(row_ptr(j.y, row, j.ld_y, j.y_type)), j.y_type, c, x);
}

// Rows too wide for registers: a block per row, three walks over it (the later
// ones served by L1 and L2).
__global__ void __launch_bounds__(kWideThreads) layer_norm_wide_kernel(const __grid_constant__ LayerNormJob j) {
  __shared__ float scratch[2][32];
  for (int64_t row = blockIdx.x; row < j.tokens; row += gridDim.x) {
    const void* x = row_ptr(j.x, row, j.ld_x, j.x_type);
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) s[0] += load_elem(x, c, j.x_type);
    team_sum<1>(s, kWideThreads, 0, scratch[0]);
    const float mean = s[0] / static_cast<float>(j.n);
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float v = load_elem(x, c, j.x_type) - mean;
      s[0] = fmaf(v, v, s[0]);
    }
    team_sum<1>(s, kWideThreads, 0, scratch[1]);
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

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Every thread keeps the sums of its columns of dy xh and dy in registers over
// all its rows; at the end the block's teams are joined in shared memory, in a
// fixed order, and written once, as row blockIdx.x of partial
// ([blocks][2][n]). Up to kHoldV chunks a thread, xh and g stay in registers
// between the row sums and dx; above, the ring is read a second time.
template <int TX, int TY, int V, bool VEC>
__global__ void __launch_bounds__(kBlock, 1)
    layer_norm_backward_kernel(const __grid_constant__ LayerNormBackwardJob j, const __grid_constant__ RowShape r,
                               float* partial) {
  char* ring = smem();
  __shared__ float scratch[2][2 * 32];
  constexpr bool kHold = V <= kHoldV;
  const int T = r.T, team = threadIdx.x / T, t = threadIdx.x - team * T;
  const int n = static_cast<int>(j.n);
  const float inv_n = 1.0f / static_cast<float>(n);
  const bool idle = team >= r.teams;           // threads behind the last whole team: touch nothing
  float* weight = reinterpret_cast<float*>(ring + r.params);
  const uint32_t mine = static_cast<uint32_t>(min(team, r.teams - 1) * r.stages * r.stage_bytes);
  const Columns<V, VEC> c(t, n);
  const int64_t step = static_cast<int64_t>(gridDim.x) * r.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * r.teams + team;
  const int64_t ahead = step * (r.stages - 1);
  const int64_t x_step = step * j.ld_x * elem_bytes(j.x_type), dy_step = step * j.ld_dy * elem_bytes(j.dy_type);
  const int64_t dx_step = step * j.ld_dx * elem_bytes(j.dx_type);
  const char* next_x = static_cast<const char*>(row_ptr(j.x, row, j.ld_x, j.x_type));
  const char* next_dy = static_cast<const char*>(row_ptr(j.dy, row, j.ld_dy, j.dy_type));
  const char* here_x = next_x;
  const char* here_dy = next_dy;
  char* dx = j.dx != nullptr ? static_cast<char*>(row_ptr(j.dx, row, j.ld_dx, j.dx_type)) : nullptr;
  const auto fetch = [&](int slot, int64_t which) {
    if (which < j.tokens && !idle) {
      const uint32_t stage = mine + slot * r.stage_bytes;
      fetch_row<kBytes<TX>, V, VEC>(stage, next_x, which == 0, n, t, T);
      fetch_row<kBytes<TY>, V, VEC>(stage + r.second, next_dy, which == 0, n, t, T);
    }
    copy_commit();
    next_x += x_step;
    next_dy += dy_step;
  };
  const int width = max(T, 32) / 32 * V * kWarpCols;     // columns of a team's slots
  clear_tails(ring, r.teams * r.stages, r.stage_bytes, n * elem_bytes(j.x_type) / 16 * 16, r.second);
  clear_tails(ring + r.second, r.teams * r.stages, r.stage_bytes, n * elem_bytes(j.dy_type) / 16 * 16,
              r.stage_bytes - r.second);
  if (!VEC) __syncthreads();                   // copies write there too, later
  for (int s = 0; s + 1 < r.stages; ++s) fetch(s, row + s * step);
  const auto stat = [&](const float* p, int64_t at) { return at < j.tokens && !idle ? p[at] : 0.0f; };
  float mean = stat(j.mean, row), rstd = stat(j.rstd, row);
  stage_params<VEC>(weight, j.weight, j.param_type, n, width, 1.0f);
  __syncthreads();
  F2 dw[2 * V], db[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) dw[i] = db[i] = f2(0.0f);
  if (T <= 32 || !idle) {
    int slot = 0, flip = 0;
    for (int64_t base = row - team; base < j.tokens; base += step) {
      const bool live = row < j.tokens && !idle;
      fetch(slot == 0 ? r.stages - 1 : slot - 1, row + ahead);
      const F2 m = f2(-mean), scale = f2(rstd);
      mean = stat(j.mean, row + step);         // a row ahead, like the ring
      rstd = stat(j.rstd, row + step);
      copy_wait(r.stages - 1);
      arrive_sync<VEC>(T, team);
      const uint32_t sx = mine + slot * r.stage_bytes + (VEC ? 0 : granule_shift(here_x));
      const uint32_t sy = mine + slot * r.stage_bytes + r.second + (VEC ? 0 : granule_shift(here_dy));
      F2 xh[kHold ? 2 * V : 2], g[kHold ? 2 * V : 2], s0 = f2(0.0f), s1 = f2(0.0f);
      // xh, dy and w of chunk k
      const auto load = [&](int k, F2* px, F2* py, F2* pw) {
        read_chunk<TX, V, VEC>(sx, j.x_type, c, k, px[0], px[1]);
        read_chunk<TY, V, VEC>(sy, j.dy_type, c, k, py[0], py[1]);
        param_chunk<V, VEC>(r.params, c, k, pw[0], pw[1]);
        px[0] = (px[0] + m) * scale;
        px[1] = (px[1] + m) * scale;
      };
      if (live) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          F2* px = xh + (kHold ? 2 * k : 0);
          F2* pg = g + (kHold ? 2 * k : 0);
          F2 dy[2], w[2];
          load(k, px, dy, w);
          // columns past n: dy is zero there, and xh is finite (x = 0)
          pg[0] = dy[0] * w[0];
          pg[1] = dy[1] * w[1];
          s0 = s0 + (pg[0] + pg[1]);
          s1 = fma2(pg[0], px[0], fma2(pg[1], px[1], s1));
          dw[2 * k] = fma2(dy[0], px[0], dw[2 * k]);
          dw[2 * k + 1] = fma2(dy[1], px[1], dw[2 * k + 1]);
          db[2 * k] = db[2 * k] + dy[0];
          db[2 * k + 1] = db[2 * k + 1] + dy[1];
        }
      }
      if (j.dx != nullptr) {                   // uniform over the grid
        float s[2] = {both(s0), both(s1)};
        team_sum<2>(s, T, team, scratch[flip]);
        flip ^= 1;
        const F2 c1 = f2(-s[0] * inv_n), c2 = f2(-s[1] * inv_n);
        if (live) {
          const auto finish = [&](auto td) {
            constexpr int TD = decltype(td)::value;
            if constexpr (kHold) {
#pragma unroll
              for (int i = 0; i < 2 * V; ++i) xh[i] = scale * fma2(xh[i], c2, g[i] + c1);
              write_typed<TD, V, VEC>(dx, j.dx_type, c, xh);
            } else {
#pragma unroll
              for (int k = 0; k < V; ++k) {
                F2 dy[2], w[2];
                load(k, xh, dy, w);
                write_chunk<TD, V, VEC, false>(dx, j.dx_type, c, k, scale * fma2(xh[0], c2, fma2(dy[0], w[0], c1)),
                                               scale * fma2(xh[1], c2, fma2(dy[1], w[1], c1)));
              }
            }
          };
          if (j.dx_type == kF32) finish(std::integral_constant<int, kF32>{});
          else finish(std::integral_constant<int, TX == kF32 ? kAny16 : TX>{});
        }
      }
      arrive_sync<VEC>(T, team);               // the slot is free for the next copy
      slot = slot + 1 == r.stages ? 0 : slot + 1;
      row += step;
      here_x += x_step;
      here_dy += dy_step;
      if (dx != nullptr) dx += dx_step;
    }
  }
  if (partial == nullptr) return;
  if (r.teams == 1 && T >= 32) {               // nothing to join
    if (idle) return;
    char* out = reinterpret_cast<char*>(partial + static_cast<int64_t>(blockIdx.x) * 2 * n);
    write_typed<kF32, V, VEC>(out, kF32, c, dw);
    write_typed<kF32, V, VEC>(out + static_cast<size_t>(n) * 4, kF32, c, db);
    return;
  }
  copy_wait(0);
  __syncthreads();                             // the ring becomes the teams' sums: [team][2][width]
  float* sums = reinterpret_cast<float*>(ring);
  int rows = r.teams;
  if (T < 32) {                                // teams of one warp first
    rows = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < 2 * V; ++i)
      for (int o = T; o < 32; o <<= 1) {
        F2 p, q;
        p.v = __shfl_xor_sync(0xffffffffu, dw[i].v, o);
        q.v = __shfl_xor_sync(0xffffffffu, db[i].v, o);
        dw[i] = dw[i] + p;
        db[i] = db[i] + q;
      }
  }
  if (T >= 32 ? !idle : (threadIdx.x & 31) < T) {
    float2* to = reinterpret_cast<float2*>(sums + static_cast<size_t>(T >= 32 ? team : threadIdx.x >> 5) * 2 * width) + t;
    const int lanes = max(T, 32);
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      to[i * lanes] = split(dw[i]);
      to[width / 2 + i * lanes] = split(db[i]);
    }
  }
  __syncthreads();
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * n;
  for (int col = threadIdx.x; col < 2 * n; col += blockDim.x) {
    const int cc = col < n ? col : col - n;
    // thread, pair and half that hold column cc
    const int in = cc % (V * kWarpCols), warp = cc / (V * kWarpCols);
    const int elem = VEC ? in / kWarpCols * kChunk + in % kChunk : in / 32;
    const int lane = VEC ? in % kWarpCols / kChunk : in % 32;
    const int at = ((elem >> 1) * max(T, 32) + warp * 32 + lane) * 2 + (elem & 1) + (col < n ? 0 : width);
    float s = sums[at];
    for (int k = 1; k < rows; ++k) s += sums[static_cast<size_t>(k) * 2 * width + at];
    out[col] = s;
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
    team_sum<2>(s, kWideThreads, 0, scratch[flip]);
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

bool rows_aligned(const void* p, int64_t ld, int64_t n, int type) {
  const int es = elem_bytes(type);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && n * es % 16 == 0;
}

unsigned grid_of(int64_t blocks, int64_t cap) { return static_cast<unsigned>(std::max<int64_t>(1, std::min(blocks, cap))); }

// Bytes of one row of a tensor in the ring: the team's columns; where the row
// may start inside its first granule, one granule more and one of zeros.
int64_t slot_columns(const RowShape& r) { return int64_t{std::max(r.T, 32)} / 32 * r.V * kWarpCols; }
int ring_bytes(const RowShape& r, int type, bool vec) {
  return static_cast<int>(slot_columns(r) * elem_bytes(type) + (vec ? 0 : 48));
}

// What a kernel asks of the search below.
struct RowWant {
  int64_t tokens, n;
  bool vec;
  int max_v;
  int type, second_type;                       // second_type < 0: one tensor
  int params;                                  // fp32 vectors of a row's columns in shared memory
};

// Places teams and ring of a block for a given T and V: as many teams as rows
// call for and shared memory holds with a ring of two rows each, whole warps of
// them. False: not even one.
bool place_ring(const RowWant& q, RowShape* r) {
  const int first = ring_bytes(*r, q.type, q.vec);
  r->second = first;
  r->stage_bytes = first + (q.second_type < 0 ? 0 : ring_bytes(*r, q.second_type, q.vec));
  const int64_t smem = kSmemPerSm - q.params * slot_columns(*r) * static_cast<int64_t>(sizeof(float));
  if (smem < r->stage_bytes) return false;
  int64_t teams = std::min<int64_t>(kBlock / r->T, (q.tokens + kSms - 1) / kSms);
  teams = std::max<int64_t>(1, std::min<int64_t>(teams, smem / (2 * int64_t{r->stage_bytes})));
  if (r->T < 32 && teams * r->T > 32) teams = teams * r->T / 32 * 32 / r->T;
  r->teams = static_cast<int>(teams);
  r->stages = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxStages, smem / (teams * r->stage_bytes))));
  r->params = r->teams * r->stages * r->stage_bytes;
  return true;
}

// Teams for rows of n columns. VEC rows of up to 16 chunks: one chunk a thread,
// several teams a warp. Else whole warps of V chunks a thread, for the V for which
// kernels exist: the least of
//   rounds x (share of the block's threads at work x (V + 8) + V + 12)
// where a round is a row for every team: a row costs a thread the issue slots of
// its V chunks and of about 8 more (sums across threads, root, addresses), and
// the wait of a chain as long as V and about 12 more. Measured, us:
//   forward   16384 x 320 fp16    V = 1, 3, 8, 16: 22.7, 8.5, 13.3, 19.9
//             8192 x 4096 bf16    V = 1, 4, 8, 16: 159, 44, 34, 28.5
//   backward  8192 x 4096         V = 2, 4, 8: 96, 72, 63
//             32768 x 1280 bf16   V = 1, 4, 5, 8: 232, 76, 61, 80
//             333 x 1001          V = 1, 2, 4, 8: 10.3, 9.2, 10.7, 13.8
bool row_shape(const RowWant& q, RowShape* best) {
  const int64_t chunks = (q.n + kChunk - 1) / kChunk;
  if (chunks <= 16 && q.vec) {
    best->V = 1;
    best->T = 1;
    while (best->T < chunks) best->T *= 2;
    return place_ring(q, best);
  }
  double least = -1.0;
  for (int v : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16}) {
    if (v > q.max_v) break;
    if (!q.vec && v != 1 && v != 2 && v != 4 && v != 8 && !(v == 6 && q.second_type >= 0)) continue;
    RowShape r;
    const int64_t t = (chunks + 32 * v - 1) / (32 * v) * 32;
    if (t > kBlock) continue;
    r.T = static_cast<int>(t);
    r.V = v;
    if (!place_ring(q, &r)) continue;
    const int64_t rounds = (q.tokens + int64_t{kSms} * r.teams - 1) / (int64_t{kSms} * r.teams);
    const double cost = static_cast<double>(rounds) * (static_cast<double>(r.teams * r.T) / kBlock * (v + 8) + v + 12.0);
    if (least < 0.0 || cost <= least) {
      least = cost;
      *best = r;
    }
  }
  return least >= 0.0;
}

// One row a team of up to kMaxRowT threads and V chunks: 1, 2 or 4, the
// narrowest slices that hold the row.
bool single_row_shape(int64_t n, RowShape* r) {
  const int64_t chunks = (n + kChunk - 1) / kChunk;
  for (int v : {1, 2, 4}) {
    const int64_t t = (chunks + 32 * v - 1) / (32 * v) * 32;
    if (t > (v == 4 ? kMaxRowT : kMaxRowT / 2)) continue;
    r->T = static_cast<int>(t);
    r->V = v;
    r->teams = std::max(1, 128 / r->T);
    return true;
  }
  return false;
}

// Lets a kernel take the ring's share of shared memory; asked for once per
// kernel and device (`done`: a bit per device), since the call costs more than a
// launch.
cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemPerSm));
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int TX, int V, bool VEC>
cudaError_t launch_fwd(const LayerNormJob& j, const RowShape& r, unsigned grid, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(layer_norm_kernel<TX, V, VEC>), &done);
  if (e != cudaSuccess) return e;
  layer_norm_kernel<TX, V, VEC><<<grid, r.threads(), smem, s>>>(j, r);
  return counted(cudaGetLastError());
}
template <int TX, int TY, int V, bool VEC>
cudaError_t launch_bwd(const LayerNormBackwardJob& j, const RowShape& r, unsigned grid, size_t smem, float* partial,
                       cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(layer_norm_backward_kernel<TX, TY, V, VEC>), &done);
  if (e != cudaSuccess) return e;
  layer_norm_backward_kernel<TX, TY, V, VEC><<<grid, r.threads(), smem, s>>>(j, r, partial);
  return counted(cudaGetLastError());
}

// The V of row_shape.
template <int TX>
cudaError_t fwd_by_v(const LayerNormJob& j, const RowShape& r, bool vec, unsigned grid, size_t smem, cudaStream_t s) {
  switch (vec ? r.V : -r.V) {
    case 1: return launch_fwd<TX, 1, true>(j, r, grid, smem, s);
    case 2: return launch_fwd<TX, 2, true>(j, r, grid, smem, s);
    case 3: return launch_fwd<TX, 3, true>(j, r, grid, smem, s);
    case 4: return launch_fwd<TX, 4, true>(j, r, grid, smem, s);
    case 5: return launch_fwd<TX, 5, true>(j, r, grid, smem, s);
    case 6: return launch_fwd<TX, 6, true>(j, r, grid, smem, s);
    case 8: return launch_fwd<TX, 8, true>(j, r, grid, smem, s);
    case 10: return launch_fwd<TX, 10, true>(j, r, grid, smem, s);
    case 12: return launch_fwd<TX, 12, true>(j, r, grid, smem, s);
    case 16: return launch_fwd<TX, 16, true>(j, r, grid, smem, s);
    case -1: return launch_fwd<TX, 1, false>(j, r, grid, smem, s);
    case -2: return launch_fwd<TX, 2, false>(j, r, grid, smem, s);
    case -4: return launch_fwd<TX, 4, false>(j, r, grid, smem, s);
    case -8: return launch_fwd<TX, 8, false>(j, r, grid, smem, s);
  }
  return cudaErrorInvalidConfiguration;
}
template <int TX, int TY>
cudaError_t bwd_by_v(const LayerNormBackwardJob& j, const RowShape& r, bool vec, unsigned grid, size_t smem,
                     float* partial, cudaStream_t s) {
  switch (vec ? r.V : -r.V) {
    case 1: return launch_bwd<TX, TY, 1, true>(j, r, grid, smem, partial, s);
    case 2: return launch_bwd<TX, TY, 2, true>(j, r, grid, smem, partial, s);
    case 3: return launch_bwd<TX, TY, 3, true>(j, r, grid, smem, partial, s);
    case 4: return launch_bwd<TX, TY, 4, true>(j, r, grid, smem, partial, s);
    case 5: return launch_bwd<TX, TY, 5, true>(j, r, grid, smem, partial, s);
    case 6: return launch_bwd<TX, TY, 6, true>(j, r, grid, smem, partial, s);
    case 8: return launch_bwd<TX, TY, 8, true>(j, r, grid, smem, partial, s);
    case -1: return launch_bwd<TX, TY, 1, false>(j, r, grid, smem, partial, s);
    case -2: return launch_bwd<TX, TY, 2, false>(j, r, grid, smem, partial, s);
    case -4: return launch_bwd<TX, TY, 4, false>(j, r, grid, smem, partial, s);
    case -6: return launch_bwd<TX, TY, 6, false>(j, r, grid, smem, partial, s);
    case -8: return launch_bwd<TX, TY, 8, false>(j, r, grid, smem, partial, s);
  }
  return cudaErrorInvalidConfiguration;
}
cudaError_t bwd_by_type(const LayerNormBackwardJob& j, const RowShape& r, bool vec, unsigned grid, size_t smem,
                        float* partial, cudaStream_t s) {
  const bool x32 = j.x_type == kF32, y32 = j.dy_type == kF32;
  // bf16 has kernels of its own, where dx is bf16 or fp32 too; the other pairs
  // with 16-bit types select between the conversions
  if (j.x_type == kBf16 && j.dx_type != kF16) {
    if (j.dy_type == kBf16) return bwd_by_v<kBf16, kBf16>(j, r, vec, grid, smem, partial, s);
    if (y32) return bwd_by_v<kBf16, kF32>(j, r, vec, grid, smem, partial, s);
  }
  if (x32 && y32) return bwd_by_v<kF32, kF32>(j, r, vec, grid, smem, partial, s);
  if (x32) return bwd_by_v<kF32, kAny16>(j, r, vec, grid, smem, partial, s);
  if (y32) return bwd_by_v<kAny16, kF32>(j, r, vec, grid, smem, partial, s);
  return bwd_by_v<kAny16, kAny16>(j, r, vec, grid, smem, partial, s);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormJob& j, cudaStream_t s) {
  const bool vec = rows_aligned(j.x, j.ld_x, j.n, j.x_type) && rows_aligned(j.y, j.ld_y, j.n, j.y_type) &&
                   reinterpret_cast<uintptr_t>(j.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(j.bias) % 16 == 0;
  RowShape r;
  // Few rows: no ring. Single elements leave the ring a smaller lead: 1031 x 5003
  // takes 12.4 us this way and 18.7 with it.
  if (j.tokens <= (vec ? 1 : 8) * kSms && single_row_shape(j.n, &r)) {
    const unsigned grid = static_cast<unsigned>((j.tokens + r.teams - 1) / r.teams);
    const int threads = r.threads();
    switch (r.V) {
      case 1:
        if (vec) layer_norm_row_kernel<1, true><<<grid, threads, 0, s>>>(j, r);
        else layer_norm_row_kernel<1, false><<<grid, threads, 0, s>>>(j, r);
        break;
      case 2:
        if (vec) layer_norm_row_kernel<2, true><<<grid, threads, 0, s>>>(j, r);
        else layer_norm_row_kernel<2, false><<<grid, threads, 0, s>>>(j, r);
        break;
      default:
        if (vec) layer_norm_row_kernel<4, true><<<grid, threads, 0, s>>>(j, r);
        else layer_norm_row_kernel<4, false><<<grid, threads, 0, s>>>(j, r);
        break;
    }
    return counted(cudaGetLastError());
  }
  if (!row_shape(RowWant{j.tokens, j.n, vec, kFwdMaxV, j.x_type, -1, 2}, &r)) {
    layer_norm_wide_kernel<<<grid_of(j.tokens, 1 << 20), kWideThreads, 0, s>>>(j);
    return counted(cudaGetLastError());
  }
  const unsigned grid = grid_of((j.tokens + r.teams - 1) / r.teams, kSms);
  const size_t smem = static_cast<size_t>(r.params) + 2 * static_cast<size_t>(slot_columns(r)) * sizeof(float);
  if (j.x_type == kF32) return fwd_by_v<kF32>(j, r, vec, grid, smem, s);
  if (j.x_type == kBf16) return fwd_by_v<kBf16>(j, r, vec, grid, smem, s);
  return fwd_by_v<kF16>(j, r, vec, grid, smem, s);
}

namespace {
// The number of partial sums depends on tokens and n alone, so that the
// workspace does: as many blocks as SMs, if there are rows for them. Rows too
// wide for the ring (two fp32 tensors, any alignment) go to the wide kernels.
struct BackwardSums {
  bool wide = false;
  int64_t blocks = 0;
};
BackwardSums backward_sums(int64_t tokens, int64_t n) {
  BackwardSums b;
  RowShape r;
  b.wide = !row_shape(RowWant{tokens, n, false, kBwdMaxV, kF32, kF32, 1}, &r) ||
           !row_shape(RowWant{tokens, n, true, kBwdMaxV, kF32, kF32, 1}, &r);
  const int64_t strips = (n + kColThreads - 1) / kColThreads;
  b.blocks = b.wide ? std::min<int64_t>(std::max<int64_t>(1, kSms * 8 / strips), std::max<int64_t>(1, tokens / 8))
                    : std::max<int64_t>(1, std::min<int64_t>(kSms, tokens));
  return b;
}
}  // namespace

size_t layer_norm_backward_ws(int64_t tokens, int64_t n) {
  const BackwardSums b = backward_sums(tokens, n);
  return (static_cast<size_t>(b.blocks) * 2 * static_cast<size_t>(n) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardJob& j, void* ws, cudaStream_t s) {
  const BackwardSums b = backward_sums(j.tokens, j.n);
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
  } else if (j.dx != nullptr || sums) {
    const bool vec = rows_aligned(j.x, j.ld_x, j.n, j.x_type) && rows_aligned(j.dy, j.ld_dy, j.n, j.dy_type) &&
                     (j.dx == nullptr || rows_aligned(j.dx, j.ld_dx, j.n, j.dx_type)) &&
                     reinterpret_cast<uintptr_t>(j.weight) % 16 == 0;
    RowShape r;
    // single elements take more registers: V = 8 spills (3000 x 5003: 65 us, V = 6 58)
    if (!row_shape(RowWant{j.tokens, j.n, vec, vec ? kBwdMaxV : 6, j.x_type, j.dy_type, 1}, &r) &&
        !row_shape(RowWant{j.tokens, j.n, vec, kBwdMaxV, j.x_type, j.dy_type, 1}, &r))
      return cudaErrorInvalidConfiguration;
    // the joined sums take the place of ring and parameters
    const size_t join = static_cast<size_t>(r.T >= 32 ? r.teams : r.threads() / 32) * 2 * slot_columns(r) * sizeof(float);
    const size_t smem = std::max(static_cast<size_t>(r.params) + static_cast<size_t>(slot_columns(r)) * sizeof(float), join);
    const cudaError_t e = bwd_by_type(j, r, vec, static_cast<unsigned>(b.blocks), smem, partial, s);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  layer_norm_reduce_kernel<<<static_cast<unsigned>((2 * j.n + 31) / 32), 32 * kReduceWarps, 0, s>>>(
      partial, b.blocks, j.n, j.dweight, j.dbias, j.accumulate);
  return counted(cudaGetLastError());
}

}  // namespace intlora
