// Rows of a tokens x n matrix in teams of threads, for the layer norm kernels:
// the shape of teams and rings, the ring itself, and the arithmetic on a thread's
// columns.
//
// Layer norm and its gradients are bound by memory as long as the instructions
// an element takes stay few: at 6.5 TB/s an SM has 22 issue slots for an element
// of the bf16 forward and 33 of the bf16 backward. So: every row is read from
// memory once; blocks are persistent, and their teams of T threads walk over the
// rows with a grid stride, copying the rows that come next into a ring in shared
// memory (cp.async: no registers, no wait that could fail to end) while they work
// on the present one; a warp of a team holds V x 128 neighbouring columns, so that
// its addresses are one base and constants; sums and products are done two at a
// time (f32x2); types are compile-time in the loops; the parameters are turned
// into fp32 in shared memory once per block. Teams of up to 32 threads never
// leave their warp; wider ones join their row sums through shared memory and a
// named barrier of their own, so that no team waits for another.
//
// Two ways through the ring:
//   VEC   rows start at 16-byte boundaries and fill whole 16-byte granules: a
//         warp copies its own columns; a thread works on chunks of 4 of them
//   else  (gradients alone; the forward needs no ring for such rows) the team
//         copies the row's granules, wherever the row starts in the first one, and
//         a thread works on single columns, 32 apart. A granule that begins before
//         the tensor is fetched element by element and one that ends behind the
//         row is cut short: nothing outside [first element, last element] of the
//         tensor is read.
#pragma once

#include <algorithm>
#include <atomic>

#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "intlora_kernels.h"
#include "train_ops.h"

namespace intlora {

namespace {

constexpr int kSms = 148;
constexpr int kChunk = 4;                      // elements of a chunk
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
  int T = 0, V = 0, L = 32;                    // threads of a team, chunks of a thread, lanes of a Form
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
// The form of a row at compile time: V chunks a thread, VEC or not, and the L
// lanes that share neighbouring chunks: 32, or 16 for two rows a warp (VEC).
// Columns of a thread. VEC: chunk k begins at first + k kCols; else its element
// e is at first + (4 k + e) 32.
// ---------------------------------------------------------------------------
template <int V_, bool VEC_, int L_ = 32>
struct Form {
  static constexpr int V = V_, L = L_;
  static constexpr bool VEC = VEC_;
  static constexpr int kCols = L * kChunk;     // columns of one chunk of the lanes
  static_assert(VEC || L == 32, "single elements are 32 apart");
};
template <typename F>
struct Columns {
  int first;
  int count;                                   // of chunks (VEC) or elements below n
  __device__ __forceinline__ Columns(int t, int n) {
    const int lane = t & (F::L - 1), group = t / F::L;
    first = group * F::V * F::kCols + (F::VEC ? lane * kChunk : lane);
    count = F::VEC ? max(0, (n - first + F::kCols - 1) / F::kCols) : max(0, (n - first + 31) / 32);
  }
  __device__ __forceinline__ bool has(int k, int e) const { return F::VEC ? k < count : k * kChunk + e < count; }
  __device__ __forceinline__ bool full() const { return count >= (F::VEC ? F::V : F::V * kChunk); }
};

// Chunk k of a row in shared memory as floats; what lies behind the n columns
// there is zero.
template <int TYPE, typename F>
__device__ __forceinline__ void read_chunk(uint32_t row, int type, const Columns<F>& c, int k, F2& a, F2& b) {
  constexpr int es = kBytes<TYPE>;
  const char* p = smem() + (row + c.first * es) + k * F::kCols * es;
  if (F::VEC) {
    get4<TYPE>(p, type, a, b);
  } else {
    a = f2(get1<TYPE>(p, type), get1<TYPE>(p + 32 * es, type));
    b = f2(get1<TYPE>(p + 64 * es, type), get1<TYPE>(p + 96 * es, type));
  }
}
// A thread's part of a row in memory, as raw words: what several tensors' loads
// need is in flight before the first is converted. Nothing at or past n is read.
template <typename F>
struct RawRow {
  uint32_t w[F::V * kChunk];
  __device__ __forceinline__ void load(const void* row, int type, const Columns<F>& c) {
    const int es = elem_bytes(type);
    const char* p = static_cast<const char*>(row) + c.first * es;
#pragma unroll
    for (int i = 0; i < F::V * kChunk; ++i) w[i] = 0u;
    if (row == nullptr) return;
#pragma unroll
    for (int k = 0; k < F::V; ++k) {
      if (F::VEC) {
        if (!c.has(k, 0)) continue;
        if (type == kF32) {
          const uint4 a = *reinterpret_cast<const uint4*>(p + k * F::kCols * 4);
          w[4 * k] = a.x; w[4 * k + 1] = a.y; w[4 * k + 2] = a.z; w[4 * k + 3] = a.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(p + k * F::kCols * 2);
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
    for (int k = 0; k < F::V; ++k) {
      if (F::VEC && type != kF32) {
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
template <int TYPE, typename F, bool FULL>
__device__ __forceinline__ void write_chunk(char* row, int type, const Columns<F>& c, int k, F2 a, F2 b) {
  constexpr int es = kBytes<TYPE>;
  char* to = row + c.first * es + k * F::kCols * es;
  if (F::VEC) {
    put4<TYPE>(to, type, c.has(k, 0), a, b);
  } else {
    const float2 p = split(a), q = split(b);
    if (FULL || c.has(k, 0)) put1<TYPE>(to, type, p.x);
    if (FULL || c.has(k, 1)) put1<TYPE>(to + 32 * es, type, p.y);
    if (FULL || c.has(k, 2)) put1<TYPE>(to + 64 * es, type, q.x);
    if (FULL || c.has(k, 3)) put1<TYPE>(to + 96 * es, type, q.y);
  }
}
template <int TYPE, typename F>
__device__ __forceinline__ void write_typed(char* row, int type, const Columns<F>& c, const F2* x) {
  if (!F::VEC && c.full()) {
#pragma unroll
    for (int k = 0; k < F::V; ++k) write_chunk<TYPE, F, true>(row, type, c, k, x[2 * k], x[2 * k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < F::V; ++k) write_chunk<TYPE, F, false>(row, type, c, k, x[2 * k], x[2 * k + 1]);
  }
}
// Writes a thread's part of a row.
template <typename F>
__device__ __forceinline__ void write_row(char* row, int type, const Columns<F>& c, const F2* x) {
  if (type == kF32) write_typed<kF32, F>(row, type, c, x);
  else if (type == kBf16) write_typed<kBf16, F>(row, type, c, x);
  else write_typed<kF16, F>(row, type, c, x);
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
template <typename F>
__device__ __forceinline__ void param_chunk(uint32_t p, const Columns<F>& c, int k, F2& a, F2& b) {
  read_chunk<kF32, F>(p, kF32, c, k, a, b);
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

// Starts the copy of a row that begins at src into its place in the ring. Nothing
// before base belongs to the tensor.
template <int ES, typename F>
__device__ __forceinline__ void fetch_row(uint32_t stage, const char* src, const void* base, int n, int t, int T) {
  constexpr int es = ES;
  if (F::VEC) {
    const int at = t / F::L * F::V * F::kCols * es + (t & (F::L - 1)) * 16;
    const int end = min(n * es, (t / F::L + 1) * F::V * F::kCols * es) - at;
#pragma unroll
    for (int i = 0; i < (es == 4 ? F::V : (F::V + 1) / 2); ++i)
      if (i * F::L * 16 < end) copy16(stage + at + i * F::L * 16, src + at + i * F::L * 16);
  } else {
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15u);
    const int end = shift + n * es;            // of the row, from its first granule on
    const char* from = src - shift;
    // the first granule begins before the tensor: the first row, or one of the
    // first rows where several begin in one granule
    const bool cut = from < static_cast<const char*>(base);
    const int whole = end / 16 * 16;
#pragma unroll 1
    for (int g = (t == 0 && cut ? T : t) * 16; g < whole; g += T * 16) copy16(stage + g, from + g);
    if (t == 0 && cut) {
      for (int b = shift; b < 16; b += es) {   // zeros where the row ends in the granule
        if (es == 4)
          *reinterpret_cast<uint32_t*>(smem() + stage + b) = b < end ? *reinterpret_cast<const uint32_t*>(from + b) : 0u;
        else
          *reinterpret_cast<uint16_t*>(smem() + stage + b) =
              b < end ? *reinterpret_cast<const uint16_t*>(from + b) : uint16_t{0};
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

inline bool rows_aligned(const void* p, int64_t ld, int64_t n, int type) {
  const int es = elem_bytes(type);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && n * es % 16 == 0;
}

inline unsigned grid_of(int64_t blocks, int64_t cap) { return static_cast<unsigned>(std::max<int64_t>(1, std::min(blocks, cap))); }

// Bytes of one row of a tensor in the ring: the team's columns; where the row
// may start inside its first granule, one granule more and one of zeros.
inline int64_t slot_columns(const RowShape& r) { return int64_t{std::max(r.T, r.L)} * r.V * kChunk; }
inline int ring_bytes(const RowShape& r, int type, bool vec) {
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
inline bool place_ring(const RowWant& q, RowShape* r) {
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
// several teams a warp. Else whole warps, or half a warp, of V chunks a thread,
// for the V for which kernels exist: the least of
//   rounds x (share of the block's threads at work x (V + 8) + V + 12)
// where a round is a row for every team: a row costs a thread the issue slots of
// its V chunks and of about 8 more (sums across threads, root, addresses), and
// the wait of a chain as long as V and about 12 more. Measured, us:
//   forward   16384 x 320 fp16    V = 1, 3, 8, 16: 22.7, 8.5, 13.3, 19.9; half a warp V = 5: 6.8
//             8192 x 4096 bf16    V = 1, 4, 8, 16: 159, 44, 34, 28.5
//   backward  8192 x 4096         V = 2, 4, 8: 96, 72, 63
//             32768 x 1280 bf16   V = 1, 4, 5, 8: 232, 76, 61, 80
//             333 x 1001          V = 1, 2, 4, 8: 10.3, 9.2, 10.7, 13.8
inline bool row_shape(const RowWant& q, RowShape* best) {
  const int64_t chunks = (q.n + kChunk - 1) / kChunk;
  if (chunks <= 16 && q.vec) {
    best->V = 1;
    best->T = 1;
    while (best->T < chunks) best->T *= 2;
    return place_ring(q, best);
  }
  double least = -1.0;
  for (int lanes : {32, 16}) {
    for (int v : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16}) {
      if (v > q.max_v || (lanes == 16 && (!q.vec || v > 8 || 16 * v < chunks))) continue;
      if (!q.vec && v != 1 && v != 2 && v != 4 && v != 6 && v != 8) continue;
      RowShape r;
      const int64_t t = lanes == 16 ? 16 : (chunks + 32 * v - 1) / (32 * v) * 32;
      if (t > kBlock) continue;
      r.T = static_cast<int>(t);
      r.V = v;
      r.L = lanes;
      if (!place_ring(q, &r)) continue;
      const int64_t rounds = (q.tokens + int64_t{kSms} * r.teams - 1) / (int64_t{kSms} * r.teams);
      const double cost =
          static_cast<double>(rounds) * (static_cast<double>(r.teams * r.T) / kBlock * (v + 8) + v + 12.0);
      if (least < 0.0 || cost <= least) {
        least = cost;
        *best = r;
      }
    }
  }
  return least >= 0.0;
}

// One row a team of up to kMaxRowT threads and V chunks, no ring. Up to 3 rows an
// SM the shortest chain counts: the narrowest slices that hold the row. More rows
// (single elements alone come here): what counts is how many fit on an SM, so the
// fewest registers, T (V + 2). us by V = 1, 2, 4 (with types at run time):
//   300 x 1001 3.3, 3.5, 3.8; 1031 x 1001 6.0, 6.1, 4.6; 1031 x 1501 7.8, 6.4, 6.9
//   300 x 4001 -, 6.2, 5.2; 1031 x 4001 -, 13.4, 10.9
// (V = 8 spills: 1031 x 5003 fp32 17.7 instead of 13.2.)
inline bool single_row_shape(int64_t tokens, int64_t n, RowShape* r) {
  const int64_t chunks = (n + kChunk - 1) / kChunk;
  int64_t least = 0;
  for (int v : {1, 2, 4}) {
    const int64_t t = (chunks + 32 * v - 1) / (32 * v) * 32;
    if (t > (v == 4 ? kMaxRowT : kMaxRowT / 2)) continue;
    const int64_t cost = t * (v + 2);
    if (least > 0 && (tokens <= 3 * kSms || cost >= least)) continue;
    least = cost;
    r->T = static_cast<int>(t);
    r->V = v;
    r->teams = std::max(1, 128 / r->T);
  }
  return least > 0;
}

// Lets a kernel take the ring's share of shared memory; asked for once per
// kernel and device (`done`: a bit per device), since the call costs more than a
// launch.
inline cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemPerSm));
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace

}  // namespace intlora
