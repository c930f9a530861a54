// Elements of fp32, bf16 and fp16 tensors whose type is known at run time.
//
// A thread's slice of a row is V chunks of 8 elements. It is fetched as raw
// words first and converted afterwards, so that the loads of several tensors
// are in flight together; the switch on the type is taken once per slice and
// is uniform over the grid.
//
// Column of element e of chunk k for thread t of T that share a row:
//   VEC:  (k T + t) 8 + e      16-byte loads and stores: rows start at a
//                              16-byte boundary and hold a multiple of 8
//                              elements
//   else: (k 8 + e) T + t      one element per access, neighbouring threads
//                              on neighbouring columns: any alignment, any n
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace intlora {

enum ElemType : int32_t { kF32 = 0, kBf16 = 1, kF16 = 2 };

__host__ __device__ inline int elem_bytes(int type) { return type == kF32 ? 4 : 2; }

__device__ __forceinline__ float elem_from_bits(uint32_t bits, int type) {
  if (type == kF32) return __uint_as_float(bits);
  if (type == kBf16) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// Rounds once, to nearest, ties to even.
__device__ __forceinline__ uint32_t elem_to_bits(float v, int type) {
  if (type == kF32) return __float_as_uint(v);
  if (type == kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int type) {
  if (type == kF32) return static_cast<const float*>(p)[i];
  return elem_from_bits(static_cast<const uint16_t*>(p)[i], type);
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int type, float v) {
  if (type == kF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(elem_to_bits(v, type));
}

// Eight elements packed in 16-bit words <-> floats.
__device__ __forceinline__ void unpack8(const uint32_t* w, int type, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == kBf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float* v, int type) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == kBf16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive elements from element i on (16-byte aligned).
__device__ __forceinline__ void load8(const void* p, int64_t i, int type, float* v) {
  if (type == kF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    unpack8(w, type, v);
  }
}
__device__ __forceinline__ void store8(void* p, int64_t i, int type, const float* v) {
  if (type == kF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = pack8(v, type);
  }
}

template <bool VEC>
__device__ __forceinline__ int slice_col(int k, int e, int t, int T) {
  return VEC ? (k * T + t) * 8 + e : (k * 8 + e) * T + t;
}

// Raw words of one thread's slice of a row. VEC: a chunk of fp32 takes 8
// words, of a 16-bit type 4; else: one word per element.
template <int V>
struct RawSlice {
  uint32_t w[8 * V];
};

// Columns at or past n read as zero.
template <int V, bool VEC>
__device__ __forceinline__ void load_slice(RawSlice<V>& r, const void* row, int type, int n, int t, int T) {
  if (type == kF32) {
    const float* p = static_cast<const float*>(row);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (VEC) {
        const int c = slice_col<VEC>(k, 0, t, T);
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (c < n) {
          a = *reinterpret_cast<const uint4*>(p + c);
          b = *reinterpret_cast<const uint4*>(p + c + 4);
        }
        r.w[8 * k] = a.x; r.w[8 * k + 1] = a.y; r.w[8 * k + 2] = a.z; r.w[8 * k + 3] = a.w;
        r.w[8 * k + 4] = b.x; r.w[8 * k + 5] = b.y; r.w[8 * k + 6] = b.z; r.w[8 * k + 7] = b.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = slice_col<VEC>(k, e, t, T);
          r.w[8 * k + e] = c < n ? __float_as_uint(p[c]) : 0u;
        }
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (VEC) {
        const int c = slice_col<VEC>(k, 0, t, T);
        uint4 a = make_uint4(0, 0, 0, 0);
        if (c < n) a = *reinterpret_cast<const uint4*>(p + c);
        r.w[8 * k] = a.x; r.w[8 * k + 1] = a.y; r.w[8 * k + 2] = a.z; r.w[8 * k + 3] = a.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = slice_col<VEC>(k, e, t, T);
          r.w[8 * k + e] = c < n ? p[c] : 0u;
        }
      }
    }
  }
}

// Chunk k of a raw slice as floats.
template <int V, bool VEC>
__device__ __forceinline__ void slice_chunk(const RawSlice<V>& r, int type, int k, float* v) {
  if (VEC && type != kF32) {
    unpack8(&r.w[8 * k], type, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = elem_from_bits(r.w[8 * k + e], type);
  }
}

// Writes chunk k of a thread's slice (columns at or past n are skipped).
template <bool VEC>
__device__ __forceinline__ void store_chunk(void* row, int type, int n, int t, int T, int k, const float* v) {
  if (VEC) {
    const int c = slice_col<VEC>(k, 0, t, T);
    if (c < n) store8(row, c, type, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = slice_col<VEC>(k, e, t, T);
      if (c < n) store_elem(row, c, type, v[e]);
    }
  }
}

__device__ __forceinline__ const void* row_ptr(const void* p, int64_t row, int64_t ld, int type) {
  return static_cast<const char*>(p) + row * ld * elem_bytes(type);
}
__device__ __forceinline__ void* row_ptr(void* p, int64_t row, int64_t ld, int type) {
  return static_cast<char*>(p) + row * ld * elem_bytes(type);
}

}  // namespace intlora
