// Elements of fp32, bf16 and fp16 tensors: conversions, and accesses of one and
// of eight elements. The type is a run-time value; where it is a constant the
// compiler folds the choice.
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

// 32 bytes from and to a 32-byte boundary in one access (two of 16 bytes would
// touch every 32-byte sector twice).
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Eight consecutive elements from element i on, at a multiple of 8 elements
// (32 bytes of fp32, 16 of a 16-bit type).
__device__ __forceinline__ void load8(const void* p, int64_t i, int type, float* v) {
  if (type == kF32) {
    uint32_t w[8];
    load32(static_cast<const float*>(p) + i, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    unpack8(w, type, v);
  }
}
__device__ __forceinline__ void store8(void* p, int64_t i, int type, const float* v) {
  if (type == kF32) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[e]);
    store32(static_cast<float*>(p) + i, w);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = pack8(v, type);
  }
}

// A kernel that follows another one on the stream and reads what that one wrote
// may be set up while the other still runs: it is launched by launch_after, and
// waits here, before its first access to memory, until the other has ended and
// its writes are visible. (Launched plainly, the second kernel begins about 1 us
// later.) What the other has written is read by plain loads: the read-only path
// (__ldg) is for memory that nothing writes from the kernel's launch on, and such
// loads need not stay behind this wait.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Rows that start at multiples of 8 elements.
inline bool rows_by_8(const void* p, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(8 * elem_bytes(type)) == 0 && ld % 8 == 0;
}

__device__ __forceinline__ const void* row_ptr(const void* p, int64_t row, int64_t ld, int type) {
  return static_cast<const char*>(p) + row * ld * elem_bytes(type);
}
__device__ __forceinline__ void* row_ptr(void* p, int64_t row, int64_t ld, int type) {
  return static_cast<char*>(p) + row * ld * elem_bytes(type);
}

}  // namespace intlora
