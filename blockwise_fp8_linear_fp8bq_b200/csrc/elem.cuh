// elem.cuh -- element types of the row operators (embedding, norms, gradient
// clipping): BF16, FP16 and FP32 values read into and rounded once from FP32,
// in packs of 1 or several per memory access.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace fp8bq {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}

// Two values, in one instruction where they share a register.
__device__ __forceinline__ float2 to_float2(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ float2 to_float2(const __nv_bfloat16* v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(v));
}
__device__ __forceinline__ float2 to_float2(const __half* v) {
  return __half22float2(*reinterpret_cast<const __half2*>(v));
}
__device__ __forceinline__ void from_float2(float* d, float2 v) {
  d[0] = v.x;
  d[1] = v.y;
}
__device__ __forceinline__ void from_float2(__nv_bfloat16* d, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(d) = __float22bfloat162_rn(v);
}
__device__ __forceinline__ void from_float2(__half* d, float2 v) {
  *reinterpret_cast<__half2*>(d) = __float22half2_rn(v);
}

// VEC consecutive elements, moved in accesses of up to 16 bytes; the address
// is aligned to the smaller of 16 bytes and the pack's size.
template <class T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
  T v[VEC];
  __device__ __forceinline__ float f(int i) const { return to_float(v[i]); }
  __device__ __forceinline__ float2 f2(int i) const { return to_float2(v + 2 * i); }  // values 2 i, 2 i + 1
  __device__ __forceinline__ void set2(int i, float2 w) { from_float2(v + 2 * i, w); }
};

// STREAM: read once, so evicted first from the caches.
template <bool STREAM = false, class T, int VEC>
__device__ __forceinline__ void load_pack(Pack<T, VEC>& p, const T* src) {
  constexpr int kBytes = static_cast<int>(sizeof(T)) * VEC;
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const uint4* s = reinterpret_cast<const uint4*>(src) + i;
      reinterpret_cast<uint4*>(p.v)[i] = STREAM ? __ldcs(s) : *s;
    }
  } else if constexpr (kBytes == 8) {
    const uint2* s = reinterpret_cast<const uint2*>(src);
    *reinterpret_cast<uint2*>(p.v) = STREAM ? __ldcs(s) : *s;
  } else if constexpr (kBytes == 4) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(src);
    *reinterpret_cast<uint32_t*>(p.v) = STREAM ? __ldcs(s) : *s;
  } else {
    static_assert(kBytes == 2, "packs of 2, 4, 8 or a multiple of 16 bytes");
    const uint16_t* s = reinterpret_cast<const uint16_t*>(src);
    *reinterpret_cast<uint16_t*>(p.v) = STREAM ? __ldcs(s) : *s;
  }
}

template <bool STREAM = false, class T, int VEC>
__device__ __forceinline__ void store_pack(T* dst, const Pack<T, VEC>& p) {
  constexpr int kBytes = static_cast<int>(sizeof(T)) * VEC;
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      uint4* d = reinterpret_cast<uint4*>(dst) + i;
      const uint4 w = reinterpret_cast<const uint4*>(p.v)[i];
      if (STREAM)
        __stcs(d, w);
      else
        *d = w;
    }
  } else if constexpr (kBytes == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p.v);
    if (STREAM)
      __stcs(reinterpret_cast<uint2*>(dst), w);
    else
      *reinterpret_cast<uint2*>(dst) = w;
  } else if constexpr (kBytes == 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p.v);
    if (STREAM)
      __stcs(reinterpret_cast<uint32_t*>(dst), w);
    else
      *reinterpret_cast<uint32_t*>(dst) = w;
  } else {
    static_assert(kBytes == 2, "packs of 2, 4, 8 or a multiple of 16 bytes");
    const uint16_t w = *reinterpret_cast<const uint16_t*>(p.v);
    if (STREAM)
      __stcs(reinterpret_cast<uint16_t*>(dst), w);
    else
      *reinterpret_cast<uint16_t*>(dst) = w;
  }
}

// Whether rows of leading dimension ld (elements of `size` bytes) at `p` can
// be accessed in packs of `bytes` bytes.
inline bool rows_aligned(const void* p, int64_t ld, int64_t size, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0 && (ld * size) % bytes == 0;
}

}  // namespace fp8bq
