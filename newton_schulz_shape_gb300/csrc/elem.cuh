// Element types of the training-step operators (bf16, fp16, fp32) and their
// conversion to and from the fp32 in which every sum, norm and softmax is
// held. A result is rounded to the element type once, to nearest even, when
// it is stored.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/nsgb300.h"

namespace nsk {

// ------------------------------------------------------------ host checks
inline bool dtype_ok(int dtype) { return dtype == NS_DT_BF16 || dtype == NS_DT_FP16 || dtype == NS_DT_FP32; }
inline int elem_bytes(int dtype) { return dtype == NS_DT_FP32 ? 4 : 2; }
// Whether an address can hold elements of `bytes` bytes (null can).
inline bool element_aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements, moved as one aligned word of V * sizeof(T) bytes and
// held packed: a 16-bit pair stays in one register until it is used.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  static_assert(sizeof(T) * V % 4 == 0, "whole registers");
  uint32_t w[sizeof(T) * V / 4];
};
template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
};
template <>
struct Vec<__half, 1> {
  __half v;
};

template <typename T, int V>
__device__ __forceinline__ float get(const Vec<T, V>& x, int i) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(x.w[i]);
  } else if constexpr (V == 1) {
    return to_float(x.v);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return __uint_as_float(i & 1 ? x.w[i / 2] & 0xffff0000u : x.w[i / 2] << 16);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x.w[i / 2]));
    return i & 1 ? f.y : f.x;
  }
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
  Vec<T, V> x;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x.w[i] = __float_as_uint(f[i]);
  } else if constexpr (V == 1) {
    x.v = from_float<T>(f[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[i], f[i + 1]);
        x.w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(f[i], f[i + 1]);
        x.w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  return x;
}

// The largest of x and y value by value, and of all of x: exact in the element
// type, NaN left out.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> max_vec(const Vec<T, V>& x, const Vec<T, V>& y) {
  Vec<T, V> z;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) * V / 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      z.w[i] = __float_as_uint(fmaxf(__uint_as_float(x.w[i]), __uint_as_float(y.w[i])));
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x.w[i]),
                                       *reinterpret_cast<const __nv_bfloat162*>(&y.w[i]));
      z.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __hmax2(*reinterpret_cast<const __half2*>(&x.w[i]), *reinterpret_cast<const __half2*>(&y.w[i]));
      z.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return z;
}
template <typename T, int V>
__device__ __forceinline__ float max_of(const Vec<T, V>& x) {
  float m = get(x, 0);
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, get(x, i));
  return m;
}

// Two fp32 values that one instruction works on.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return d;
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> fill_vec(float v) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = v;
  return pack<T, V>(f);
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> zero_vec() {
  return fill_vec<T, V>(0.0f);
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& x) {
  *reinterpret_cast<Vec<T, V>*>(p) = x;
}
// The same for 16 bytes that are written once (evicted first).
template <typename T>
__device__ __forceinline__ void store_once(T* p, const Vec<T, 16 / sizeof(T)>& x) {
  __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&x));
}

// Elements before the first 16-byte boundary of p, at most n.
template <typename T>
__device__ __forceinline__ long long head_of(const T* p, long long n) {
  const long long h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  return h < n ? h : n;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// An index of 4 or 8 bytes, as callers hold them.
__device__ __forceinline__ long long load_index(const void* p, int bytes, long long i) {
  return bytes == 8 ? static_cast<const long long*>(p)[i] : static_cast<const int*>(p)[i];
}

}  // namespace nsk
