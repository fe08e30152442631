// ar_ops.h -- element types and small reductions shared by the operator
// kernels (layer norm, gradient norm and clipping).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ar.h"

namespace ar {

constexpr int kOpsCUs = 256;   // compute units of an MI355X; grids are sized to it

template <int DT> struct Elem;
template <> struct Elem<arFloat32> { typedef float type; };
template <> struct Elem<arFloat16> { typedef _Float16 type; };
template <> struct Elem<arBfloat16> { typedef __bf16 type; };

inline bool opsFloatType(int dtype) { return dtype == arFloat32 || dtype == arFloat16 || dtype == arBfloat16; }

// 16 bytes of elements.  Only element alignment is assumed: global memory
// takes 16-byte accesses at any element address here, so rows of odd width
// and views at odd offsets use the same loads as aligned ones.
template <int DT> constexpr int kVec = 16 / (int)sizeof(typename Elem<DT>::type);

template <typename T, int V>
struct VecOf {
  typedef T type __attribute__((ext_vector_type(V)));
  typedef T packed __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};

template <int V>
using FloatVec = float __attribute__((ext_vector_type(V)));

template <typename T, int V>
__device__ __forceinline__ typename VecOf<T, V>::type loadVec(const T* p) {
  return *(const typename VecOf<T, V>::packed*)p;
}

template <typename T, int V>
__device__ __forceinline__ void storeVec(T* p, typename VecOf<T, V>::type v) {
  *(typename VecOf<T, V>::packed*)p = v;
}

// The same for memory that is not used again soon (non-temporal).
template <typename T, int V>
__device__ __forceinline__ typename VecOf<T, V>::type loadStream(const T* p) {
  return __builtin_nontemporal_load((const typename VecOf<T, V>::packed*)p);
}

template <typename T, int V>
__device__ __forceinline__ void storeStream(T* p, typename VecOf<T, V>::type v) {
  __builtin_nontemporal_store(v, (typename VecOf<T, V>::packed*)p);
}

// Sum over a wavefront; every lane receives it.  A butterfly: each of the 64
// lanes adds the same pairs, so the order is fixed.
__device__ __forceinline__ float waveSum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace ar
