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

template <int CTRL>
__device__ __forceinline__ float addDpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over a wavefront or its halves or quarters of 16 or 32 lanes; every lane
// of the part receives it.  Lanes swap inside rows of 16 (quads, then the half
// row and row mirrored: the other half's sum is the same in each of its lanes
// by then), then the rows' sums are swapped or read across.  The order is
// fixed and the same for every lane.
template <int LANES>
__device__ __forceinline__ float laneSum(float v) {
  static_assert(LANES == 16 || LANES == 32 || LANES == 64, "parts of a wavefront");
  v = addDpp<0xb1>(v);    // quad_perm 1,0,3,2
  v = addDpp<0x4e>(v);    // quad_perm 2,3,0,1
  v = addDpp<0x141>(v);   // row_half_mirror
  v = addDpp<0x140>(v);   // row_mirror
  const int b = __builtin_bit_cast(int, v);
  if (LANES == 32) return v + __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(b, 0x401f));   // lane ^ 16
  if (LANES == 64) {
    const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
    const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
    const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
    const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
    return (r0 + r1) + (r2 + r3);
  }
  return v;
}

__device__ __forceinline__ float waveSum(float v) { return laneSum<64>(v); }

}  // namespace ar
