// ar_ops.h -- element types and small reductions shared by the operator
// kernels (layer norm, gradient norm and clipping).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ar.h"

namespace ar {

constexpr int kOpsCUs = 256;   // compute units of an MI355X; grids are sized to it

// Launches a kernel of one argument and returns that launch's own result:
// hipGetLastError would also report what an earlier call of the thread, the
// library's or not, has left there.  A failure is not left for the next to find.
template <typename A>
hipError_t launchKernel(void (*kernel)(A), dim3 grid, dim3 block, const A& args, hipStream_t st) {
  void* list[] = {const_cast<A*>(&args)};
  const hipError_t e = hipLaunchKernel((const void*)kernel, grid, block, list, 0, st);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

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

// v plus what lane permutation CTRL brings, in the rows of ROWS.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float addDpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, true));
}

// Sum over rows of 16 lanes; every lane receives its row's.  Lanes swap in
// quads, then with the half row and the row mirrored: the other half's sum is
// the same in each of its lanes by then.  The order is fixed and the same for
// every lane.
__device__ __forceinline__ float rowSum(float v) {
  v = addDpp<0xb1>(v);    // quad_perm 1,0,3,2
  v = addDpp<0x4e>(v);    // quad_perm 2,3,0,1
  v = addDpp<0x141>(v);   // row_half_mirror
  return addDpp<0x140>(v);   // row_mirror
}

// Sum over a wavefront, right in its last lane: row 0's sum is passed to row 1
// and row 2's to row 3, then row 1's to row 3.
__device__ __forceinline__ float waveSumLast(float v) {
  v = rowSum(v);
  v = addDpp<0x142, 0xa>(v);      // row_bcast 15
  return addDpp<0x143, 0xc>(v);   // row_bcast 31
}

// Sum over a wavefront or its halves or quarters of 16 or 32 lanes; every lane
// of the part receives it.
template <int LANES>
__device__ __forceinline__ float laneSum(float v) {
  static_assert(LANES == 16 || LANES == 32 || LANES == 64, "parts of a wavefront");
  if (LANES == 64) {
    const int all = __builtin_bit_cast(int, waveSumLast(v));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(all, 63));
  }
  v = rowSum(v);
  if (LANES == 32)   // with lane ^ 16
    v += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401f));
  return v;
}

__device__ __forceinline__ float waveSum(float v) { return laneSum<64>(v); }

}  // namespace ar
