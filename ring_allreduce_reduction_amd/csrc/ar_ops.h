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

// Sum over a wavefront; every lane receives it.  A butterfly: each of the 64
// lanes adds the same pairs, so the order is fixed.
__device__ __forceinline__ float waveSum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace ar
