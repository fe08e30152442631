// ar_gradnorm.hip -- the global norm over a list of tensors, and clipping.
//
//   norm = |s| sqrt(sum g^2)  or  |s| max |g|,   out = g (s min(1, M / (norm + eps))).
//
// The list is cut into spans of about equal cost, one workgroup each.  The
// first kernel leaves one partial per span; what follows combines the
// partials in a fixed order.
#include <math.h>
#include <string.h>

#include <cmath>

#include <new>
#include <vector>

#include "ar_api.h"
#include "ar_internal.h"
#include "ar_ops.h"

namespace ar {
namespace {

constexpr int kNormBlock = 256;
constexpr int kMaxSpans = 8 * kOpsCUs;
constexpr size_t kSpanBytes = 16 * 1024;      // a span's cost at least
constexpr size_t kSegmentCost = 2 * 1024;     // what a segment costs beside its bytes

// A piece of one tensor inside one span.
struct Segment {
  const void* src;
  void* dst;
  int64_t count;
  int dtype;
  int pad;
};
static_assert(sizeof(Segment) == 32, "Segment layout");

constexpr uint64_t kListMagic = 0x41524c4953543031ull;   // "ARLIST01"

struct NormArgs {
  const Segment* segments;
  const int* first;        // span s has segments [first[s], first[s + 1])
  double* partial;         // one per span
  float* norm;             // may be null when clipping
  double scale, maxNorm, eps;
  int nSpans;
};

// A thread's running value.  Squares add up in 64 bits: a product of two
// floats is exact there, and no square overflows or vanishes.  The largest
// absolute value is kept as its bits, which order as the values do with
// infinity above all numbers and NaN above infinity.
template <int KIND> struct Running;
template <> struct Running<arNorm2> {
  typedef double type;
  static __device__ __forceinline__ double add(double acc, float g) { return fma((double)g, (double)g, acc); }
  static __device__ __forceinline__ double join(double a, double b) { return a + b; }
  static __device__ __forceinline__ double value(double a) { return a; }
};
template <> struct Running<arNormMax> {
  typedef uint32_t type;
  static __device__ __forceinline__ uint32_t add(uint32_t acc, float g) {
    return max(acc, __float_as_uint(g) & 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ double value(uint32_t a) { return (double)__uint_as_float(a); }
};

template <int KIND>
__device__ __forceinline__ double join(double a, double b) {
  if (KIND == arNorm2) return a + b;
  return b > a || b != b ? b : a;      // a NaN stays
}

// Combines one value per thread, in a fixed order; every thread receives it.
template <int KIND>
__device__ __forceinline__ double blockJoin(double v, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = join<KIND>(v, __shfl_xor(v, o, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = lds[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) s = join<KIND>(s, lds[w]);
  return s;
}

// Four 16-byte loads a thread in flight; element e of every vector adds to
// sum e % 4, so that four chains of additions run side by side.
template <int KIND, int DT>
__device__ __forceinline__ void addSegment(typename Running<KIND>::type (&acc)[4], const Segment& g) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>, UN = 4;
  const T* p = (const T*)g.src;
  const int64_t nv = g.count / V;
  int64_t i = threadIdx.x;
  for (; i + (UN - 1) * kNormBlock < nv; i += UN * kNormBlock) {
    typename VecOf<T, V>::type x[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) x[u] = loadVec<T, V>(p + (i + u * kNormBlock) * V);
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e % 4] = Running<KIND>::add(acc[e % 4], (float)x[u][e]);
  }
  for (; i < nv; i += kNormBlock) {
    const typename VecOf<T, V>::type x = loadVec<T, V>(p + i * V);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e % 4] = Running<KIND>::add(acc[e % 4], (float)x[e]);
  }
  i = nv * V + threadIdx.x;
  if (i < g.count) acc[0] = Running<KIND>::add(acc[0], (float)p[i]);
}

template <int KIND>
__global__ void __launch_bounds__(kNormBlock) normSpans(const NormArgs a) {
  __shared__ double lds[kNormBlock / 64];
  typedef Running<KIND> R;
  typename R::type acc[4] = {0, 0, 0, 0};
  const int end = a.first[blockIdx.x + 1];
  for (int s = a.first[blockIdx.x]; s < end; ++s) {
    const Segment g = a.segments[s];
    if (g.dtype == arFloat32) addSegment<KIND, arFloat32>(acc, g);
    else if (g.dtype == arFloat16) addSegment<KIND, arFloat16>(acc, g);
    else addSegment<KIND, arBfloat16>(acc, g);
  }
  const double all = blockJoin<KIND>(R::value(R::join(R::join(acc[0], acc[1]), R::join(acc[2], acc[3]))), lds);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = all;
}

// The norm from the partials, the same in every workgroup that asks.
template <int KIND>
__device__ __forceinline__ double normOf(const NormArgs& a, double* lds) {
  double acc = 0.0;
  for (int s = threadIdx.x; s < a.nSpans; s += kNormBlock) acc = join<KIND>(acc, a.partial[s]);
  acc = blockJoin<KIND>(acc, lds);
  return fabs(a.scale) * (KIND == arNorm2 ? sqrt(acc) : acc);
}

template <int KIND>
__global__ void __launch_bounds__(kNormBlock) normFinish(const NormArgs a) {
  __shared__ double lds[kNormBlock / 64];
  const double n = normOf<KIND>(a, lds);
  if (threadIdx.x == 0) a.norm[0] = (float)n;
}

template <int DT>
__device__ __forceinline__ void scaleSegment(const Segment& g, float f) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>, UN = 4;
  typedef typename VecOf<T, V>::type Vec;
  const T* p = (const T*)g.src;
  T* q = (T*)g.dst;
  const int64_t nv = g.count / V;
  int64_t i = threadIdx.x;
  for (; i + (UN - 1) * kNormBlock < nv; i += UN * kNormBlock) {
    Vec x[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) x[u] = loadVec<T, V>(p + (i + u * kNormBlock) * V);
#pragma unroll
    for (int u = 0; u < UN; ++u)
      storeVec<T, V>(q + (i + u * kNormBlock) * V,
                     __builtin_convertvector(__builtin_convertvector(x[u], FloatVec<V>) * f, Vec));
  }
  for (; i < nv; i += kNormBlock)
    storeVec<T, V>(q + i * V,
                   __builtin_convertvector(__builtin_convertvector(loadVec<T, V>(p + i * V), FloatVec<V>) * f, Vec));
  i = nv * V + threadIdx.x;
  if (i < g.count) q[i] = (T)((float)p[i] * f);
}

template <int KIND>
__global__ void __launch_bounds__(kNormBlock) clipSpans(const NormArgs a) {
  __shared__ double lds[kNormBlock / 64];
  const double n = normOf<KIND>(a, lds);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm != nullptr) a.norm[0] = (float)n;
  const double c = n + a.eps <= a.maxNorm ? 1.0 : a.maxNorm / (n + a.eps);
  const float f = (float)(a.scale * c);
  // from the last span back: what the norm read last is what the caches still hold
  const int span = a.nSpans - 1 - (int)blockIdx.x;
  const int end = a.first[span + 1];
  for (int s = a.first[span]; s < end; ++s) {
    const Segment g = a.segments[s];
    if (f == 1.0f && g.src == g.dst) continue;   // nothing would change
    if (g.dtype == arFloat32) scaleSegment<arFloat32>(g, f);
    else if (g.dtype == arFloat16) scaleSegment<arFloat16>(g, f);
    else scaleSegment<arBfloat16>(g, f);
  }
}

}  // namespace
}  // namespace ar

struct arTensorList {
  uint64_t magic;
  int device;
  int nSpans;
  bool outputs;
  char* table;               // device: nSpans + 1 ints, then the segments
  const ar::Segment* segments;
};

namespace ar {
namespace {

bool listOk(const arTensorList* l) { return l != nullptr && (uintptr_t)l % 8 == 0 && l->magic == kListMagic; }

// Cuts the tensors into spans: walks them in order and closes a span once its
// cost (bytes, and kSegmentCost a segment) reaches the target, a tensor larger
// than what is left of the span split there at a 4 KiB grain of its own bytes.
void cutSpans(int nTensors, const void* const* src, void* const* dst, const size_t* counts,
              const arDataType_t* dtypes, std::vector<Segment>& segments, std::vector<int>& first) {
  double cost = 0.0;
  for (int i = 0; i < nTensors; ++i)
    if (counts[i] > 0) cost += (double)counts[i] * elemSize(dtypes[i]) + kSegmentCost;
  size_t target = (size_t)(cost / kMaxSpans) + 1;
  if (target < kSpanBytes) target = kSpanBytes;
  constexpr size_t grain = 4096;
  target = (target + grain - 1) / grain * grain + grain;
  first.push_back(0);
  size_t room = target;
  for (int i = 0; i < nTensors; ++i) {
    const size_t esz = (size_t)elemSize(dtypes[i]);
    size_t done = 0;
    while (done < counts[i]) {
      if (room < kSegmentCost + grain) {
        first.push_back((int)segments.size());
        room = target;
      }
      const size_t can = (room - kSegmentCost) / grain * grain / esz;
      const size_t n = counts[i] - done < can ? counts[i] - done : can;
      Segment g{};
      g.src = (const char*)src[i] + done * esz;
      g.dst = dst != nullptr ? (char*)dst[i] + done * esz : nullptr;
      g.count = (int64_t)n;
      g.dtype = dtypes[i];
      segments.push_back(g);
      const size_t used = n * esz + kSegmentCost;
      room = room > used ? room - used : 0;
      done += n;
    }
  }
  if ((int)segments.size() > first.back()) first.push_back((int)segments.size());
}

arResult_t createList(arTensorList_t* out, int nTensors, const void* const* src, void* const* dst,
                      const size_t* counts, const arDataType_t* dtypes) {
  if (out == nullptr) return arInvalidArgument;
  *out = nullptr;
  if (nTensors < 0 || nTensors > 1 << 20) return arInvalidArgument;
  if (nTensors > 0 && (src == nullptr || counts == nullptr || dtypes == nullptr)) return arInvalidArgument;
  std::vector<Extent> v;
  v.reserve((size_t)nTensors * 2);
  for (int i = 0; i < nTensors; ++i) {
    if (!opsFloatType(dtypes[i]) || counts[i] > (size_t)1 << 40) return arInvalidArgument;
    if (counts[i] == 0) continue;
    const size_t esz = (size_t)elemSize(dtypes[i]), bytes = counts[i] * esz;
    if (src[i] == nullptr || (uintptr_t)src[i] % esz != 0) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)src[i], bytes, 1, bytes, false, i});
    if (dst == nullptr) continue;
    if (dst[i] == nullptr || (uintptr_t)dst[i] % esz != 0) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)dst[i], bytes, 1, bytes, true, i});
  }
  if (dst != nullptr && outputsOverlap(v)) return arInvalidArgument;
  std::vector<Segment> segments;
  std::vector<int> first;
  cutSpans(nTensors, src, dst, counts, dtypes, segments, first);

  int dev = 0, ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess || ndev < 1) return arHipError;
  if (hipGetDevice(&dev) != hipSuccess) return arHipError;
  arTensorList* l = new (std::nothrow) arTensorList();
  if (l == nullptr) return arSystemError;
  l->device = dev;
  l->nSpans = (int)first.size() - 1;
  l->outputs = dst != nullptr;
  const size_t head = (first.size() * sizeof(int) + 31) / 32 * 32;
  std::vector<char> table;
  try {
    table.assign(head + segments.size() * sizeof(Segment), 0);
  } catch (...) {
    delete l;
    throw;
  }
  memcpy(table.data(), first.data(), first.size() * sizeof(int));
  if (!segments.empty()) memcpy(table.data() + head, segments.data(), segments.size() * sizeof(Segment));
  if (hipMalloc((void**)&l->table, table.size()) != hipSuccess) {
    delete l;
    return arHipError;
  }
  if (hipMemcpy(l->table, table.data(), table.size(), hipMemcpyHostToDevice) != hipSuccess) {
    (void)hipFree(l->table);
    delete l;
    return arHipError;
  }
  l->segments = (const Segment*)(l->table + head);
  l->magic = kListMagic;
  *out = l;
  return arSuccess;
}

size_t listWorkspace(const arTensorList* l) {
  return ((size_t)(l->nSpans > 0 ? l->nSpans : 1) * sizeof(double) + 15) / 16 * 16;
}

template <int KIND>
hipError_t launchNorm(const NormArgs& a, bool clip, hipStream_t st) {
  if (a.nSpans > 0) hipLaunchKernelGGL(normSpans<KIND>, dim3(a.nSpans), dim3(kNormBlock), 0, st, a);
  if (!clip)
    hipLaunchKernelGGL(normFinish<KIND>, dim3(1), dim3(kNormBlock), 0, st, a);
  else if (a.nSpans > 0)
    hipLaunchKernelGGL(clipSpans<KIND>, dim3(a.nSpans), dim3(kNormBlock), 0, st, a);
  else if (a.norm != nullptr)
    hipLaunchKernelGGL(normFinish<KIND>, dim3(1), dim3(kNormBlock), 0, st, a);
  return hipGetLastError();
}

arResult_t runNorm(arTensorList* l, bool clip, int kind, float scale, float maxNorm, float eps, float* norm,
                   void* workspace, size_t workspaceBytes, hipStream_t st) {
  if (!listOk(l) || (kind != arNorm2 && kind != arNormMax) || !std::isfinite(scale)) return arInvalidArgument;
  if ((!clip && norm == nullptr) || (uintptr_t)norm % 4 != 0) return arInvalidArgument;
  if (clip && (!(maxNorm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps))) return arInvalidArgument;
  if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceBytes < listWorkspace(l))
    return arInvalidArgument;
  if (groupOpen() || (clip && !l->outputs)) return arInvalidUsage;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return arHipError;
  if (dev != l->device) return arInvalidUsage;
  NormArgs a{};
  a.segments = l->segments;
  a.first = (const int*)l->table;
  a.partial = (double*)workspace;
  a.norm = norm;
  a.scale = scale;
  a.maxNorm = maxNorm;
  a.eps = eps;
  a.nSpans = l->nSpans;
  const hipError_t e = kind == arNorm2 ? launchNorm<arNorm2>(a, clip, st) : launchNorm<arNormMax>(a, clip, st);
  return e == hipSuccess ? arSuccess : arHipError;
}

}  // namespace
}  // namespace ar

extern "C" arResult_t arTensorListCreate(arTensorList_t* list, int nTensors, const void* const* src,
                                         void* const* dst, const size_t* counts, const arDataType_t* dtypes) {
  ApiRange range("arTensorListCreate");
  try {
    return ar::createList(list, nTensors, src, dst, counts, dtypes);
  } catch (const std::bad_alloc&) {
    return arSystemError;
  }
}

extern "C" arResult_t arTensorListWorkspace(arTensorList_t list, size_t* bytes) {
  if (!ar::listOk(list) || bytes == nullptr) return arInvalidArgument;
  *bytes = ar::listWorkspace(list);
  return arSuccess;
}

extern "C" arResult_t arTensorListDestroy(arTensorList_t list) {
  if (list == nullptr) return arSuccess;
  if (!ar::listOk(list)) return arInvalidArgument;
  list->magic = 0;
  const hipError_t e = hipFree(list->table);
  delete list;
  return e == hipSuccess ? arSuccess : arHipError;
}

extern "C" arResult_t arGradNorm(arTensorList_t list, arNormKind_t kind, float scale, float* norm, void* workspace,
                                 size_t workspaceBytes, void* stream) {
  ApiRange range("arGradNorm");
  return ar::noteGroupError(
      ar::runNorm(list, false, kind, scale, 0.0f, 0.0f, norm, workspace, workspaceBytes, (hipStream_t)stream));
}

extern "C" arResult_t arGradClip(arTensorList_t list, arNormKind_t kind, float scale, float maxNorm, float eps,
                                 float* norm, void* workspace, size_t workspaceBytes, void* stream) {
  ApiRange range("arGradClip");
  return ar::noteGroupError(
      ar::runNorm(list, true, kind, scale, maxNorm, eps, norm, workspace, workspaceBytes, (hipStream_t)stream));
}
