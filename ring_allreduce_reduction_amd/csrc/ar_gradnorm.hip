// ar_gradnorm.hip -- the global norm over a list of tensors, and clipping.
//
//   norm = |s| sqrt(sum g^2)  or  |s| max |g|,   out = g (s min(1, M / (norm + eps))).
//
// The list is cut into tiles; workgroup b takes tiles b, b + grid, ...  The
// first kernel leaves one partial per workgroup; what follows combines the
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

// Bound by memory: 2 flops a value for the norm, 3 to scale it.  The factor
// depends on every value, so a list past the caches is read twice.
constexpr int kNormBlock = 256;
// Tiles of 32 KiB, two workgroups a CU: the workgroups sweep the list as one
// window that moves through memory.  8 x 256 MiB fp32: 315 us (6.8 TB/s; a
// bare read of as much runs at 7.1); 4 workgroups a CU 324, 8 334; one
// contiguous span a workgroup instead of tiles 319-380 by the count, one a
// wavefront 348; cached instead of non-temporal loads 370.
constexpr int kNormGrid = 2 * kOpsCUs;
constexpr size_t kTileMax = 32 * 1024;
// Short lists take shorter tiles, down to one 16-byte vector a thread, so that
// every workgroup still has at least eight or the list is all in flight at once.
constexpr size_t kTileMin = 4096;
constexpr int kTilesEach = 8;
constexpr size_t kMostTiles = (size_t)1 << 25;   // 1 TiB of large tensors, 1 GiB of tiles
// The second pass writes as much as it reads and likes more workgroups: 8 x
// 128 MiB bf16 norm and clip 513 us with 16 a CU, 532 with 8, 550 with 4.
constexpr int kClipGrid = 16 * kOpsCUs;
// What the norm reads last it reads through the caches, and the second pass
// begins there: 474 MB fp16 220-235 us against 262 all non-temporal, 246 all
// cached; 128, 192, 256 and 384 MB kept 239, 234, 235, 240.
constexpr size_t kKeepBytes = (size_t)224 << 20;
// Lists of few tiles run in one workgroup and one launch.  Called back to back
// from the host a launch less saves 3 us (8.6 -> 5.5); replayed from a graph
// the norm of 16, 64, 128 tiles takes 3.1, 4.7, 7.0 us against 4.4 in two
// launches, norm and clip of 8, 16, 32 tiles 4.2, 5.4, 7.6 against 5.3.
constexpr int kSmallBlock = 1024;
constexpr int kSmallNormTiles = 64;
constexpr int kSmallClipTiles = 16;

// A piece of one tensor.
struct Tile {
  const void* src;
  void* dst;
  int count;
  int dtype;
  int64_t pad;
};
static_assert(sizeof(Tile) == 32, "Tile layout");

constexpr uint64_t kListMagic = 0x41524c4953543031ull;   // "ARLIST01"

struct NormArgs {
  const Tile* tiles;
  double* partial;         // one per workgroup of normTiles
  float* norm;             // may be null when clipping
  double scale, maxNorm, eps;
  int nTiles;
  int nPartial;
  int keepFrom;            // tiles from here on are read again soon: through the caches
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

// GROUP threads (a workgroup or a wavefront) add a tile: UN 16-byte loads a
// thread in flight; element e of every vector adds to sum e % 4, so that four
// chains of additions run side by side.
template <int KIND, int DT, bool KEEP, int GROUP>
__device__ __forceinline__ void addTile(typename Running<KIND>::type (&acc)[4], const Tile& g) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>, UN = 4;
  const T* p = (const T*)g.src;
  const int nv = g.count / V;
  int i = threadIdx.x % GROUP;
  for (; i + (UN - 1) * GROUP < nv; i += UN * GROUP) {
    typename VecOf<T, V>::type x[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const T* q = p + (i + u * GROUP) * V;
      x[u] = KEEP ? loadVec<T, V>(q) : loadStream<T, V>(q);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e % 4] = Running<KIND>::add(acc[e % 4], (float)x[u][e]);
  }
  for (; i < nv; i += GROUP) {
    const typename VecOf<T, V>::type x = loadVec<T, V>(p + i * V);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e % 4] = Running<KIND>::add(acc[e % 4], (float)x[e]);
  }
  i = nv * V + threadIdx.x % GROUP;
  if (i < g.count) acc[0] = Running<KIND>::add(acc[0], (float)p[i]);
}

template <int KIND, bool KEEP, int GROUP>
__device__ __forceinline__ void addTyped(typename Running<KIND>::type (&acc)[4], const Tile& g) {
  if (g.dtype == arFloat32) addTile<KIND, arFloat32, KEEP, GROUP>(acc, g);
  else if (g.dtype == arFloat16) addTile<KIND, arFloat16, KEEP, GROUP>(acc, g);
  else addTile<KIND, arBfloat16, KEEP, GROUP>(acc, g);
}

// Combines a thread's four sums over the workgroup.
template <int KIND>
__device__ __forceinline__ double joinAll(const typename Running<KIND>::type (&acc)[4], double* lds) {
  typedef Running<KIND> R;
  return blockJoin<KIND>(R::value(R::join(R::join(acc[0], acc[1]), R::join(acc[2], acc[3]))), lds);
}

template <int KIND>
__global__ void __launch_bounds__(kNormBlock) normTiles(const NormArgs a) {
  __shared__ double lds[kNormBlock / kWave];
  typename Running<KIND>::type acc[4] = {0, 0, 0, 0};
  int t = blockIdx.x;
  Tile g = a.tiles[t];
  while (t < a.nTiles) {
    const int next = t + (int)gridDim.x;
    const Tile ahead = a.tiles[next < a.nTiles ? next : t];
    if (t < a.keepFrom) addTyped<KIND, false, kNormBlock>(acc, g);
    else addTyped<KIND, true, kNormBlock>(acc, g);
    g = ahead;
    t = next;
  }
  const double all = joinAll<KIND>(acc, lds);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = all;
}

// The norm from the partials, the same in every workgroup that asks.
template <int KIND>
__device__ __forceinline__ double normOf(const NormArgs& a, double* lds) {
  double acc = 0.0;
  for (int s = threadIdx.x; s < a.nPartial; s += kNormBlock) acc = join<KIND>(acc, a.partial[s]);
  acc = blockJoin<KIND>(acc, lds);
  return fabs(a.scale) * (KIND == arNorm2 ? sqrt(acc) : acc);
}

template <int KIND>
__global__ void __launch_bounds__(kNormBlock) normFinish(const NormArgs a) {
  __shared__ double lds[kNormBlock / kWave];
  const double n = normOf<KIND>(a, lds);
  if (threadIdx.x == 0) a.norm[0] = (float)n;
}

template <int DT, int GROUP>
__device__ __forceinline__ void scaleTile(const Tile& g, float f) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>, UN = 4;
  typedef typename VecOf<T, V>::type Vec;
  const T* p = (const T*)g.src;
  T* q = (T*)g.dst;
  const int nv = g.count / V;
  int i = threadIdx.x % GROUP;
  for (; i + (UN - 1) * GROUP < nv; i += UN * GROUP) {
    Vec x[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) x[u] = loadStream<T, V>(p + (i + u * GROUP) * V);
#pragma unroll
    for (int u = 0; u < UN; ++u)
      storeStream<T, V>(q + (i + u * GROUP) * V,
                        __builtin_convertvector(__builtin_convertvector(x[u], FloatVec<V>) * f, Vec));
  }
  for (; i < nv; i += GROUP)
    storeStream<T, V>(q + i * V, __builtin_convertvector(
                                     __builtin_convertvector(loadStream<T, V>(p + i * V), FloatVec<V>) * f, Vec));
  i = nv * V + threadIdx.x % GROUP;
  if (i < g.count) q[i] = (T)((float)p[i] * f);
}

template <int GROUP>
__device__ __forceinline__ void scaleTyped(const Tile& g, float f) {
  if (f == 1.0f && g.src == g.dst) return;   // nothing would change
  if (g.dtype == arFloat32) scaleTile<arFloat32, GROUP>(g, f);
  else if (g.dtype == arFloat16) scaleTile<arFloat16, GROUP>(g, f);
  else scaleTile<arBfloat16, GROUP>(g, f);
}

// The factor of every value, from the norm: 64 bits, rounded once.
__device__ __forceinline__ float clipFactor(const NormArgs& a, double norm) {
  const double c = norm + a.eps <= a.maxNorm ? 1.0 : a.maxNorm / (norm + a.eps);
  return (float)(a.scale * c);
}

template <int KIND>
__global__ void __launch_bounds__(kNormBlock) clipTiles(const NormArgs a) {
  __shared__ double lds[kNormBlock / kWave];
  const double n = normOf<KIND>(a, lds);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm != nullptr) a.norm[0] = (float)n;
  const float f = clipFactor(a, n);
  // from the last tile back: what the norm read last is what the caches still hold
  int t = a.nTiles - 1 - (int)blockIdx.x;
  Tile g = a.tiles[t];
  while (t >= 0) {
    const int next = t - (int)gridDim.x;
    const Tile ahead = a.tiles[next >= 0 ? next : t];
    scaleTyped<kNormBlock>(g, f);
    g = ahead;
    t = next;
  }
}

// The whole of a short list in one workgroup: its wavefronts take tiles in turn.
template <int KIND, bool CLIP>
__global__ void __launch_bounds__(kSmallBlock) smallList(const NormArgs a) {
  __shared__ double lds[kSmallBlock / kWave];
  typename Running<KIND>::type acc[4] = {0, 0, 0, 0};
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  for (int t = wave; t < a.nTiles; t += kSmallBlock / kWave) addTyped<KIND, true, kWave>(acc, a.tiles[t]);
  const double all = joinAll<KIND>(acc, lds);
  const double n = fabs(a.scale) * (KIND == arNorm2 ? sqrt(all) : all);
  if (threadIdx.x == 0 && a.norm != nullptr) a.norm[0] = (float)n;
  if (!CLIP) return;
  const float f = clipFactor(a, n);
  for (int t = wave; t < a.nTiles; t += kSmallBlock / kWave) scaleTyped<kWave>(a.tiles[t], f);
}

}  // namespace
}  // namespace ar

struct arTensorList {
  uint64_t magic;
  int device;
  int nTiles;
  int keepFrom;              // the first tile of the last kKeepBytes
  bool outputs;
  ar::Tile* tiles;           // device
};

namespace ar {
namespace {

bool listOk(const arTensorList* l) { return l != nullptr && (uintptr_t)l % 8 == 0 && l->magic == kListMagic; }

// False where the list would need more than kMostTiles.
bool cutTiles(int nTensors, const void* const* src, void* const* dst, const size_t* counts,
              const arDataType_t* dtypes, std::vector<Tile>& tiles) {
  double bytes = 0.0;
  for (int i = 0; i < nTensors; ++i) bytes += (double)counts[i] * elemSize(dtypes[i]);
  size_t tile = kTileMin;
  while (tile < kTileMax && (double)tile * kTilesEach * kNormGrid < bytes) tile *= 2;
  size_t need = 0;
  for (int i = 0; i < nTensors; ++i) need += (counts[i] * (size_t)elemSize(dtypes[i]) + tile - 1) / tile;
  if (need > kMostTiles) return false;
  tiles.reserve(need);
  for (int i = 0; i < nTensors; ++i) {
    const size_t esz = (size_t)elemSize(dtypes[i]);
    for (size_t done = 0; done < counts[i]; done += tile / esz) {
      Tile g{};
      g.src = (const char*)src[i] + done * esz;
      g.dst = dst != nullptr ? (char*)dst[i] + done * esz : nullptr;
      g.count = (int)(counts[i] - done < tile / esz ? counts[i] - done : tile / esz);
      g.dtype = dtypes[i];
      tiles.push_back(g);
    }
  }
  return true;
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
  std::vector<Tile> tiles;
  if (!cutTiles(nTensors, src, dst, counts, dtypes, tiles)) return arInvalidArgument;

  int dev = 0, ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess || ndev < 1) return arHipError;
  if (hipGetDevice(&dev) != hipSuccess) return arHipError;
  arTensorList* l = new (std::nothrow) arTensorList();
  if (l == nullptr) return arSystemError;
  l->device = dev;
  l->nTiles = (int)tiles.size();
  l->outputs = dst != nullptr;
  l->keepFrom = l->nTiles;
  for (size_t kept = 0; l->keepFrom > 0; --l->keepFrom) {
    const Tile& g = tiles[(size_t)l->keepFrom - 1];
    kept += (size_t)g.count * (size_t)elemSize(g.dtype);
    if (kept > kKeepBytes) break;
  }
  if (l->nTiles > 0) {
    const size_t bytes = tiles.size() * sizeof(Tile);
    if (hipMalloc((void**)&l->tiles, bytes) != hipSuccess) {
      (void)hipGetLastError();   // reported here; not left for the thread's next launch to find
      delete l;
      return arHipError;
    }
    if (hipMemcpy(l->tiles, tiles.data(), bytes, hipMemcpyHostToDevice) != hipSuccess) {
      (void)hipFree(l->tiles);
      (void)hipGetLastError();
      delete l;
      return arHipError;
    }
  }
  l->magic = kListMagic;
  *out = l;
  return arSuccess;
}

int gridOf(const arTensorList* l) { return l->nTiles < kNormGrid ? l->nTiles : kNormGrid; }

size_t listWorkspace(const arTensorList* l) {
  return ((size_t)(l->nTiles > 0 ? gridOf(l) : 1) * sizeof(double) + 15) / 16 * 16;
}

template <int KIND>
hipError_t launchNorm(const NormArgs& a, bool clip, hipStream_t st) {
  if (a.nTiles <= (clip ? kSmallClipTiles : kSmallNormTiles)) {   // an empty list too: its norm is 0
    return launchKernel(clip ? smallList<KIND, true> : smallList<KIND, false>, dim3(1), dim3(kSmallBlock), a, st);
  }
  const hipError_t e = launchKernel(normTiles<KIND>, dim3(a.nPartial), dim3(kNormBlock), a, st);
  if (e != hipSuccess) return e;
  if (!clip) return launchKernel(normFinish<KIND>, dim3(1), dim3(kNormBlock), a, st);
  return launchKernel(clipTiles<KIND>, dim3(a.nTiles < kClipGrid ? a.nTiles : kClipGrid), dim3(kNormBlock), a, st);
}

arResult_t runNorm(arTensorList* l, bool clip, int kind, float scale, float maxNorm, float eps, float* norm,
                   void* workspace, size_t workspaceBytes, hipStream_t st) {
  if (!listOk(l) || (kind != arNorm2 && kind != arNormMax) || !std::isfinite(scale)) return arInvalidArgument;
  if ((!clip && norm == nullptr) || (uintptr_t)norm % 4 != 0) return arInvalidArgument;
  if (clip && (!(maxNorm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps))) return arInvalidArgument;
  if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceBytes < listWorkspace(l))
    return arInvalidArgument;
  const uintptr_t n = (uintptr_t)norm, w = (uintptr_t)workspace;
  if (n + sizeof(float) > w && n < w + listWorkspace(l)) return arInvalidArgument;
  if (groupOpen() || (clip && !l->outputs)) return arInvalidUsage;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return arHipError;
  if (dev != l->device) return arInvalidUsage;
  NormArgs a{};
  a.tiles = l->tiles;
  a.partial = (double*)workspace;
  a.norm = norm;
  a.scale = scale;
  a.maxNorm = maxNorm;
  a.eps = eps;
  a.nTiles = l->nTiles;
  a.nPartial = gridOf(l);
  a.keepFrom = clip ? l->keepFrom : l->nTiles;
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
  if (hipFree(list->tiles) != hipSuccess) {   // the list stays whole: the caller may try again
    (void)hipGetLastError();
    return arHipError;
  }
  list->magic = 0;
  delete list;
  return arSuccess;
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
