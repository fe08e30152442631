// ar_dropout.hip -- what follows a row-parallel layer's AllReduce: bias,
// dropout and residual over the rows of N virtual ranks, and their gradients.
//
//   y = residual + k s (x + bias),   dx = k s dy,   dbias = sum over rows of dx,
//
// with k in {0, 1} drawn by counter, so that the backward pass draws it again
// and nothing is stored: Philox4x32 of ten rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) gives 128 bits for
// 8 columns of a row, 16 a column: k = 1 where they are T = round(65536 p) or
// more, and s = 65536 / (65536 - T), so that the mean is x + bias exactly.
#include <cmath>
#include <new>
#include <vector>

#include "ar_rows.h"

namespace ar {
namespace {

constexpr int kDropBlock = 256;
constexpr int kDropCols = 8;    // of a thread: one block of 128 bits

struct DropArgs {
  const void* x[kOpRanks];          // forward: x, backward: dy
  const void* bias[kOpRanks];
  const void* residual[kOpRanks];
  void* y[kOpRanks];                // forward: y, backward: dx or null
  uint32_t firstRow[kOpRanks];
  int rowStart[kOpRanks + 1];       // rank r has rows [rowStart[r], rowStart[r + 1]) of the launch
  int sliceStart[kOpRanks + 1];     // and slices of rows [sliceStart[r], sliceStart[r + 1])
  int64_t xStride, residualStride, yStride;
  int cols, nranks;
  int rowsLog;                      // a workgroup takes 2^rowsLog rows at a time
  int tiles;                        // workgroups across the columns
  uint32_t threshold;               // T in the upper half
  int mode;                         // kKeepAll, kDraw, kKeepNone
  float scale;
  uint32_t key0, key1;
  uint64_t offset;
  const uint64_t* step;
  float* partial;                   // backward: this launch's first row of partial sums, or null
  int partialCols;                  // cols up to a multiple of 8
};

enum { kKeepAll, kDraw, kKeepNone };

typedef uint32_t Words __attribute__((ext_vector_type(4)));

__device__ __forceinline__ Words philox(Words c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t p = (uint64_t)0xD2511F53u * c[0], q = (uint64_t)0xCD9E8D57u * c[2];
    c = Words{(uint32_t)(q >> 32) ^ c[1] ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ c[3] ^ k1, (uint32_t)p};
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// Column e of the 8: a 16-bit half of word e / 2, the lower one first.  The
// threshold's lower half is 0, so the upper one needs no shift.
__device__ __forceinline__ bool kept(const Words& w, int e, uint32_t threshold) {
  return (e % 2 ? w[e / 2] : w[e / 2] << 16) >= threshold;
}

__device__ __forceinline__ Words wordsOf(const DropArgs& a, uint64_t offset, uint32_t row, uint32_t group) {
  if (a.mode == kDraw) return philox(Words{group, row, (uint32_t)offset, (uint32_t)(offset >> 32)}, a.key0, a.key1);
  return (Words)(a.mode == kKeepAll ? ~0u : 0u);   // the threshold is 0, or above 0
}

// The first n (at most 8) elements at p.
template <int DT>
__device__ __forceinline__ FloatVec<8> load8(const typename Elem<DT>::type* p, int n) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>;
  FloatVec<8> f = (FloatVec<8>)0.0f;
  if (n >= 8) {
    typename VecOf<T, V>::type v[8 / V];
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) v[i] = loadVec<T, V>(p + i * V);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)v[e / V][e % V];
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) f[e] = (float)p[e];
  }
  return f;
}

template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, int n, const FloatVec<8>& f) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      typename VecOf<T, V>::type v;
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = (T)f[i * V + e];
      storeVec<T, V>(p + i * V, v);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) p[e] = (T)f[e];
  }
}

// Where a thread works: its 8 columns and its rank's rows, every step-th from
// the first.  Threads past the columns have n <= 0.
struct DropPlace {
  int rank, column, n;
  int row, rows, step;
  uint32_t group;
};

__device__ __forceinline__ DropPlace placeOf(const DropArgs& a) {
  DropPlace p;
  const int across = kDropBlock >> a.rowsLog;
  const int tile = (int)(blockIdx.x % (unsigned)a.tiles), slice = (int)(blockIdx.x / (unsigned)a.tiles);
  p.rank = 0;
  while (slice >= a.sliceStart[p.rank + 1]) ++p.rank;
  p.group = (uint32_t)(tile * across) + (threadIdx.x & (unsigned)(across - 1));
  p.column = (int)p.group * kDropCols;
  p.n = a.cols - p.column;
  p.row = ((slice - a.sliceStart[p.rank]) << a.rowsLog) + (int)(threadIdx.x / (unsigned)across);
  p.rows = a.rowStart[p.rank + 1] - a.rowStart[p.rank];
  p.step = (a.sliceStart[p.rank + 1] - a.sliceStart[p.rank]) << a.rowsLog;
  return p;
}

template <int DT, int WT>
__global__ void __launch_bounds__(kDropBlock) dropoutAdd(const DropArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  const DropPlace at = placeOf(a);
  if (at.n <= 0) return;
  const uint64_t offset = a.offset + (a.step ? *a.step : 0);
  const T* x = (const T*)a.x[at.rank] + at.column;
  const T* residual = a.residual[at.rank] ? (const T*)a.residual[at.rank] + at.column : nullptr;
  T* y = (T*)a.y[at.rank] + at.column;
  FloatVec<8> bias = (FloatVec<8>)0.0f;
  if (a.bias[at.rank]) bias = load8<WT>((const W*)a.bias[at.rank] + at.column, at.n);
  for (int64_t i = at.row; i < at.rows; i += at.step) {
    const FloatVec<8> v = load8<DT>(x + i * a.xStride, at.n);
    const FloatVec<8> z = residual ? load8<DT>(residual + i * a.residualStride, at.n) : (FloatVec<8>)0.0f;
    const Words w = wordsOf(a, offset, a.firstRow[at.rank] + (uint32_t)i, at.group);
    FloatVec<8> out;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = kept(w, e, a.threshold) ? fmaf(v[e] + bias[e], a.scale, z[e]) : z[e];
    store8<DT>(y + i * a.yStride, at.n, out);
  }
}

template <int DT, bool SUMS>
__global__ void __launch_bounds__(kDropBlock) dropoutAddBackward(const DropArgs a) {
  typedef typename Elem<DT>::type T;
  __shared__ float lds[SUMS ? kDropBlock : 1][kDropCols];
  const DropPlace at = placeOf(a);
  FloatVec<8> sum = (FloatVec<8>)0.0f;
  if (at.n > 0) {
    const uint64_t offset = a.offset + (a.step ? *a.step : 0);
    const T* dy = (const T*)a.x[at.rank] + at.column;
    T* dx = a.y[at.rank] ? (T*)a.y[at.rank] + at.column : nullptr;
    for (int64_t i = at.row; i < at.rows; i += at.step) {
      const FloatVec<8> v = load8<DT>(dy + i * a.xStride, at.n);
      const Words w = wordsOf(a, offset, a.firstRow[at.rank] + (uint32_t)i, at.group);
      FloatVec<8> out;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = kept(w, e, a.threshold) ? v[e] : 0.0f;
        if (SUMS) sum[e] += d;
        out[e] = d * a.scale;
      }
      if (dx) store8<DT>(dx + i * a.yStride, at.n, out);
    }
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) lds[threadIdx.x][e] = sum[e];
    __syncthreads();
    const int across = kDropBlock >> a.rowsLog;
    const int tile = (int)(blockIdx.x % (unsigned)a.tiles), slice = (int)(blockIdx.x / (unsigned)a.tiles);
    float* partial = a.partial + (size_t)slice * a.partialCols + (size_t)tile * across * kDropCols;
    for (int c = threadIdx.x; c < across * kDropCols && tile * across * kDropCols + c < a.cols; c += kDropBlock) {
      float s = 0.0f;
      for (int k = 0; k < 1 << a.rowsLog; ++k) s += lds[k * across + c / kDropCols][c % kDropCols];
      partial[c] = s;
    }
  }
}

// Joins the slices' partial sums, 64 columns a workgroup: 64 threads of 16 to
// a row take every 64th slice, then they are joined in order.
struct DropSumArgs {
  void* dbias[AR_MAX_RANKS];
  const float* partial;
  int partialCols, slices, nranks, cols;
  float scale;
};

constexpr int kJoinBlock = 1024, kJoinCols = 64, kJoinSlices = kJoinBlock / (kJoinCols / 4);

template <int WT>
__global__ void __launch_bounds__(kJoinBlock) dropoutBiasGrads(const DropSumArgs a) {
  typedef typename Elem<WT>::type W;
  __shared__ float lds[kJoinSlices][kJoinCols];
  const int lane = threadIdx.x % (kJoinCols / 4), slice = threadIdx.x / (kJoinCols / 4);
  for (int64_t first = (int64_t)blockIdx.x * kJoinCols; first < a.cols; first += (int64_t)gridDim.x * kJoinCols) {
    const int64_t c = first + lane * 4;
    FloatVec<4> sum = (FloatVec<4>)0.0f;
    if (c < a.cols) {
#pragma unroll 4
      for (int k = slice; k < a.slices; k += kJoinSlices)
        sum += *(const FloatVec<4>*)(a.partial + (size_t)k * a.partialCols + c);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) lds[slice][lane * 4 + e] = sum[e];
    __syncthreads();
    const int64_t col = first + threadIdx.x;
    if (threadIdx.x < kJoinCols && col < a.cols) {
      float all = 0.0f;
      for (int k = 0; k < kJoinSlices; ++k) all += lds[k][threadIdx.x];
      for (int r = 0; r < a.nranks; ++r) ((W*)a.dbias[r])[col] = (W)(all * a.scale);
    }
    __syncthreads();   // before the next columns' sums
  }
}

// How a launch is cut: 2^(8 - rowsLog) threads side by side over the columns.
struct DropCut {
  int rowsLog, tiles;
};

DropCut dropCut(int cols) {
  const int groups = (cols + kDropCols - 1) / kDropCols;
  for (int log = 0; log < 8; ++log) {
    const int across = kDropBlock >> log;
    const int tiles = (groups + across - 1) / across;
    if (across <= 16 ? across < 2 * groups : (int64_t)tiles * across <= groups + groups / 8) return {log, tiles};
  }
  return {8, groups};
}

// Slices of the rows of a launch, at most (but one to each rank with rows).
int dropSlices(int64_t rows, const DropCut& k, bool sums) {
  const int64_t each = (int64_t)1 << k.rowsLog;
  int64_t most = (sums ? 8 : 64) * kOpsCUs / k.tiles;
  if (most < 1) most = 1;
  const int64_t full = (rows + each - 1) / each;
  return (int)(full < most ? full : most);
}

template <int DT, int WT>
struct DropForward {
  static hipError_t run(const DropArgs& a, dim3 grid, hipStream_t st) {
    return launchKernel(dropoutAdd<DT, WT>, grid, dim3(kDropBlock), a, st);
  }
};

template <int DT>
struct DropBackward {
  static hipError_t run(const DropArgs& a, dim3 grid, hipStream_t st) {
    return launchKernel(a.partial ? dropoutAddBackward<DT, true> : dropoutAddBackward<DT, false>, grid,
                        dim3(kDropBlock), a, st);
  }
};

template <int WT>
struct DropBiasGrads {
  static hipError_t run(const DropSumArgs& a, hipStream_t st) {
    return launchKernel(dropoutBiasGrads<WT>, dim3(gridOf(((int64_t)a.cols + kJoinCols - 1) / kJoinCols, kJoinBlock)),
                        dim3(kJoinBlock), a, st);
  }
};

// The draw: rows' indices, threshold and scale.  False for a bad argument.
bool drawOk(const size_t* rows, const uint64_t* firstRow, int nranks, double p, const uint64_t* step) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  if (step != nullptr && !aligned(step, 8)) return false;
  uint64_t next = 0;
  for (int r = 0; r < nranks; ++r) {
    const uint64_t first = firstRow ? firstRow[r] : next;
    next = first + rows[r];
    if (rows[r] > 0 && (first > (uint64_t)1 << 32 || next > (uint64_t)1 << 32)) return false;
  }
  return true;
}

void fillDraw(DropArgs* a, double p, uint64_t seed, uint64_t offset, const uint64_t* step) {
  const int t = (int)std::floor(p * 65536.0 + 0.5);
  a->mode = t == 0 ? kKeepAll : t >= 65536 ? kKeepNone : kDraw;
  a->threshold = (uint32_t)(t >= 65536 ? 1 : t) << 16;
  a->scale = t >= 65536 ? 0.0f : (float)(65536.0 / (65536 - t));
  a->key0 = (uint32_t)seed;
  a->key1 = (uint32_t)(seed >> 32);
  a->offset = offset;
  a->step = step;
}

// This launch's rows and their slices; returns the grid's slices.
int fillDropRows(DropArgs* a, const size_t* rows, const uint64_t* firstRow, int nranks, int first, size_t cols,
                 bool sums) {
  a->nranks = nranks - first < kOpRanks ? nranks - first : kOpRanks;
  uint64_t next = 0;
  for (int r = 0; r < first; ++r) next += rows[r];
  a->rowStart[0] = 0;
  for (int r = 0; r < a->nranks; ++r) {
    a->rowStart[r + 1] = a->rowStart[r] + (int)rows[first + r];
    a->firstRow[r] = (uint32_t)(firstRow ? firstRow[first + r] : next);
    next += rows[first + r];
  }
  a->cols = (int)cols;
  a->partialCols = (int)((cols + 7) / 8 * 8);
  const DropCut k = dropCut((int)cols);
  a->rowsLog = k.rowsLog;
  a->tiles = k.tiles;
  const int64_t n = a->rowStart[a->nranks];
  return n == 0 ? 0 : shareOut(a->rowStart, a->nranks, 1 << k.rowsLog, dropSlices(n, k, sums), a->sliceStart);
}

arResult_t dropForward(const void* const* x, const void* const* bias, const void* const* residual, void* const* y,
                       const size_t* rows, const uint64_t* firstRow, int nranks, size_t cols, size_t xStride,
                       size_t residualStride, size_t yStride, double p, uint64_t seed, uint64_t offset,
                       const uint64_t* step, int dtype, int wtype, hipStream_t st) {
  Shape s;
  if (!shapeOk(rows, nranks, cols, &s) || !strideOk(xStride, cols) || !strideOk(yStride, cols) ||
      (residual != nullptr && !strideOk(residualStride, cols)))
    return arInvalidArgument;
  if (!opsFloatType(dtype) || (wtype != dtype && wtype != arFloat32)) return arInvalidArgument;
  if (!drawOk(rows, firstRow, nranks, p, step)) return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  if (s.total == 0) return arSuccess;
  if (x == nullptr || y == nullptr) return arInvalidArgument;
  const int esz = elemSize(dtype), wsz = elemSize(wtype);
  std::vector<Extent> v;
  v.reserve((size_t)nranks * 4 + 1);
  if (step != nullptr && !addFlat(v, step, 1, 8, false)) return arInvalidArgument;
  for (int r = 0; r < nranks; ++r) {
    if (rows[r] == 0) continue;
    bool ok = addRows(v, x[r], rows[r], cols, xStride, esz, false, r) &&
              addRows(v, y[r], rows[r], cols, yStride, esz, true, r);
    if (residual != nullptr) ok = ok && addRows(v, residual[r], rows[r], cols, residualStride, esz, false, r);
    if (bias != nullptr) ok = ok && addFlat(v, bias[r], cols, wsz, false);
    if (!ok) return arInvalidArgument;
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  DropArgs a{};
  fillDraw(&a, p, seed, offset, step);
  for (int l = 0; l < s.launches; ++l) {
    const int first = l * kOpRanks;
    const int slices = fillDropRows(&a, rows, firstRow, nranks, first, cols, false);
    if (slices == 0) continue;
    for (int r = 0; r < a.nranks; ++r) {
      const bool any = rows[first + r] > 0;
      a.x[r] = any ? x[first + r] : nullptr;
      a.y[r] = any ? y[first + r] : nullptr;
      a.bias[r] = any && bias ? bias[first + r] : nullptr;
      a.residual[r] = any && residual ? residual[first + r] : nullptr;
    }
    a.xStride = (int64_t)xStride;
    a.yStride = (int64_t)yStride;
    a.residualStride = (int64_t)residualStride;
    const dim3 grid((unsigned)slices * (unsigned)a.tiles);
    if (byTypes<DropForward, const DropArgs&, dim3, hipStream_t>(dtype, wtype, a, grid, st) != hipSuccess)
      return arHipError;
  }
  return arSuccess;
}

arResult_t dropWorkspace(const size_t* rows, int nranks, size_t cols, size_t* bytes) {
  Shape s;
  if (bytes == nullptr || !shapeOk(rows, nranks, cols, &s)) return arInvalidArgument;
  const DropCut k = dropCut((int)cols);
  size_t slices = 0;
  for (int l = 0; l < s.launches; ++l) {
    const int64_t n = rowsOfLaunch(rows, nranks, l * kOpRanks);
    const int most = n > 0 ? dropSlices(n, k, true) : 0;
    slices += (size_t)(most > 0 && most < kOpRanks ? kOpRanks : most);   // one at least for each rank with rows
  }
  *bytes = (slices > 0 ? slices : 1) * ((cols + 7) / 8 * 8) * sizeof(float);
  return arSuccess;
}

arResult_t dropBackward(const void* const* dy, void* const* dx, void* const* dbias, const size_t* rows,
                        const uint64_t* firstRow, int nranks, size_t cols, size_t dyStride, size_t dxStride, double p,
                        uint64_t seed, uint64_t offset, const uint64_t* step, int dtype, int wtype, void* workspace,
                        size_t workspaceGiven, hipStream_t st) {
  Shape s;
  if (!shapeOk(rows, nranks, cols, &s) || !strideOk(dyStride, cols) || (dx != nullptr && !strideOk(dxStride, cols)))
    return arInvalidArgument;
  if (!opsFloatType(dtype) || (wtype != dtype && wtype != arFloat32)) return arInvalidArgument;
  if (!drawOk(rows, firstRow, nranks, p, step)) return arInvalidArgument;
  if (dx == nullptr && dbias == nullptr) return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  if (s.total > 0 && dy == nullptr) return arInvalidArgument;
  const int esz = elemSize(dtype), wsz = elemSize(wtype);
  std::vector<Extent> v;
  v.reserve((size_t)nranks * 3 + 2);
  if (step != nullptr && !addFlat(v, step, 1, 8, false)) return arInvalidArgument;
  if (dbias != nullptr) {
    size_t need = 0;
    const arResult_t r = dropWorkspace(rows, nranks, cols, &need);
    if (r != arSuccess) return r;
    if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceGiven < need) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)workspace, need, 1, need, true, -1});
  }
  for (int r = 0; r < nranks; ++r) {
    bool ok = true;
    if (rows[r] > 0) {
      ok = addRows(v, dy[r], rows[r], cols, dyStride, esz, false, r);
      if (dx != nullptr) ok = ok && addRows(v, dx[r], rows[r], cols, dxStride, esz, true, r);
    }
    if (dbias != nullptr) ok = ok && addFlat(v, dbias[r], cols, wsz, true);
    if (!ok) return arInvalidArgument;
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  DropArgs a{};
  fillDraw(&a, p, seed, offset, step);
  int partials = 0;
  for (int l = 0; l < s.launches; ++l) {
    const int first = l * kOpRanks;
    const int slices = fillDropRows(&a, rows, firstRow, nranks, first, cols, dbias != nullptr);
    if (slices == 0) continue;
    for (int r = 0; r < a.nranks; ++r) {
      const bool any = rows[first + r] > 0;
      a.x[r] = any ? dy[first + r] : nullptr;
      a.y[r] = any && dx ? dx[first + r] : nullptr;
    }
    a.xStride = (int64_t)dyStride;
    a.yStride = (int64_t)dxStride;
    if (dbias != nullptr) a.partial = (float*)workspace + (size_t)partials * a.partialCols;
    const dim3 grid((unsigned)slices * (unsigned)a.tiles);
    if (byType<DropBackward, const DropArgs&, dim3, hipStream_t>(dtype, a, grid, st) != hipSuccess) return arHipError;
    partials += slices;
  }
  if (dbias == nullptr) return arSuccess;
  DropSumArgs g{};
  for (int r = 0; r < nranks; ++r) g.dbias[r] = dbias[r];
  g.partial = (const float*)workspace;
  g.partialCols = (int)((cols + 7) / 8 * 8);
  g.slices = partials;
  g.nranks = nranks;
  g.cols = (int)cols;
  g.scale = a.scale;
  return byType<DropBiasGrads, const DropSumArgs&, hipStream_t>(wtype, g, st) == hipSuccess ? arSuccess : arHipError;
}

}  // namespace
}  // namespace ar

extern "C" arResult_t arDropoutAdd(const void* const* x, const void* const* bias, const void* const* residual,
                                   void* const* y, const size_t* rows, const uint64_t* firstRow, int nranks,
                                   size_t cols, size_t xStride, size_t residualStride, size_t yStride, double p,
                                   uint64_t seed, uint64_t offset, const uint64_t* step, arDataType_t dtype,
                                   arDataType_t wtype, void* stream) {
  ApiRange range("arDropoutAdd");
  try {
    return ar::noteGroupError(ar::dropForward(x, bias, residual, y, rows, firstRow, nranks, cols, xStride,
                                              residualStride, yStride, p, seed, offset, step, dtype, wtype,
                                              (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}

extern "C" arResult_t arDropoutAddBackwardWorkspace(const size_t* rows, int nranks, size_t cols, size_t* bytes) {
  return ar::dropWorkspace(rows, nranks, cols, bytes);
}

extern "C" arResult_t arDropoutAddBackward(const void* const* dy, void* const* dx, void* const* dbias,
                                           const size_t* rows, const uint64_t* firstRow, int nranks, size_t cols,
                                           size_t dyStride, size_t dxStride, double p, uint64_t seed, uint64_t offset,
                                           const uint64_t* step, arDataType_t dtype, arDataType_t wtype,
                                           void* workspace, size_t workspaceBytes, void* stream) {
  ApiRange range("arDropoutAddBackward");
  try {
    return ar::noteGroupError(ar::dropBackward(dy, dx, dbias, rows, firstRow, nranks, cols, dyStride, dxStride, p,
                                               seed, offset, step, dtype, wtype, workspace, workspaceBytes,
                                               (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}
