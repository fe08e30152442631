// ar_logprob.hip -- the tokens' log-probabilities from logits whose vocabulary
// is cut over N virtual ranks, and their gradient.
//
// A row's logits x over all shards, its target t and a scale a > 0:
//   M = max x,  S = sum exp(a (x - M)),  logp = a (x_t - M) - ln S,
//   dx_j = a g ([j = t] - exp(a (x_j - M) - ln S)).
// Every exponent is formed from a difference of logits, so that masks of the
// type's lowest value, and rows of nothing else, neither overflow nor cancel;
// M and ln S are kept apart for the same reason.  One pass: a thread keeps the
// largest value it has met and the sum relative to it.
#include <cmath>
#include <new>
#include <vector>

#include "ar_rows.h"

namespace ar {
namespace {

constexpr int kLpBlock = 256;
constexpr int kLpVecs = 4;       // of a thread in flight
constexpr float kLog2e = 1.44269504088896340736f;

struct LpArgs {
  const void* x[kOpRanks];
  void* dx[kOpRanks];               // backward
  int64_t xStride[kOpRanks], dxStride[kOpRanks];
  int64_t colStart[kOpRanks + 1];   // shard r holds columns [colStart[r], colStart[r + 1]) of the vocabulary
  int pieceStart[kOpRanks + 1];     // and pieces [pieceStart[r], pieceStart[r + 1]) of the launch
  int pieceCols;
  int64_t vocabulary;               // the columns of every launch's shards
  const int64_t* targets;
  const float* dlogp;
  float* logp;
  float* top;
  float* logSum;
  float2* partial;                  // the row's pieces' (largest value, sum), `pieces` a row, this launch's first
  int pieces;
  int rows, nranks;
  float scale, scaleLog2e;
};

// A largest value and the sum of exp(scale (x - it)) of what was met.  Of
// nothing, or -inf alone: (-inf, 0).
struct Running {
  float top, sum;
};

__device__ __forceinline__ Running nothing() { return Running{-INFINITY, 0.0f}; }

// What differences are taken to, so that -inf differs from it by -inf.
__device__ __forceinline__ float baseOf(float top) { return top == -INFINITY ? 0.0f : top; }

__device__ __forceinline__ float expOf(float x, float base, float scaleLog2e) {
  return __builtin_amdgcn_exp2f((x - base) * scaleLog2e);
}

__device__ __forceinline__ Running join(const Running& a, const Running& b, float c) {
  Running r;
  r.top = fmaxf(a.top, b.top);
  const float base = baseOf(r.top);
  r.sum = a.sum * expOf(a.top, base, c) + b.sum * expOf(b.top, base, c);
  return r;
}

template <int N>
__device__ __forceinline__ void meet(Running* run, const float (&f)[N], float c) {
  float top = run->top;
#pragma unroll
  for (int e = 0; e < N; ++e) top = fmaxf(top, f[e]);
  const float base = baseOf(top);
  float s[4] = {run->sum * expOf(run->top, base, c), 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < N; ++e) s[e % 4] += expOf(f[e], base, c);
  run->top = top;
  run->sum = (s[0] + s[1]) + (s[2] + s[3]);
}

// A workgroup's share [from, to) of a shard's row.
template <int DT, int BLOCK>
__device__ __forceinline__ void meetColumns(Running* run, const typename Elem<DT>::type* x, int64_t from, int64_t to,
                                            float c) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>;
  const int64_t whole = from + (to - from) / V * V;
  for (int64_t i = from + threadIdx.x * V; i < whole; i += (int64_t)BLOCK * V * kLpVecs) {
    typename VecOf<T, V>::type v[kLpVecs];
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u) {
      v[u] = (typename VecOf<T, V>::type)(T)-INFINITY;
      if (i + u * BLOCK * V < whole) v[u] = loadVec<T, V>(x + i + u * BLOCK * V);
    }
    float f[V * kLpVecs];
#pragma unroll
    for (int e = 0; e < V * kLpVecs; ++e) f[e] = (float)v[e / V][e % V];
    meet(run, f, c);
  }
  if (whole + threadIdx.x < to) {
    const float f[1] = {(float)x[whole + threadIdx.x]};
    meet(run, f, c);
  }
}

// Over a workgroup; thread 0 receives it.
template <int BLOCK>
__device__ __forceinline__ Running joinBlock(Running run, float c, Running* lds) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) {
    const Running other = {__shfl_xor(run.top, m), __shfl_xor(run.sum, m)};
    run = join(run, other, c);
  }
  if (BLOCK == kWave) return run;
  __syncthreads();   // lds may still be read from the row before
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = run;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < BLOCK / kWave; ++w) run = join(run, lds[w], c);
  return run;
}

// The target's logit, read early; NaN for a target past the vocabulary.
template <int DT>
__device__ __forceinline__ float targetLogit(const LpArgs& a, int64_t row, int64_t t) {
  for (int r = 0; r < a.nranks; ++r)
    if (t >= a.colStart[r] && t < a.colStart[r + 1])
      return (float)((const typename Elem<DT>::type*)a.x[r])[row * a.xStride[r] + (t - a.colStart[r])];
  return NAN;
}

__device__ __forceinline__ void putRow(const LpArgs& a, int64_t row, const Running& run, float logit) {
  const float logSum = logf(run.sum);
  a.logp[row] = (logit - run.top) * a.scale - logSum;
  if (a.top) a.top[row] = run.top;
  if (a.logSum) a.logSum[row] = logSum;
}

__device__ __forceinline__ void putIgnored(const LpArgs& a, int64_t row) {
  a.logp[row] = 0.0f;
  if (a.top) a.top[row] = 0.0f;
  if (a.logSum) a.logSum[row] = 0.0f;
}

// A workgroup a row.
template <int DT, int BLOCK>
__global__ void __launch_bounds__(BLOCK) tokenLogprobRows(const LpArgs a) {
  __shared__ Running lds[BLOCK / kWave];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t t = a.targets[row];
    if (t < 0) {
      if (threadIdx.x == 0) putIgnored(a, row);
      continue;
    }
    float logit = 0.0f;
    if (threadIdx.x == 0) logit = targetLogit<DT>(a, row, t);
    Running run = nothing();
    for (int r = 0; r < a.nranks; ++r)
      meetColumns<DT, BLOCK>(&run, (const typename Elem<DT>::type*)a.x[r] + row * a.xStride[r], 0,
                             a.colStart[r + 1] - a.colStart[r], a.scaleLog2e);
    run = joinBlock<BLOCK>(run, a.scaleLog2e, lds);
    if (threadIdx.x == 0) putRow(a, row, run, logit);
  }
}

// Few rows, or more shards than a launch holds: a workgroup a piece of a row
// leaves the piece's running values; tokenLogprobJoin joins them.
template <int DT>
__global__ void __launch_bounds__(kLpBlock) tokenLogprobPieces(const LpArgs a) {
  __shared__ Running lds[kLpBlock / kWave];
  const int piece = blockIdx.x;
  int r = 0;
  while (piece >= a.pieceStart[r + 1]) ++r;
  const int64_t from = (int64_t)(piece - a.pieceStart[r]) * a.pieceCols, cols = a.colStart[r + 1] - a.colStart[r];
  const int64_t to = from + a.pieceCols < cols ? from + a.pieceCols : cols;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const int64_t t = a.targets[row];
    if (t < 0) continue;
    Running run = nothing();
    meetColumns<DT, kLpBlock>(&run, (const typename Elem<DT>::type*)a.x[r] + row * a.xStride[r], from, to,
                              a.scaleLog2e);
    run = joinBlock<kLpBlock>(run, a.scaleLog2e, lds);
    if (threadIdx.x == 0) {
      a.partial[row * a.pieces + piece] = make_float2(run.top, run.sum);
      // the piece that holds the target leaves its logit
      const int64_t at = t - a.colStart[r];
      if (at >= from && at < to)
        a.logp[row] = (float)((const typename Elem<DT>::type*)a.x[r])[row * a.xStride[r] + at];
    }
  }
}

// A wavefront a row.
__global__ void __launch_bounds__(kWave) tokenLogprobJoin(const LpArgs a) {
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t t = a.targets[row];
    if (t < 0) {
      if (threadIdx.x == 0) putIgnored(a, row);
      continue;
    }
    Running run = nothing();
    for (int i = threadIdx.x; i < a.pieces; i += kWave) {
      const float2 p = a.partial[row * a.pieces + i];
      run = join(run, Running{p.x, p.y}, a.scaleLog2e);
    }
    run = joinBlock<kWave>(run, a.scaleLog2e, nullptr);
    if (threadIdx.x == 0) putRow(a, row, run, t < a.vocabulary ? a.logp[row] : NAN);
  }
}

template <int DT>
__global__ void __launch_bounds__(kLpBlock) tokenLogprobBackward(const LpArgs a) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>;
  typedef typename VecOf<T, V>::type Vec;
  const int piece = blockIdx.x;
  int r = 0;
  while (piece >= a.pieceStart[r + 1]) ++r;
  const int64_t from = (int64_t)(piece - a.pieceStart[r]) * a.pieceCols, cols = a.colStart[r + 1] - a.colStart[r];
  const int64_t to = from + a.pieceCols < cols ? from + a.pieceCols : cols;
  const int64_t whole = from + (to - from) / V * V;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const T* x = (const T*)a.x[r] + row * a.xStride[r];
    T* dx = (T*)a.dx[r] + row * a.dxStride[r];
    const int64_t t = a.targets[row];
    float g = t < 0 ? 0.0f : a.dlogp[row] * a.scale;
    if (g == 0.0f) {
      for (int64_t i = from + threadIdx.x * V; i < whole; i += kLpBlock * V) storeVec<T, V>(dx + i, (Vec)(T)0.0f);
      if (whole + threadIdx.x < to) dx[whole + threadIdx.x] = (T)0.0f;
      continue;
    }
    if (t >= a.vocabulary) g = NAN;
    const float base = baseOf(a.top[row]), logSum = a.logSum[row] * kLog2e;
    const int64_t at = t - a.colStart[r];
    for (int64_t i = from + threadIdx.x * V; i < whole; i += kLpBlock * V) {
      const Vec v = loadVec<T, V>(x + i);
      Vec out;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float p = __builtin_amdgcn_exp2f(fmaf((float)v[e] - base, a.scaleLog2e, -logSum));
        out[e] = (T)(g * ((i + e == at ? 1.0f : 0.0f) - p));
      }
      storeVec<T, V>(dx + i, out);
    }
    if (whole + threadIdx.x < to) {
      const int64_t i = whole + threadIdx.x;
      const float p = __builtin_amdgcn_exp2f(fmaf((float)x[i] - base, a.scaleLog2e, -logSum));
      dx[i] = (T)(g * ((i == at ? 1.0f : 0.0f) - p));
    }
  }
}

constexpr int kLpPiece = 8192;         // columns of a piece, at least
constexpr int kLpRowsMost = 16 * kOpsCUs;

// The columns of a piece: a pure function of the shards, so that the workspace
// is known from them.
struct LpCut {
  bool whole;        // a workgroup a row
  int pieceCols;
  int64_t pieces;    // of all shards
};

LpCut lpCut(const size_t* cols, int nranks, size_t rows) {
  LpCut k;
  k.whole = nranks <= kOpRanks && rows >= 4 * (size_t)kOpsCUs;
  k.pieceCols = kLpPiece;
  // a workgroup's grid of pieces stays small against a long vocabulary's
  while (true) {
    k.pieces = 0;
    for (int r = 0; r < nranks; ++r) k.pieces += (int64_t)((cols[r] + k.pieceCols - 1) / k.pieceCols);
    if (k.pieces <= 4096) break;
    k.pieceCols *= 2;
  }
  return k;
}

// Shards: their count, widths and strides.
bool shardsOk(const size_t* cols, const size_t* strides, int nranks, size_t rows, int64_t* vocabulary) {
  if (cols == nullptr || nranks < 1 || nranks > AR_MAX_RANKS || rows > (size_t)kRowsMax) return false;
  *vocabulary = 0;
  for (int r = 0; r < nranks; ++r) {
    if (cols[r] > kRowsMaxCols) return false;
    if (strides != nullptr && !strideOk(strides[r], cols[r] > 0 ? cols[r] : 1)) return false;
    *vocabulary += (int64_t)cols[r];
  }
  return *vocabulary > 0;
}

arResult_t lpWorkspace(size_t rows, const size_t* cols, int nranks, size_t* bytes) {
  int64_t vocabulary;
  if (bytes == nullptr || !shardsOk(cols, nullptr, nranks, rows, &vocabulary)) return arInvalidArgument;
  const LpCut k = lpCut(cols, nranks, rows);
  *bytes = k.whole ? 0 : (rows * (size_t)k.pieces * sizeof(float2) + 15) / 16 * 16;
  return arSuccess;
}

void fillShards(LpArgs* a, const void* const* x, const size_t* cols, const size_t* strides, int nranks, int first,
                int pieceCols) {
  a->nranks = nranks - first < kOpRanks ? nranks - first : kOpRanks;
  a->pieceCols = pieceCols;
  int64_t at = 0;
  for (int r = 0; r < first; ++r) at += (int64_t)cols[r];
  a->colStart[0] = at;
  a->pieceStart[0] = 0;
  for (int r = 0; r < a->nranks; ++r) {
    const size_t c = cols[first + r];
    a->x[r] = c > 0 ? x[first + r] : nullptr;
    a->xStride[r] = (int64_t)(strides ? strides[first + r] : c);
    a->colStart[r + 1] = a->colStart[r] + (int64_t)c;
    a->pieceStart[r + 1] = a->pieceStart[r] + (int)((c + pieceCols - 1) / pieceCols);
  }
}

dim3 pieceGrid(const LpArgs& a) {
  const int rows = a.rows < 65535 ? a.rows : 65535;
  return dim3((unsigned)a.pieceStart[a.nranks], (unsigned)rows);
}

template <int DT>
struct LpRows {
  static hipError_t run(const LpArgs& a, hipStream_t st) {
    const int grid = a.rows < kLpRowsMost ? a.rows : kLpRowsMost;
    return launchKernel(tokenLogprobRows<DT, kLpBlock>, dim3(grid), dim3(kLpBlock), a, st);
  }
};

template <int DT>
struct LpPieces {
  static hipError_t run(const LpArgs& a, hipStream_t st) {
    return launchKernel(tokenLogprobPieces<DT>, pieceGrid(a), dim3(kLpBlock), a, st);
  }
};

template <int DT>
struct LpBackward {
  static hipError_t run(const LpArgs& a, hipStream_t st) {
    return launchKernel(tokenLogprobBackward<DT>, pieceGrid(a), dim3(kLpBlock), a, st);
  }
};

bool scaleOk(float scale) { return scale > 0.0f && std::isfinite(scale); }

arResult_t lpForward(const void* const* logits, const size_t* cols, const size_t* strides, int nranks, size_t rows,
                     const int64_t* targets, float scale, float* logp, float* top, float* logSum, int dtype,
                     void* workspace, size_t workspaceGiven, hipStream_t st) {
  int64_t vocabulary;
  if (!shardsOk(cols, strides, nranks, rows, &vocabulary) || !opsFloatType(dtype) || !scaleOk(scale))
    return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  if (rows == 0) return arSuccess;
  if (logits == nullptr) return arInvalidArgument;
  const LpCut k = lpCut(cols, nranks, rows);
  std::vector<Extent> v;
  v.reserve((size_t)nranks + 5);
  bool ok = addFlat(v, targets, rows, 8, false) && addFlat(v, logp, rows, 4, true);
  if (top != nullptr) ok = ok && addFlat(v, top, rows, 4, true);
  if (logSum != nullptr) ok = ok && addFlat(v, logSum, rows, 4, true);
  for (int r = 0; r < nranks; ++r)
    if (cols[r] > 0)
      ok = ok && addRows(v, logits[r], rows, cols[r], strides ? strides[r] : cols[r], elemSize(dtype), false, -1);
  if (!ok) return arInvalidArgument;
  if (!k.whole) {
    size_t need = 0;
    const arResult_t r = lpWorkspace(rows, cols, nranks, &need);
    if (r != arSuccess) return r;
    if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceGiven < need) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)workspace, need, 1, need, true, -1});
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  LpArgs a{};
  a.targets = targets;
  a.logp = logp;
  a.top = top;
  a.logSum = logSum;
  a.rows = (int)rows;
  a.scale = scale;
  a.scaleLog2e = (float)((double)scale * 1.44269504088896340736);
  a.vocabulary = vocabulary;
  a.pieces = (int)k.pieces;
  if (k.whole) {
    fillShards(&a, logits, cols, strides, nranks, 0, k.pieceCols);
    return byType<LpRows, const LpArgs&, hipStream_t>(dtype, a, st) == hipSuccess ? arSuccess : arHipError;
  }
  int piece = 0;
  for (int first = 0; first < nranks; first += kOpRanks) {
    fillShards(&a, logits, cols, strides, nranks, first, k.pieceCols);
    a.partial = (float2*)workspace + piece;
    piece += a.pieceStart[a.nranks];
    if (a.pieceStart[a.nranks] > 0 && byType<LpPieces, const LpArgs&, hipStream_t>(dtype, a, st) != hipSuccess)
      return arHipError;
  }
  a.partial = (float2*)workspace;
  const int grid = a.rows < kLpRowsMost ? a.rows : kLpRowsMost;
  return launchKernel(tokenLogprobJoin, dim3(grid), dim3(kWave), a, st) == hipSuccess ? arSuccess : arHipError;
}

arResult_t lpBackward(const float* dlogp, const void* const* logits, const size_t* cols, const size_t* strides,
                      int nranks, size_t rows, const int64_t* targets, float scale, const float* top,
                      const float* logSum, void* const* dlogits, const size_t* dstrides, int dtype, hipStream_t st) {
  int64_t vocabulary;
  if (!shardsOk(cols, strides, nranks, rows, &vocabulary) || !shardsOk(cols, dstrides, nranks, rows, &vocabulary) ||
      !opsFloatType(dtype) || !scaleOk(scale))
    return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  if (rows == 0) return arSuccess;
  if (logits == nullptr || dlogits == nullptr) return arInvalidArgument;
  std::vector<Extent> v;
  v.reserve((size_t)nranks * 2 + 4);
  const int esz = elemSize(dtype);
  bool ok = addFlat(v, targets, rows, 8, false) && addFlat(v, dlogp, rows, 4, false) &&
            addFlat(v, top, rows, 4, false) && addFlat(v, logSum, rows, 4, false);
  for (int r = 0; r < nranks; ++r)
    if (cols[r] > 0)
      ok = ok && addRows(v, logits[r], rows, cols[r], strides ? strides[r] : cols[r], esz, false, r) &&
           addRows(v, dlogits[r], rows, cols[r], dstrides ? dstrides[r] : cols[r], esz, true, r);
  if (!ok || outputsOverlap(v)) return arInvalidArgument;
  LpArgs a{};
  a.targets = targets;
  a.dlogp = dlogp;
  a.top = const_cast<float*>(top);
  a.logSum = const_cast<float*>(logSum);
  a.rows = (int)rows;
  a.scale = scale;
  a.scaleLog2e = (float)((double)scale * 1.44269504088896340736);
  a.vocabulary = vocabulary;
  const LpCut k = lpCut(cols, nranks, rows);
  for (int first = 0; first < nranks; first += kOpRanks) {
    fillShards(&a, logits, cols, strides, nranks, first, k.pieceCols);
    for (int r = 0; r < a.nranks; ++r) {
      a.dx[r] = cols[first + r] > 0 ? dlogits[first + r] : nullptr;
      a.dxStride[r] = (int64_t)(dstrides ? dstrides[first + r] : cols[first + r]);
    }
    if (a.pieceStart[a.nranks] > 0 && byType<LpBackward, const LpArgs&, hipStream_t>(dtype, a, st) != hipSuccess)
      return arHipError;
  }
  return arSuccess;
}

}  // namespace
}  // namespace ar

extern "C" arResult_t arTokenLogprobWorkspace(size_t rows, const size_t* cols, int nranks, size_t* bytes) {
  return ar::lpWorkspace(rows, cols, nranks, bytes);
}

extern "C" arResult_t arTokenLogprob(const void* const* logits, const size_t* cols, const size_t* strides, int nranks,
                                     size_t rows, const int64_t* targets, float scale, float* logp, float* top,
                                     float* logSum, arDataType_t dtype, void* workspace, size_t workspaceBytes,
                                     void* stream) {
  ApiRange range("arTokenLogprob");
  try {
    return ar::noteGroupError(ar::lpForward(logits, cols, strides, nranks, rows, targets, scale, logp, top, logSum,
                                            dtype, workspace, workspaceBytes, (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}

extern "C" arResult_t arTokenLogprobBackward(const float* dlogp, const void* const* logits, const size_t* cols,
                                             const size_t* strides, int nranks, size_t rows, const int64_t* targets,
                                             float scale, const float* top, const float* logSum,
                                             void* const* dlogits, const size_t* dlogitsStrides, arDataType_t dtype,
                                             void* stream) {
  ApiRange range("arTokenLogprobBackward");
  try {
    return ar::noteGroupError(ar::lpBackward(dlogp, logits, cols, strides, nranks, rows, targets, scale, top, logSum,
                                             dlogits, dlogitsStrides, dtype, (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}
