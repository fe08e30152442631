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
//
// Times in comments are of calls in a replayed graph; a call from the host takes
// up to 2.2 us longer where it is short.
#include <cmath>
#include <new>
#include <type_traits>
#include <vector>

#include "ar_rows.h"

namespace ar {
namespace {

constexpr int kLpBlock = 256;
constexpr int kLpVecs = 4;       // of a thread in flight
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// Ranks of a launch at most.  Up to kOpRanks of them travel in arguments of
// that size, which take the host a little less time to hand over (one token of 8 x
// 16000, calls from the host: 7.8 us, 7.9 with twice the size; 20 ranks through the
// binding 7.6, 10.4 in two launches and a join).
constexpr int kLpRanks = 2 * kOpRanks;

struct LpCall {
  int64_t vocabulary;               // the columns of every launch's shards
  const int64_t* targets;
  const float* dlogp;
  float* logp;
  float* top;
  float* logSum;
  float2* partial;                  // (largest value, sum) of a row's parts, `parts` a row, this launch's first; or null
  int parts;
  int rows, nranks;
  float scale, scaleLog2e;
};

template <int RANKS>
struct LpArgs : LpCall {
  const void* x[RANKS];
  int64_t xStride[RANKS];
  int64_t colStart[RANKS + 1];      // shard r holds columns [colStart[r], colStart[r + 1]) of the vocabulary
  int pieceStart[RANKS + 1];        // and pieces [pieceStart[r], pieceStart[r + 1]) of the launch

  // Those of another size, whose ranks fit.
  template <int OTHER>
  static LpArgs of(const LpArgs<OTHER>& a) {
    LpArgs to{};
    (LpCall&)to = a;
    for (int r = 0; r < a.nranks; ++r) {
      to.x[r] = a.x[r];
      to.xStride[r] = a.xStride[r];
    }
    for (int r = 0; r <= a.nranks; ++r) {
      to.colStart[r] = a.colStart[r];
      to.pieceStart[r] = a.pieceStart[r];
    }
    return to;
  }
};

template <int RANKS>
struct LpBackArgs {
  LpArgs<RANKS> call;
  void* dx[RANKS];
  int64_t dxStride[RANKS];

  template <int OTHER>
  static LpBackArgs of(const LpBackArgs<OTHER>& b) {
    LpBackArgs to{};
    to.call = LpArgs<RANKS>::of(b.call);
    for (int r = 0; r < b.call.nranks; ++r) {
      to.dx[r] = b.dx[r];
      to.dxStride[r] = b.dxStride[r];
    }
    return to;
  }
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

// N more logits.  The exponents are scaleLog2e x less the largest's, `ref`, in
// one rounding each; what ref itself was rounded by is taken off the sum to
// first order, which up to 2^12 leaves 2^-26 of it.  Past that (large offsets,
// rows of nothing but the lowest value) differences come first, an operation
// more a logit.
template <int N>
__device__ __forceinline__ void meet(Running* run, const float (&f)[N], float c) {
  float top = run->top;
#pragma unroll
  for (int e = 0; e < N; ++e) top = fmaxf(top, f[e]);
  const float base = baseOf(top), ref = base * c;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (fabsf(ref) <= 0x1p12f) {
#pragma unroll
    for (int e = 0; e < N; ++e) s[e % 4] += __builtin_amdgcn_exp2f(fmaf(f[e], c, -ref));
    s[0] = (s[0] + s[1]) + (s[2] + s[3]);
    s[0] = fmaf(s[0], fmaf(base, c, -ref) * -kLn2, s[0]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) s[e % 4] += expOf(f[e], base, c);
    s[0] = (s[0] + s[1]) + (s[2] + s[3]);
  }
  run->sum = fmaf(run->sum, expOf(run->top, base, c), s[0]);
  run->top = top;
}

// Loads past the caches or through them.
template <typename T, int V, bool STREAM>
__device__ __forceinline__ typename VecOf<T, V>::type loadAs(const T* p) {
  return STREAM ? loadStream<T, V>(p) : loadVec<T, V>(p);
}

// A row's part [from, to) as a workgroup takes it: [first, last) by vectors that
// start at 16 bytes of `p`, the row, and the few elements around them one a
// thread.
struct Part {
  int from, first, last, to;
};

template <typename T, int V>
__device__ __forceinline__ Part partOf(const T* p, int from, int to) {
  const int first = from + (int)((0 - (uintptr_t)(p + from)) % 16 / sizeof(T));
  if (first >= to) return Part{from, to, to, to};
  return Part{from, first, first + (to - first) / V * V, to};
}

// Calls f(column) for a thread's vectors, STEP columns apart, then g(column)
// for its one of the rest.  `thread` counts from 0 among those that share p;
// the vectors begin with thread `skip`, the threads before it come in behind the
// last of them, `behind` columns on.
template <int V, int STEP, typename F, typename G>
__device__ __forceinline__ void forPart(const Part& p, int thread, F f, G g, int skip = 0, int behind = 0) {
  int c = p.first + (thread - skip) * V;
  if (thread < skip) c += behind;
  for (; c < p.last; c += STEP) f(c);
  const int head = p.first - p.from, rest = head + (p.to - p.last);   // at most 2 (V - 1)
  if (thread < rest) g(thread < head ? p.from + thread : p.last + (thread - head));
}

// THREADS threads' part of a shard's row: four vectors a thread in flight, -inf
// past the last one.
template <int DT, int THREADS, bool STREAM>
__device__ __forceinline__ void meetColumns(Running* run, int thread, const typename Elem<DT>::type* x, int from, int to,
                                            float c) {
  typedef typename Elem<DT>::type T;
  constexpr int V = kVec<DT>;
  typedef typename VecOf<T, V>::type Vec;
  const Part part = partOf<T, V>(x, from, to);
  const auto some = [&](auto count, int i) {
    constexpr int N = decltype(count)::value;
    Vec v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = (Vec)(T)-INFINITY;
      if (i + k * THREADS * V < part.last) v[k] = loadAs<T, V, STREAM>(x + i + k * THREADS * V);
    }
    float f[V * N];
#pragma unroll
    for (int e = 0; e < V * N; ++e) f[e] = (float)v[e / V][e % V];
    meet(run, f, c);
  };
  forPart<V, THREADS * V * kLpVecs>(
      part, thread,
      [&](int i) {
        // how many of the four any thread of the wavefront has
        const int left = part.last - i + thread * V;
        if (__ballot(left > 2 * THREADS * V)) some(std::integral_constant<int, kLpVecs>(), i);
        else if (__ballot(left > THREADS * V)) some(std::integral_constant<int, 2>(), i);
        else some(std::integral_constant<int, 1>(), i);
      },
      [&](int i) {
        const float f[1] = {(float)x[i]};
        meet(run, f, c);
      });
}

// Over THREADS threads of a workgroup side by side; the first one receives it.
template <int THREADS>
__device__ __forceinline__ Running joinThreads(Running run, float c, Running* lds) {
  constexpr int LANES = THREADS < kWave ? THREADS : kWave;
  const float top = laneMax<LANES>(run.top);
  run.sum = laneSum<LANES>(run.sum * expOf(run.top, baseOf(top), c));
  run.top = top;
  if (THREADS <= kWave) return run;
  __syncthreads();   // lds may still be read from the row before
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = run;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < THREADS / kWave; ++w) run = join(run, lds[w], c);
  return run;
}

// The target's logit, read early; NaN where the launch's shards have none.
template <int DT, int RANKS>
__device__ __forceinline__ float targetLogit(const LpArgs<RANKS>& a, int64_t row, int64_t t) {
  for (int r = 0; r < a.nranks; ++r)
    if (t >= a.colStart[r] && t < a.colStart[r + 1])
      return (float)((const typename Elem<DT>::type*)a.x[r])[row * a.xStride[r] + (t - a.colStart[r])];
  return NAN;
}

// Of several launches each leaves the running values of its shards, and the one
// with the target its logit, for tokenLogprobJoin.
template <int RANKS>
__device__ __forceinline__ void putPart(const LpArgs<RANKS>& a, int64_t row, int64_t t, const Running& run, float logit) {
  a.partial[row * a.parts] = make_float2(run.top, run.sum);
  if (t >= a.colStart[0] && t < a.colStart[a.nranks]) a.logp[row] = logit;
}

template <typename A>
__device__ __forceinline__ void putRow(const A& a, int64_t row, const Running& run, float logit) {
  const float logSum = logf(run.sum);
  a.logp[row] = (logit - run.top) * a.scale - logSum;
  if (a.top) a.top[row] = run.top;
  if (a.logSum) a.logSum[row] = logSum;
}

template <typename A>
__device__ __forceinline__ void putIgnored(const A& a, int64_t row) {
  a.logp[row] = 0.0f;
  if (a.top) a.top[row] = 0.0f;
  if (a.logSum) a.logSum[row] = 0.0f;
}

// ROW threads take a row, SHARD of them a shard at a time.
template <int DT, int RANKS, int BLOCK, int ROW, int SHARD, bool STREAM>
__global__ void __launch_bounds__(BLOCK) tokenLogprobRows(const LpArgs<RANKS> a) {
  typedef typename Elem<DT>::type T;
  static_assert(ROW == BLOCK || ROW <= kWave, "rows of a wavefront's parts meet no barrier");
  constexpr int ROWS = BLOCK / ROW;
  __shared__ Running lds[BLOCK / kWave];
  const int thread = (int)threadIdx.x % SHARD;
  // a wavefront's shards are its own
  int shard = (int)threadIdx.x % ROW / SHARD;
  if (SHARD >= kWave) shard = __builtin_amdgcn_readfirstlane(shard);
  const bool first = threadIdx.x % ROW == 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / ROW : 0); row < a.rows;
       row += (int64_t)gridDim.x * ROWS) {
    const int64_t t = a.targets[row];
    if (t < 0) {
      if (first && !a.partial) putIgnored(a, row);
      continue;
    }
    float logit = 0.0f;
    if (first) logit = targetLogit<DT>(a, row, t);
    Running run = nothing();
    for (int r = shard; r < a.nranks; r += ROW / SHARD)
      meetColumns<DT, SHARD, STREAM>(&run, thread, (const T*)a.x[r] + row * a.xStride[r], 0,
                                     (int)(a.colStart[r + 1] - a.colStart[r]), a.scaleLog2e);
    run = joinThreads<ROW>(run, a.scaleLog2e, lds);
    if (first && a.partial) putPart(a, row, t, run, logit);
    else if (first) putRow(a, row, run, logit);
  }
}

// A workgroup's piece of its shard: shard r's columns cut into as many equal
// parts (but for 16 columns) as it has pieces.
struct PieceAt {
  int rank, from, to;
};

template <int RANKS>
__device__ __forceinline__ PieceAt pieceAt(const LpArgs<RANKS>& a) {
  PieceAt p;
  p.rank = 0;
  while ((int)blockIdx.x >= a.pieceStart[p.rank + 1]) ++p.rank;
  const unsigned pieces = a.pieceStart[p.rank + 1] - a.pieceStart[p.rank], piece = blockIdx.x - a.pieceStart[p.rank];
  const unsigned cols = (unsigned)(a.colStart[p.rank + 1] - a.colStart[p.rank]);
  const unsigned each = ((cols + pieces - 1) / pieces + 15) / 16 * 16;
  p.from = (int)((uint64_t)each * piece < cols ? each * piece : cols);
  p.to = (int)(p.from + each < cols ? p.from + each : cols);
  return p;
}

// Few rows of a long vocabulary: a workgroup a piece of a row leaves the
// piece's running values; tokenLogprobJoin joins them.
template <int DT, int RANKS>
__global__ void __launch_bounds__(kLpBlock) tokenLogprobPieces(const LpArgs<RANKS> a) {
  typedef typename Elem<DT>::type T;
  __shared__ Running lds[kLpBlock / kWave];
  const PieceAt p = pieceAt(a);
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const int64_t t = a.targets[row];
    if (t < 0) continue;
    const T* x = (const T*)a.x[p.rank] + row * a.xStride[p.rank];
    // the piece that holds the target leaves its logit
    const int64_t at = t - a.colStart[p.rank];
    if (threadIdx.x == 0 && at >= p.from && at < p.to) a.logp[row] = (float)x[at];
    Running run = nothing();
    meetColumns<DT, kLpBlock, false>(&run, (int)threadIdx.x, x, p.from, p.to, a.scaleLog2e);
    run = joinThreads<kLpBlock>(run, a.scaleLog2e, lds);
    if (threadIdx.x == 0) a.partial[row * a.parts + blockIdx.x] = make_float2(run.top, run.sum);
  }
}

// What tokenLogprobJoin needs of a call.
struct LpJoinArgs {
  const int64_t* targets;
  float *logp, *top, *logSum;
  const float2* partial;
  int64_t vocabulary;
  int parts, rows;
  float scale, scaleLog2e;
};

// A wavefront a row.
__global__ void __launch_bounds__(kWave) tokenLogprobJoin(const LpJoinArgs a) {
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t t = a.targets[row];
    if (t < 0) {
      if (threadIdx.x == 0) putIgnored(a, row);
      continue;
    }
    Running run = nothing();
    for (int i = threadIdx.x; i < a.parts; i += kWave) {
      const float2 p = a.partial[row * a.parts + i];
      run = join(run, Running{p.x, p.y}, a.scaleLog2e);
    }
    run = joinThreads<kWave>(run, a.scaleLog2e, nullptr);
    if (threadIdx.x == 0) putRow(a, row, run, t < a.vocabulary ? a.logp[row] : NAN);
  }
}

// A workgroup takes a piece of kLpBlock / THREADS rows at a time.
template <int DT, int RANKS, int THREADS, bool STREAM>
__global__ void __launch_bounds__(kLpBlock) tokenLogprobBackward(const LpBackArgs<RANKS> b) {
  typedef typename Elem<DT>::type T;
  const LpArgs<RANKS>& a = b.call;
  // vectors of a thread in flight, where it has more than a few (8192 rows x 8 x
  // 16008 bf16 689 us, 707 with one, 681 with four; 65536 x 8 x 2056 735, 780, 760)
  constexpr int V = kVec<DT>, ROWS = kLpBlock / THREADS, U = THREADS > 16 ? 2 : 1;
  typedef typename VecOf<T, V>::type Vec;
  const PieceAt p = pieceAt(a);
  const int thread = (int)threadIdx.x % THREADS;
  const auto store = [](T* to, const Vec& v) {
    if (STREAM) storeStream<T, V>(to, v);
    else storeVec<T, V>(to, v);
  };
  for (int64_t row = (int64_t)blockIdx.y * ROWS + (ROWS > 1 ? threadIdx.x / THREADS : 0); row < a.rows;
       row += (int64_t)gridDim.y * ROWS) {
    const int64_t t = a.targets[row], place = t - a.colStart[p.rank];
    const int at = place >= 0 && place < p.to ? (int)place : -1;   // the target's column here
    const float dlogp = a.dlogp[row], base = baseOf(a.top[row]), logSum = a.logSum[row] * kLog2e;
    // their product where 32 bits hold it, else 2^-127 of it; NaN past the vocabulary
    const bool far = fabsf(dlogp * a.scale) == INFINITY;
    const float g = t >= a.vocabulary ? NAN : far ? (dlogp * 0x1p-64f) * (a.scale * 0x1p-63f) : dlogp * a.scale;
    const float back = far ? 0x1p127f : 1.0f;
    const T* x = (const T*)a.x[p.rank] + row * a.xStride[p.rank];
    T* dx = (T*)b.dx[p.rank] + row * b.dxStride[p.rank];
    const Part part = partOf<T, V>(dx, p.from, p.to);
    // wavefronts store whole lines of 128 bytes (8192 rows x 8 x 16008 bf16 710 us,
    // 740 without)
    const int skip = THREADS >= kWave ? (int)((uintptr_t)(dx + part.first) % 128 / 16) : 0;
    const auto element = [&](float v, int c) {
      const float q = __builtin_amdgcn_exp2f(fmaf(v - base, a.scaleLog2e, -logSum));
      return (T)(g * ((c == at ? 1.0f : 0.0f) - q) * back);
    };
    if (t < 0 || dlogp == 0.0f)
      forPart<V, THREADS * V>(
          part, thread, [&](int c) { store(dx + c, (Vec)(T)0.0f); }, [&](int c) { dx[c] = (T)0.0f; }, skip, THREADS * V);
    else
      forPart<V, U * THREADS * V>(
          part, thread,
          [&](int c) {
            Vec v[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
              if (k == 0 || c + k * THREADS * V < part.last) v[k] = loadAs<T, V, STREAM>(x + c + k * THREADS * V);
#pragma unroll
            for (int k = 0; k < U; ++k) {
              const int first = c + k * THREADS * V;
              if (k > 0 && first >= part.last) break;
              Vec out;
#pragma unroll
              for (int e = 0; e < V; ++e) out[e] = element((float)v[k][e], first + e);
              store(dx + first, out);
            }
          },
          [&](int c) { dx[c] = element((float)x[c], c); }, skip, THREADS * V);
  }
}

// How a call is cut, a pure function of its shapes: a launch's shards of a row
// at once, or pieces of them.
struct LpCut {
  bool whole;
  int pieceCols;     // columns of a piece, at most
  int64_t parts;     // of a row: pieces of all shards, or launches; 1 needs no join
};

// Pieces need a second launch, so they are for few rows of a long vocabulary:
// 64 rows x 8 x 16000 bf16 8.4 us in pieces, 10.7 a workgroup a row; 128 rows
// 10.9, 11.8; 200 15.0, 12.4; one row x 8 x 4000 5.6, 4.7; x 8000 5.7, 6.5.  A
// piece is 8192 columns, or down to 2048 where they are few (backward 96 rows x 4
// x 8003 fp32 6.2 us, 6.8 without; more than two a CU gained nothing).
LpCut lpCut(const size_t* cols, int nranks, size_t rows) {
  LpCut k;
  size_t vocabulary = 0;
  for (int r = 0; r < nranks; ++r) vocabulary += cols[r];
  k.whole = rows >= (size_t)kOpsCUs / 2 || vocabulary <= 1 << 15;
  k.pieceCols = 8192;
  const auto count = [&] {
    k.parts = 0;
    for (int r = 0; r < nranks; ++r) k.parts += (int64_t)((cols[r] + k.pieceCols - 1) / k.pieceCols);
  };
  count();
  while (k.pieceCols > 2048 && (int64_t)rows * k.parts < 2 * kOpsCUs) {
    k.pieceCols /= 2;
    count();
  }
  while (k.parts > 4096) {   // the workspace stays small beside a long vocabulary
    k.pieceCols *= 2;
    count();
  }
  if (k.whole) k.parts = (nranks + kLpRanks - 1) / kLpRanks;
  return k;
}

// Calls whose logits are more than the caches hold load (and backward store)
// past them: 8192 rows x 8 x 16000 bf16 305 us, 345 through them; backward 673
// and 725.  Below that the backward pass, which reads the logits again, is better
// off: 512 rows (262 MB moved) 50 and 41.
constexpr size_t kLpStream = (size_t)256 << 20;

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
  *bytes = k.whole && k.parts == 1 ? 0 : (rows * (size_t)k.parts * sizeof(float2) + 15) / 16 * 16;
  return arSuccess;
}

void fillShards(LpArgs<kLpRanks>* a, const void* const* x, const size_t* cols, const size_t* strides, int nranks, int first,
                int pieceCols) {
  a->nranks = nranks - first < kLpRanks ? nranks - first : kLpRanks;
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

// Workgroups of `each` rows at a time.
template <int RANKS>
dim3 pieceGrid(const LpArgs<RANKS>& a, int each) {
  const int64_t groups = ((int64_t)a.rows + each - 1) / each, rows = groups < 65535 ? groups : 65535;
  return dim3((unsigned)a.pieceStart[a.nranks], (unsigned)rows);
}

template <int DT>
struct LpRows {
  template <int RANKS, int BLOCK, int ROW, int SHARD>
  static hipError_t launch(const LpArgs<RANKS>& a, bool stream, hipStream_t st) {
    constexpr int ROWS = BLOCK / ROW;
    return launchKernel(stream ? tokenLogprobRows<DT, RANKS, BLOCK, ROW, SHARD, true>
                               : tokenLogprobRows<DT, RANKS, BLOCK, ROW, SHARD, false>,
                        dim3(gridOf(((int64_t)a.rows + ROWS - 1) / ROWS, BLOCK)), dim3(BLOCK), a, st);
  }
  // Narrow shards: 16 threads take one, alone on a row or four of them (8192
  // rows x 8 x 250 bf16 16 us, 37 with a wavefront a shard, 62 with a workgroup;
  // x 1000 26, 35; 1 x 256 4.7, 8.3 with a wavefront a row; 1 x 2000 8.6, 10.3),
  // where there are many rows: of 300 x 8 x 1000 7.2 us and 5.9 with a wavefront a
  // shard, 1 x 2000 6.3 and 4.6.  Wider ones leave a wavefront threads without a
  // vector (110000 x 8 x 1200 352 us, 587 with a wavefront a shard; 65536 x 8 x
  // 2056 383, 450; 50000 x 8 x 2600 354, 379; 40000 x 8 x 3000 327, 321) and ask for
  // more rows (1200 x 8 x 2000 13.5, 11.6; 8192 46.6, 47.3); one to three gain less
  // (16500 x 1 x 1316 12.4, 14.9; 5000 x 3 x 1500 15.0, 12.9; 40000 x 2 x 2800 79.8,
  // 71.8).  fp32 goes by its vectors of 16 bytes too (4200 x 8 x 481 15.1, 21.1; x 1361
  // 32.1, 33.5; x 1521 39.1, 39.1; 8300 x 1 x 721 6.2, 7.4).
  static bool narrow(const LpArgs<kLpRanks>& a) {
    constexpr int V = kVec<DT>;
    const int64_t columns = (a.colStart[a.nranks] - a.colStart[0]) / a.nranks;
    const bool few = a.nranks < 4;
    return (columns <= 128 * V && a.rows >= 4 * kOpsCUs) ||
           (columns <= (few ? 192 : 352) * V && a.rows >= (few ? 32 : 16) * kOpsCUs);
  }
  static hipError_t run(const LpArgs<kLpRanks>& all, bool stream, hipStream_t st) {
    constexpr int V = kVec<DT>;
    if (all.nranks > kOpRanks) {
      if (narrow(all)) return launch<kLpRanks, kLpBlock, kWave, 16>(all, stream, st);
      return launch<kLpRanks, 512, 512, kWave>(all, stream, st);
    }
    const LpArgs<kOpRanks> a = LpArgs<kOpRanks>::of(all);
    const int64_t vocabulary = a.colStart[a.nranks] - a.colStart[0], columns = vocabulary / a.nranks;   // of a shard
    if (narrow(all)) {
      if (a.nranks < 4) return launch<kOpRanks, kLpBlock, 16, 16>(a, stream, st);
      return launch<kOpRanks, kLpBlock, kWave, 16>(a, stream, st);
    }
    // From four shards on a wavefront takes a shard at a time: shards rarely
    // fill the vectors that a whole workgroup has in flight (8192 rows x 8 x 5000
    // bf16 115 us, 139 with 256 threads together, 191 with 512; 8000 158, 162,
    // 205; 16000 317, 315, 308).  With fewer shards, rows of a few vectors that
    // are many enough go to a wavefront each (20000 x 2000 19 us, 43 with a
    // workgroup; 4096 x 8000 15.3, 15.5; 500 x 4000 5.2, 4.9; 1 x 8000 5.7, 4.2);
    // others to workgroups as wide as their vectors fill (4096 x 50257 70 us with
    // 512, 75 with 256; 50 rows x 3 x 6000 5.8 us with a wavefront a shard, 6.2
    // together; 500 x 2 x 30000 20, 14).
    if (a.nranks > 4) return launch<kOpRanks, 512, 512, kWave>(a, stream, st);
    if (a.nranks == 4) return launch<kOpRanks, kLpBlock, kLpBlock, kWave>(a, stream, st);
    const int many = a.rows < 1024 ? a.rows : 1024;
    if (vocabulary <= (int64_t)V * many) return launch<kOpRanks, kLpBlock, kWave, kWave>(a, stream, st);
    if (a.nranks > 1 && columns <= 1024 * V) return launch<kOpRanks, kLpBlock, kLpBlock, kWave>(a, stream, st);
    if (columns < 3 * 512 * V) return launch<kOpRanks, kLpBlock, kLpBlock, kLpBlock>(a, stream, st);
    return launch<kOpRanks, 512, 512, 512>(a, stream, st);
  }
};

template <int DT>
struct LpPieces {
  template <int RANKS>
  static hipError_t launch(const LpArgs<RANKS>& a, hipStream_t st) {
    return launchKernel(tokenLogprobPieces<DT, RANKS>, pieceGrid(a, 1), dim3(kLpBlock), a, st);
  }
  static hipError_t run(const LpArgs<kLpRanks>& a, hipStream_t st) {
    return a.nranks > kOpRanks ? launch(a, st) : launch(LpArgs<kOpRanks>::of(a), st);
  }
};

template <int DT>
struct LpBackward {
  template <int THREADS, int RANKS>
  static hipError_t launch(const LpBackArgs<RANKS>& b, bool stream, hipStream_t st) {
    return launchKernel(stream ? tokenLogprobBackward<DT, RANKS, THREADS, true>
                               : tokenLogprobBackward<DT, RANKS, THREADS, false>,
                        pieceGrid(b.call, kLpBlock / THREADS), dim3(kLpBlock), b, st);
  }
  static hipError_t run(const LpBackArgs<kLpRanks>& b, bool stream, hipStream_t st) {
    return b.call.nranks > kOpRanks ? byWidth(b, stream, st) : byWidth(LpBackArgs<kOpRanks>::of(b), stream, st);
  }
  template <int RANKS>
  static hipError_t byWidth(const LpBackArgs<RANKS>& b, bool stream, hipStream_t st) {
    constexpr int V = kVec<DT>;
    const LpArgs<RANKS>& a = b.call;
    int64_t widest = 0;   // of the launch's shards
    for (int r = 0; r < a.nranks; ++r) {
      const int64_t c = a.colStart[r + 1] - a.colStart[r];
      widest = c > widest ? c : widest;
    }
    // 2.1 GB of logits in 8 shards, bf16: of 100 columns 1290 us with 16 threads a
    // row, 2026 with 32; 250 1174, 1124, 1707 with 64; 520 1310, 897, 1031; 800 697
    // with 32, 687; 1032 903, 787, 1002 with 128; 1600 663 with 64, 686; 2000 738, 671,
    // 1037 with 256; 3000 652 with 128, 708; 4000 685, 666; 5000 726, 691.  fp32 by its
    // vectors of 16 bytes too (2000 rows x 8 x 93 5.2 with 16, 5.7 with 32; 441 12.1,
    // 12.5 with 64; 953 21.0, 21.1 with 128; 1681 33.8, 33.1 with 256).
    if (widest <= 24 * V) return launch<16>(b, stream, st);
    if (widest <= 112 * V) return launch<32>(b, stream, st);
    if (widest <= 240 * V) return launch<64>(b, stream, st);
    if (widest <= 400 * V) return launch<128>(b, stream, st);
    return launch<kLpBlock>(b, stream, st);
  }
};

// Up to where scale log2(e) is finite.
bool scaleOk(float scale) { return scale > 0.0f && scale <= 0x1p127f; }

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
  const bool joined = !k.whole || k.parts > 1;
  if (joined) {
    size_t need = 0;
    const arResult_t r = lpWorkspace(rows, cols, nranks, &need);
    if (r != arSuccess) return r;
    if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceGiven < need) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)workspace, need, 1, need, true, -1});
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  LpArgs<kLpRanks> a{};
  a.targets = targets;
  a.logp = logp;
  a.top = top;
  a.logSum = logSum;
  a.rows = (int)rows;
  a.scale = scale;
  a.scaleLog2e = (float)((double)scale * 1.44269504088896340736);
  a.vocabulary = vocabulary;
  a.parts = (int)k.parts;
  const bool stream = rows * (size_t)vocabulary * (size_t)elemSize(dtype) > kLpStream;
  int part = 0;
  for (int first = 0; first < nranks; first += kLpRanks) {
    fillShards(&a, logits, cols, strides, nranks, first, k.pieceCols);
    const int pieces = a.pieceStart[a.nranks];
    if (joined) a.partial = (float2*)workspace + part;
    hipError_t e = hipSuccess;
    if (k.whole) e = byType<LpRows, const LpArgs<kLpRanks>&, bool, hipStream_t>(dtype, a, stream, st);
    else if (pieces > 0) e = byType<LpPieces, const LpArgs<kLpRanks>&, hipStream_t>(dtype, a, st);
    if (e != hipSuccess) return arHipError;
    part += k.whole ? 1 : pieces;
  }
  if (!joined) return arSuccess;
  const LpJoinArgs j = {targets, logp, top, logSum, (const float2*)workspace, vocabulary, a.parts, a.rows, scale,
                        a.scaleLog2e};
  return launchKernel(tokenLogprobJoin, dim3(gridOf(a.rows, kWave)), dim3(kWave), j, st) == hipSuccess ? arSuccess
                                                                                                      : arHipError;
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
  LpBackArgs<kLpRanks> b{};
  LpArgs<kLpRanks>& a = b.call;
  a.targets = targets;
  a.dlogp = dlogp;
  a.top = const_cast<float*>(top);
  a.logSum = const_cast<float*>(logSum);
  a.rows = (int)rows;
  a.scale = scale;
  a.scaleLog2e = (float)((double)scale * 1.44269504088896340736);
  a.vocabulary = vocabulary;
  const LpCut k = lpCut(cols, nranks, rows);
  const size_t bytes = 2 * rows * (size_t)vocabulary * (size_t)esz;
  for (int first = 0; first < nranks; first += kLpRanks) {
    fillShards(&a, logits, cols, strides, nranks, first, k.pieceCols);
    for (int r = 0; r < a.nranks; ++r) {
      b.dx[r] = cols[first + r] > 0 ? dlogits[first + r] : nullptr;
      b.dxStride[r] = (int64_t)(dstrides ? dstrides[first + r] : cols[first + r]);
    }
    if (a.pieceStart[a.nranks] == 0) continue;
    if (byType<LpBackward, const LpBackArgs<kLpRanks>&, bool, hipStream_t>(dtype, b, bytes > kLpStream, st) != hipSuccess)
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
