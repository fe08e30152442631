// ar_layernorm.hip -- layer norm over the rows of N virtual ranks: forward,
// backward, and the weights' gradient summed over every rank's rows.
//
// Forward, a row of C values:  m = sum x / C,  v = sum (x - m)^2 / C,
// r = 1 / sqrt(v + eps),  y = (x - m) r g + b.  The variance is taken about
// the mean (not as the mean square less the squared mean): a row with a large
// offset loses nothing.
// Backward, h = (x - m) r, q = dy g:  dx = r (q - sum q / C - h sum(q h) / C),
// dg = sum over rows of dy h,  db = sum over rows of dy.
#include <new>
#include <vector>

#include "ar_api.h"
#include "ar_internal.h"
#include "ar_ops.h"

namespace ar {
namespace {

constexpr int kLnRanks = 32;      // ranks per launch: their pointers travel in the kernel arguments
constexpr size_t kLnMaxCols = (size_t)1 << 30;
constexpr int kLnBlock = 256;

struct LnArgs {
  const void* x[kLnRanks];
  const void* dy[kLnRanks];
  const void* gamma[kLnRanks];
  const void* beta[kLnRanks];
  void* y[kLnRanks];              // forward: y, backward: dx
  float* mean[kLnRanks];
  float* rstd[kLnRanks];
  int64_t rowStart[kLnRanks + 1]; // rank r has rows [rowStart[r], rowStart[r + 1]) of the launch
  int blockStart[kLnRanks + 1];   // and workgroups [blockStart[r], blockStart[r + 1]), where they are shared out
  int64_t xStride, yStride, dyStride;
  int cols;
  int nranks;
  float eps;
  float* partial;                 // backward: this launch's first row of partial sums
};

// The weights' gradients of every rank receive the same sums.
struct LnSumArgs {
  void* dgamma[AR_MAX_RANKS];
  void* dbeta[AR_MAX_RANKS];
  const float* partial;           // nPartial rows of [dgamma sums, dbeta sums], 2 * cols floats each
  int nPartial;
  int nranks;
  int cols;
};

__device__ __forceinline__ float blockSum(float v, float* lds) {
  v = waveSum(v);
  __syncthreads();                // lds may still be read from the sum before
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = lds[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) s += lds[w];
  return s;
}

__device__ __forceinline__ int rankOfRow(const LnArgs& a, int64_t row) {
  int r = 0;
  while (row >= a.rowStart[r + 1]) ++r;
  return r;
}

// Calls f(first element, vector of V) for a thread's whole vectors of a row of n
// elements, then g(element) for its share of the few behind them.
template <int V, int BLOCK, typename F, typename G>
__device__ __forceinline__ void forRow(int n, F f, G g) {
  const int whole = n / V * V;
#pragma unroll 4
  for (int c = threadIdx.x * V; c < whole; c += BLOCK * V) f(c);
  const int c = whole + (int)threadIdx.x;
  if (c < n) g(c);
}

// Rows too wide for registers, and rows of less than one vector: a workgroup
// per row, which is read three times (from the caches after the first).  2
// ranks of 1000 rows of 40000 bf16: 87 us with 1024 threads and 8 workgroups a
// CU, 94 with 2, 106 with 512 threads, 117 with 256.
template <int DT, int WT, int BLOCK>
__global__ void __launch_bounds__(BLOCK) layerNormRows(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = kVec<DT>;
  typedef typename VecOf<T, V>::type Vec;
  typedef typename VecOf<W, V>::type WVec;
  __shared__ float lds[BLOCK / kWave];
  const int64_t rows = a.rowStart[a.nranks];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int r = rankOfRow(a, row);
    const int64_t i = row - a.rowStart[r];
    const T* x = (const T*)a.x[r] + i * a.xStride;
    T* y = (T*)a.y[r] + i * a.yStride;
    const W* gamma = (const W*)a.gamma[r];
    const W* beta = (const W*)a.beta[r];
    float s = 0.0f;
    forRow<V, BLOCK>(a.cols,
                     [&](int c) {
                       const Vec v = loadVec<T, V>(x + c);
#pragma unroll
                       for (int e = 0; e < V; ++e) s += (float)v[e];
                     },
                     [&](int c) { s += (float)x[c]; });
    const float mean = blockSum(s, lds) / (float)a.cols;
    float q = 0.0f;
    forRow<V, BLOCK>(a.cols,
                     [&](int c) {
                       const Vec v = loadVec<T, V>(x + c);
#pragma unroll
                       for (int e = 0; e < V; ++e) q = fmaf((float)v[e] - mean, (float)v[e] - mean, q);
                     },
                     [&](int c) { q = fmaf((float)x[c] - mean, (float)x[c] - mean, q); });
    const float rstd = 1.0f / sqrtf(blockSum(q, lds) / (float)a.cols + a.eps);
    forRow<V, BLOCK>(a.cols,
                     [&](int c) {
                       const Vec v = loadVec<T, V>(x + c);
                       const WVec g = gamma ? loadVec<W, V>(gamma + c) : (WVec)(W)1.0f;
                       const WVec b = beta ? loadVec<W, V>(beta + c) : (WVec)(W)0.0f;
                       FloatVec<V> o;
#pragma unroll
                       for (int e = 0; e < V; ++e) o[e] = fmaf(((float)v[e] - mean) * rstd, (float)g[e], (float)b[e]);
                       storeStream<T, V>(y + c, __builtin_convertvector(o, Vec));
                     },
                     [&](int c) {
                       y[c] = (T)fmaf(((float)x[c] - mean) * rstd, gamma ? (float)gamma[c] : 1.0f,
                                      beta ? (float)beta[c] : 0.0f);
                     });
    if (threadIdx.x == 0 && a.mean[r] != nullptr) {
      a.mean[r][i] = mean;
      a.rstd[r][i] = rstd;
    }
  }
}

// A group of THREADS threads (part of a wavefront, one, or a workgroup) owns whole
// rows and keeps them in registers: thread t holds vectors t, t + THREADS, ...
// of a row, NP of them, so memory is read once and written once.  All but the
// last of a thread's vectors lie inside the row.  The last is moved back to
// end with the row where it would pass it, so that every load is one whole
// vector without a branch: `skip` of its elements then belong to another
// thread (all V where the vector lies wholly past the end).  They count in no
// sum; what they store is what their owner stores.
template <int THREADS, int NP, int V>
struct RowPieces {
  int last;    // first element of the last vector
  int skip;    // its elements that are another thread's
  __device__ __forceinline__ RowPieces(int t, int cols) {
    const int at = ((NP - 1) * THREADS + t) * V;
    last = at > cols - V ? cols - V : at;
    skip = at - last < V ? at - last : V;
  }
  __device__ __forceinline__ int offset(int p, int t) const { return p < NP - 1 ? (p * THREADS + t) * V : last; }
  __device__ __forceinline__ bool owns(int p, int e) const { return p < NP - 1 || e >= skip; }
  template <typename T, bool STREAM>
  __device__ __forceinline__ void load(typename VecOf<T, V>::type (&v)[NP], const T* row, int t) const {
#pragma unroll
    for (int p = 0; p < NP; ++p)
      v[p] = STREAM ? loadStream<T, V>(row + offset(p, t)) : loadVec<T, V>(row + offset(p, t));
  }
  template <typename T>
  __device__ __forceinline__ void store(int p, T* row, int t, typename VecOf<T, V>::type v) const {
    if (p < NP - 1 || skip < V) storeStream<T, V>(row + offset(p, t), v);
  }
};

// The workgroups of a launch are shared out among its ranks by their rows, so
// a workgroup meets one rank's weights only and loads them once.  The groups of
// a rank take its rows in turn: together they sweep it as one moving window.
__device__ __forceinline__ int rankOfBlock(const LnArgs& a) {
  int r = 0;
  while ((int)blockIdx.x >= a.blockStart[r + 1]) ++r;
  return r;
}

// Sum over a group's threads.  A workgroup's uses LDS buffers in turn: by the
// time one is written again every wavefront has passed the barrier after it
// was read.
template <int THREADS>
__device__ __forceinline__ float groupSum(float v, float (&lds)[2][16], int& turn) {
  v = laneSum<(THREADS < kWave ? THREADS : kWave)>(v);
  if (THREADS <= kWave) return v;
  if (threadIdx.x % kWave == 0) lds[turn][threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) s += lds[turn][w];
  turn ^= 1;
  return s;
}

// DEPTH rows are in registers at once: while one is reduced the loads of the
// others are in flight.  Bound by memory.  8 ranks of 4096 rows, 16-bit: 8192
// columns 190 us (5.7 TB/s; a bare copy of as much runs at 6.2), 4096 99 us,
// 2048 51 us; 200000 rows of 256 42 us, 2 ranks of 1000 rows of 32768 52 us.
// With the launch's rows taken in turn by all groups instead of each rank's by
// its own, 1024 columns took 67 us instead of 51 (every group met every rank's
// weights); with a run of rows per group instead of turns 8192 took 208.
template <int DT, int WT, int THREADS, int NP, int DEPTH>
__global__ void __launch_bounds__(THREADS < kLnBlock ? kLnBlock : THREADS) layerNormInRegisters(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = kVec<DT>, GROUPS = THREADS < kLnBlock ? kLnBlock / THREADS : 1;
  typedef typename VecOf<T, V>::type Vec;
  typedef typename VecOf<W, V>::type WVec;
  __shared__ float lds[2][16];
  int turn = 0;
  const int t = threadIdx.x % THREADS;
  int sub = GROUPS > 1 ? (int)threadIdx.x / THREADS : 0;
  if (THREADS == kWave) sub = __builtin_amdgcn_readfirstlane(sub);
  const int r = rankOfBlock(a);
  const int64_t rows = a.rowStart[r + 1] - a.rowStart[r];
  const int64_t step = (int64_t)(a.blockStart[r + 1] - a.blockStart[r]) * GROUPS;
  int64_t row = (int64_t)((int)blockIdx.x - a.blockStart[r]) * GROUPS + sub;
  if (row >= rows) return;
  const RowPieces<THREADS, NP, V> pieces(t, a.cols);
  const T* xs = (const T*)a.x[r];
  Vec x[DEPTH][NP];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (row + d * step < rows) pieces.template load<T, true>(x[d], xs + (row + d * step) * a.xStride, t);
  WVec g[NP], b[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    g[p] = (WVec)(W)1.0f;
    b[p] = (WVec)(W)0.0f;
  }
  if (a.gamma[r] != nullptr) pieces.template load<W, false>(g, (const W*)a.gamma[r], t);
  if (a.beta[r] != nullptr) pieces.template load<W, false>(b, (const W*)a.beta[r], t);
  const float inv = 1.0f / (float)a.cols;
  while (true) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      float s = 0.0f;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        float u = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) u += pieces.owns(p, e) ? (float)x[d][p][e] : 0.0f;
        s += u;
      }
      const float mean = groupSum<THREADS>(s, lds, turn) * inv;
      float q = 0.0f;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        float u = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float c = pieces.owns(p, e) ? (float)x[d][p][e] - mean : 0.0f;
          u = fmaf(c, c, u);
        }
        q += u;
      }
      const float rstd = 1.0f / sqrtf(groupSum<THREADS>(q, lds, turn) * inv + a.eps);
      T* y = (T*)a.y[r] + row * a.yStride;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        FloatVec<V> o;
#pragma unroll
        for (int e = 0; e < V; ++e)
          o[e] = fmaf(((float)x[d][p][e] - mean) * rstd, (float)g[p][e], (float)b[p][e]);
        pieces.template store<T>(p, y, t, __builtin_convertvector(o, Vec));
      }
      if (t == 0 && a.mean[r] != nullptr) {
        a.mean[r][row] = mean;
        a.rstd[r][row] = rstd;
      }
      if (row + DEPTH * step < rows) pieces.template load<T, true>(x[d], xs + (row + DEPTH * step) * a.xStride, t);
      row += step;
      if (row >= rows) return;
    }
  }
}

template <int DT, int WT>
__global__ void __launch_bounds__(kLnBlock) layerNormBackwardRows(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  __shared__ float lds[kLnBlock / 64];
  const int64_t rows = a.rowStart[a.nranks];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int r = rankOfRow(a, row);
    const int64_t i = row - a.rowStart[r];
    const T* x = (const T*)a.x[r] + i * a.xStride;
    const T* dy = (const T*)a.dy[r] + i * a.dyStride;
    T* dx = (T*)a.y[r] + i * a.yStride;
    const W* gamma = (const W*)a.gamma[r];
    const float mean = a.mean[r][i], rstd = a.rstd[r][i];
    float s = 0.0f, t = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kLnBlock) {
      const float q = (float)dy[c] * (gamma ? (float)gamma[c] : 1.0f);
      s += q;
      t = fmaf(q, ((float)x[c] - mean) * rstd, t);
    }
    s = blockSum(s, lds) / (float)a.cols;
    t = blockSum(t, lds) / (float)a.cols;
    for (int c = threadIdx.x; c < a.cols; c += kLnBlock) {
      const float q = (float)dy[c] * (gamma ? (float)gamma[c] : 1.0f);
      const float h = ((float)x[c] - mean) * rstd;
      dx[c] = (T)(rstd * (q - s - h * t));
    }
  }
}

// Block (column group, slice of the rows): one thread per column adds its
// slice's rows in order.
template <int DT>
__global__ void __launch_bounds__(kLnBlock) layerNormWeightSums(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  const int c = (int)blockIdx.x * kLnBlock + (int)threadIdx.x;
  if (c >= a.cols) return;
  const int64_t rows = a.rowStart[a.nranks];
  const int64_t lo = rows * blockIdx.y / gridDim.y, hi = rows * (blockIdx.y + 1) / gridDim.y;
  float dg = 0.0f, db = 0.0f;
  int r = 0;
  for (int64_t row = lo; row < hi; ++row) {
    while (row >= a.rowStart[r + 1]) ++r;
    const int64_t i = row - a.rowStart[r];
    const float d = (float)((const T*)a.dy[r])[i * a.dyStride + c];
    const float h = ((float)((const T*)a.x[r])[i * a.xStride + c] - a.mean[r][i]) * a.rstd[r][i];
    dg = fmaf(d, h, dg);
    db += d;
  }
  float* p = a.partial + (size_t)blockIdx.y * 2 * a.cols;
  p[c] = dg;
  p[a.cols + c] = db;
}

template <int WT>
__global__ void __launch_bounds__(kLnBlock) layerNormWeightGrads(const LnSumArgs a) {
  typedef typename Elem<WT>::type W;
  const int c = (int)blockIdx.x * kLnBlock + (int)threadIdx.x;
  if (c >= a.cols) return;
  float dg = 0.0f, db = 0.0f;
  for (int p = 0; p < a.nPartial; ++p) {
    dg += a.partial[(size_t)p * 2 * a.cols + c];
    db += a.partial[(size_t)p * 2 * a.cols + a.cols + c];
  }
  for (int r = 0; r < a.nranks; ++r) {
    if (a.dgamma[r] != nullptr) ((W*)a.dgamma[r])[c] = (W)dg;
    if (a.dbeta[r] != nullptr) ((W*)a.dbeta[r])[c] = (W)db;
  }
}

// Rows of partial sums a launch of `rows` rows writes.
int partialRows(int64_t rows) {
  const int64_t n = (rows + 15) / 16;
  return (int)(n < 1 ? 1 : n > kOpsCUs ? kOpsCUs : n);
}

struct Shape {
  int64_t total = 0;
  int launches = 0;
};

// Row counts, widths and strides every entry checks alike.
bool shapeOk(const size_t* rows, int nranks, size_t cols, Shape* s) {
  if (rows == nullptr || nranks < 1 || nranks > AR_MAX_RANKS || cols < 1 || cols > kLnMaxCols) return false;
  s->total = 0;
  for (int r = 0; r < nranks; ++r) {
    if (rows[r] > (size_t)1 << 40) return false;
    s->total += (int64_t)rows[r];
  }
  s->launches = (nranks + kLnRanks - 1) / kLnRanks;
  return true;
}

bool strideOk(size_t stride, size_t cols) { return stride >= cols && stride <= (size_t)1 << 32; }

bool aligned(const void* p, int esz) { return p != nullptr && (uintptr_t)p % (uintptr_t)esz == 0; }

int64_t rowsOfLaunch(const size_t* rows, int nranks, int first) {
  int64_t n = 0;
  for (int r = first; r < nranks && r < first + kLnRanks; ++r) n += (int64_t)rows[r];
  return n;
}

// Adds a rank's row buffer to the overlap check; false for a bad pointer.
bool addRows(std::vector<Extent>& v, const void* p, size_t rows, size_t cols, size_t stride, int esz, bool output,
             int pair) {
  if (rows == 0) return true;
  if (!aligned(p, esz) || rows > ((size_t)1 << 48) / stride) return false;
  v.push_back(Extent{(uintptr_t)p, cols * (size_t)esz, rows, stride * (size_t)esz, output, pair});
  return true;
}

bool addFlat(std::vector<Extent>& v, const void* p, size_t count, int esz, bool output) {
  return addRows(v, p, count ? 1 : 0, count, count, esz, output, -1);
}

template <template <int, int> class F, typename... A>
hipError_t byTypes(int dtype, int wtype, A... args) {
  if (wtype == arFloat32) {
    if (dtype == arFloat32) return F<arFloat32, arFloat32>::run(args...);
    if (dtype == arFloat16) return F<arFloat16, arFloat32>::run(args...);
    return F<arBfloat16, arFloat32>::run(args...);
  }
  if (dtype == arFloat16) return F<arFloat16, arFloat16>::run(args...);
  return F<arBfloat16, arBfloat16>::run(args...);
}

int rowGrid(int64_t rows) { return (int)(rows < 8 * kOpsCUs ? rows : 8 * kOpsCUs); }

// Shares at most about `most` workgroups of `groups` rows at a time out among
// the ranks by their rows (one at least for a rank with rows); returns the grid.
int shareBlocks(LnArgs* a, int groups, int most) {
  const int64_t rows = a->rowStart[a->nranks];
  int ranks = 0;
  for (int r = 0; r < a->nranks; ++r) ranks += a->rowStart[r + 1] > a->rowStart[r];
  const double share = most > ranks ? (double)(most - ranks) / (double)rows : 0.0;
  a->blockStart[0] = 0;
  for (int r = 0; r < a->nranks; ++r) {
    const int64_t n = a->rowStart[r + 1] - a->rowStart[r];
    const int64_t full = (n + groups - 1) / groups;
    const int64_t mine = n == 0 ? 0 : (int64_t)((double)n * share) + 1;
    a->blockStart[r + 1] = a->blockStart[r] + (int)(mine < full ? mine : full);
  }
  return a->blockStart[a->nranks];
}

template <int DT, int WT, int THREADS, int NP, int DEPTH>
void launchForward(LnArgs a, hipStream_t st) {
  constexpr int BLOCK = THREADS < kLnBlock ? kLnBlock : THREADS;
  static const int resident = [] {
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, layerNormInRegisters<DT, WT, THREADS, NP, DEPTH>, BLOCK, 0) !=
        hipSuccess || n < 1)
      n = 1;
    return n;
  }();
  const int grid = shareBlocks(&a, BLOCK / THREADS, resident * kOpsCUs);
  hipLaunchKernelGGL((layerNormInRegisters<DT, WT, THREADS, NP, DEPTH>), dim3(grid), dim3(BLOCK), 0, st, a);
}

template <int DT, int WT, int BLOCK>
void launchRows(const LnArgs& a, hipStream_t st) {
  const int64_t rows = a.rowStart[a.nranks];
  const int most = (BLOCK < 128 ? 32 : 8) * kOpsCUs;
  hipLaunchKernelGGL((layerNormRows<DT, WT, BLOCK>), dim3((unsigned)(rows < most ? rows : most)), dim3(BLOCK), 0, st, a);
}

template <int DT, int WT>
struct Forward {
  static hipError_t run(const LnArgs& a, hipStream_t st) {
    const int vecs = (a.cols + kVec<DT> - 1) / kVec<DT>;
    // Groups as small as hold the row in four vectors a thread: a wavefront
    // needs no barrier, and parts of one keep narrow rows from leaving lanes
    // idle (128 columns 41 us, 100 with a wavefront a row).  512 x 2 measured
    // 190 at 8192 columns, 256 x 4 193-197, 1024 x 1 237; 256 x 3 50 at 5001,
    // 512 x 2 58; 512 x 4 97 at 16384, 1024 x 2 101.  Two rows in flight, four
    // where a row is one vector a thread; from 1024 x 3 the registers hold one.
    if (a.cols < kVec<DT>) launchRows<DT, WT, 64>(a, st);
    else if (vecs <= 16) launchForward<DT, WT, 16, 1, 4>(a, st);
    else if (vecs <= 32) launchForward<DT, WT, 32, 1, 4>(a, st);
    else if (vecs <= 64) launchForward<DT, WT, 64, 1, 4>(a, st);
    else if (vecs <= 128) launchForward<DT, WT, 64, 2, 2>(a, st);
    else if (vecs <= 192) launchForward<DT, WT, 64, 3, 2>(a, st);
    else if (vecs <= 256) launchForward<DT, WT, 64, 4, 2>(a, st);
    else if (vecs <= 512) launchForward<DT, WT, 256, 2, 2>(a, st);
    else if (vecs <= 768) launchForward<DT, WT, 256, 3, 2>(a, st);
    else if (vecs <= 1024) launchForward<DT, WT, 512, 2, 2>(a, st);
    else if (vecs <= 1536) launchForward<DT, WT, 512, 3, 2>(a, st);
    else if (vecs <= 2048) launchForward<DT, WT, 512, 4, 2>(a, st);
    else if (vecs <= 3072) launchForward<DT, WT, 1024, 3, 1>(a, st);
    else if (vecs <= 4096) launchForward<DT, WT, 1024, 4, 1>(a, st);
    else launchRows<DT, WT, 1024>(a, st);
    return hipGetLastError();
  }
};

template <int DT, int WT>
struct Backward {
  static hipError_t run(const LnArgs& a, bool dx, hipStream_t st) {
    const int64_t rows = a.rowStart[a.nranks];
    // the weights' sums first: dx may be written over x or dy
    if (a.partial != nullptr)
      hipLaunchKernelGGL((layerNormWeightSums<DT>), dim3((a.cols + kLnBlock - 1) / kLnBlock, partialRows(rows)),
                         dim3(kLnBlock), 0, st, a);
    if (dx && rows > 0)
      hipLaunchKernelGGL((layerNormBackwardRows<DT, WT>), dim3(rowGrid(rows)), dim3(kLnBlock), 0, st, a);
    return hipGetLastError();
  }
};

template <int DT, int WT>
struct WeightGrads {
  static hipError_t run(const LnSumArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((layerNormWeightGrads<WT>), dim3((a.cols + kLnBlock - 1) / kLnBlock), dim3(kLnBlock), 0, st,
                       a);
    return hipGetLastError();
  }
};

void fillRows(LnArgs* a, const size_t* rows, int nranks, int first) {
  a->nranks = nranks - first < kLnRanks ? nranks - first : kLnRanks;
  a->rowStart[0] = 0;
  for (int r = 0; r < a->nranks; ++r) a->rowStart[r + 1] = a->rowStart[r] + (int64_t)rows[first + r];
}

arResult_t forward(const void* const* x, const void* const* gamma, const void* const* beta, void* const* y,
                   float* const* mean, float* const* rstd, const size_t* rows, int nranks, size_t cols,
                   size_t xStride, size_t yStride, float eps, int dtype, int wtype, hipStream_t st) {
  Shape s;
  if (!shapeOk(rows, nranks, cols, &s) || !strideOk(xStride, cols) || !strideOk(yStride, cols))
    return arInvalidArgument;
  if (!opsFloatType(dtype) || (wtype != dtype && wtype != arFloat32)) return arInvalidArgument;
  if (!(eps >= 0.0f) || eps > 3.4e38f) return arInvalidArgument;
  if ((mean == nullptr) != (rstd == nullptr)) return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  if (s.total == 0) return arSuccess;
  if (x == nullptr || y == nullptr) return arInvalidArgument;
  const int esz = elemSize(dtype), wsz = elemSize(wtype);
  std::vector<Extent> v;
  v.reserve((size_t)nranks * 6);
  for (int r = 0; r < nranks; ++r) {
    if (rows[r] == 0) continue;
    bool ok = addRows(v, x[r], rows[r], cols, xStride, esz, false, r) &&
              addRows(v, y[r], rows[r], cols, yStride, esz, true, r);
    if (gamma != nullptr) ok = ok && addFlat(v, gamma[r], cols, wsz, false);
    if (beta != nullptr) ok = ok && addFlat(v, beta[r], cols, wsz, false);
    if (mean != nullptr) ok = ok && addFlat(v, mean[r], rows[r], 4, true) && addFlat(v, rstd[r], rows[r], 4, true);
    if (!ok) return arInvalidArgument;
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  for (int l = 0; l < s.launches; ++l) {
    const int first = l * kLnRanks;
    LnArgs a{};
    fillRows(&a, rows, nranks, first);
    if (a.rowStart[a.nranks] == 0) continue;
    for (int r = 0; r < a.nranks; ++r) {
      if (rows[first + r] == 0) continue;
      a.x[r] = x[first + r];
      a.y[r] = y[first + r];
      a.gamma[r] = gamma ? gamma[first + r] : nullptr;
      a.beta[r] = beta ? beta[first + r] : nullptr;
      a.mean[r] = mean ? mean[first + r] : nullptr;
      a.rstd[r] = rstd ? rstd[first + r] : nullptr;
    }
    a.xStride = (int64_t)xStride;
    a.yStride = (int64_t)yStride;
    a.cols = (int)cols;
    a.eps = eps;
    if (byTypes<Forward, const LnArgs&, hipStream_t>(dtype, wtype, a, st) != hipSuccess) return arHipError;
  }
  return arSuccess;
}

arResult_t workspaceBytes(const size_t* rows, int nranks, size_t cols, size_t* bytes) {
  Shape s;
  if (bytes == nullptr || !shapeOk(rows, nranks, cols, &s)) return arInvalidArgument;
  size_t n = 0;
  for (int l = 0; l < s.launches; ++l) n += (size_t)partialRows(rowsOfLaunch(rows, nranks, l * kLnRanks));
  *bytes = n * 2 * cols * sizeof(float);
  return arSuccess;
}

arResult_t backward(const void* const* dy, const void* const* x, const void* const* gamma, const float* const* mean,
                    const float* const* rstd, void* const* dx, void* const* dgamma, void* const* dbeta,
                    const size_t* rows, int nranks, size_t cols, size_t dyStride, size_t xStride, size_t dxStride,
                    int dtype, int wtype, void* workspace, size_t workspaceGiven, hipStream_t st) {
  Shape s;
  if (!shapeOk(rows, nranks, cols, &s) || !strideOk(xStride, cols) || !strideOk(dyStride, cols) ||
      (dx != nullptr && !strideOk(dxStride, cols)))
    return arInvalidArgument;
  if (!opsFloatType(dtype) || (wtype != dtype && wtype != arFloat32)) return arInvalidArgument;
  if (dx == nullptr && dgamma == nullptr && dbeta == nullptr) return arInvalidArgument;
  if (groupOpen()) return arInvalidUsage;
  const bool weights = dgamma != nullptr || dbeta != nullptr;
  if (s.total > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)) return arInvalidArgument;
  const int esz = elemSize(dtype), wsz = elemSize(wtype);
  size_t need = 0;
  std::vector<Extent> v;
  v.reserve((size_t)nranks * 8 + 1);
  if (weights) {
    const arResult_t r = workspaceBytes(rows, nranks, cols, &need);
    if (r != arSuccess) return r;
    if (workspace == nullptr || (uintptr_t)workspace % 16 != 0 || workspaceGiven < need) return arInvalidArgument;
    v.push_back(Extent{(uintptr_t)workspace, need, 1, need, true, -1});
  }
  for (int r = 0; r < nranks; ++r) {
    bool ok = true;
    if (rows[r] > 0) {
      ok = addRows(v, dy[r], rows[r], cols, dyStride, esz, false, r) &&
           addRows(v, x[r], rows[r], cols, xStride, esz, false, r) && addFlat(v, mean[r], rows[r], 4, false) &&
           addFlat(v, rstd[r], rows[r], 4, false);
      if (dx != nullptr) ok = ok && addRows(v, dx[r], rows[r], cols, dxStride, esz, true, r);
      if (gamma != nullptr) ok = ok && addFlat(v, gamma[r], cols, wsz, false);
    }
    if (dgamma != nullptr) ok = ok && addFlat(v, dgamma[r], cols, wsz, true);
    if (dbeta != nullptr) ok = ok && addFlat(v, dbeta[r], cols, wsz, true);
    if (!ok) return arInvalidArgument;
  }
  if (outputsOverlap(v)) return arInvalidArgument;
  int nPartial = 0;
  for (int l = 0; l < s.launches; ++l) {
    const int first = l * kLnRanks;
    LnArgs a{};
    fillRows(&a, rows, nranks, first);
    const int64_t n = a.rowStart[a.nranks];
    if (n == 0 && !weights) continue;
    for (int r = 0; r < a.nranks; ++r) {
      if (rows[first + r] == 0) continue;
      a.x[r] = x[first + r];
      a.dy[r] = dy[first + r];
      a.y[r] = dx ? dx[first + r] : nullptr;
      a.gamma[r] = gamma ? gamma[first + r] : nullptr;
      a.mean[r] = const_cast<float*>(mean[first + r]);
      a.rstd[r] = const_cast<float*>(rstd[first + r]);
    }
    a.xStride = (int64_t)xStride;
    a.dyStride = (int64_t)dyStride;
    a.yStride = (int64_t)dxStride;
    a.cols = (int)cols;
    if (weights) a.partial = (float*)workspace + (size_t)nPartial * 2 * cols;
    nPartial += partialRows(n);
    if (byTypes<Backward, const LnArgs&, bool, hipStream_t>(dtype, wtype, a, dx != nullptr, st) != hipSuccess)
      return arHipError;
  }
  if (!weights) return arSuccess;
  LnSumArgs g{};
  for (int r = 0; r < nranks; ++r) {
    g.dgamma[r] = dgamma ? dgamma[r] : nullptr;
    g.dbeta[r] = dbeta ? dbeta[r] : nullptr;
  }
  g.partial = (const float*)workspace;
  g.nPartial = nPartial;
  g.nranks = nranks;
  g.cols = (int)cols;
  return byTypes<WeightGrads, const LnSumArgs&, hipStream_t>(dtype, wtype, g, st) == hipSuccess ? arSuccess
                                                                                                : arHipError;
}

}  // namespace
}  // namespace ar

extern "C" arResult_t arLayerNorm(const void* const* x, const void* const* gamma, const void* const* beta,
                                  void* const* y, float* const* mean, float* const* rstd, const size_t* rows,
                                  int nranks, size_t cols, size_t xStride, size_t yStride, float eps,
                                  arDataType_t dtype, arDataType_t wtype, void* stream) {
  ApiRange range("arLayerNorm");
  try {
    return ar::noteGroupError(ar::forward(x, gamma, beta, y, mean, rstd, rows, nranks, cols, xStride, yStride, eps,
                                          dtype, wtype, (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}

extern "C" arResult_t arLayerNormBackwardWorkspace(const size_t* rows, int nranks, size_t cols, size_t* bytes) {
  return ar::workspaceBytes(rows, nranks, cols, bytes);
}

extern "C" arResult_t arLayerNormBackward(const void* const* dy, const void* const* x, const void* const* gamma,
                                          const float* const* mean, const float* const* rstd, void* const* dx,
                                          void* const* dgamma, void* const* dbeta, const size_t* rows, int nranks,
                                          size_t cols, size_t dyStride, size_t xStride, size_t dxStride,
                                          arDataType_t dtype, arDataType_t wtype, void* workspace,
                                          size_t workspaceBytes, void* stream) {
  ApiRange range("arLayerNormBackward");
  try {
    return ar::noteGroupError(ar::backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, rows, nranks, cols, dyStride,
                                           xStride, dxStride, dtype, wtype, workspace, workspaceBytes,
                                           (hipStream_t)stream));
  } catch (const std::bad_alloc&) {
    return ar::noteGroupError(arSystemError);
  }
}
