// ar_layernorm.hip -- layer norm over the rows of N virtual ranks: forward,
// backward, and the weights' gradient summed over every rank's rows.
//
// Forward, a row of C values:  m = sum x / C,  v = sum (x - m)^2 / C,
// r = 1 / sqrt(v + eps),  y = (x - m) r g + b.  The variance is taken about
// the mean (not as the mean square less the squared mean): a large offset costs
// what rounding the sum and the mean to 32 bits costs, and no more.  Rows of one
// value whose sums are exact come out as b.
// Backward, h = (x - m) r, q = dy g:  dx = r (q - sum q / C - h sum(q h) / C),
// dg = sum over rows of dy h,  db = sum over rows of dy.
#include <cmath>
#include <new>
#include <vector>

#include "ar_api.h"
#include "ar_internal.h"
#include "ar_ops.h"

namespace ar {
namespace {

// Ranks per launch: their pointers travel in the kernel arguments, which every
// launch copies (1 KB; with 32 ranks' a one-row call took 0.4-1 us longer).
constexpr int kLnRanks = 16;
constexpr size_t kLnMaxCols = (size_t)1 << 30;
constexpr int64_t kLnMaxRows = 0x7fffffff;   // of all ranks
constexpr int kLnBlock = 256;

struct LnArgs {
  const void* x[kLnRanks];
  const void* gamma[kLnRanks];
  const void* other[kLnRanks];    // forward: beta, backward: dy
  void* y[kLnRanks];              // forward: y, backward: dx
  float* mean[kLnRanks];
  float* rstd[kLnRanks];
  int rowStart[kLnRanks + 1];     // rank r has rows [rowStart[r], rowStart[r + 1]) of the launch
  int blockStart[kLnRanks + 1];   // and workgroups [blockStart[r], blockStart[r + 1]), where they are shared out
  int64_t xStride, yStride, dyStride;
  int cols;
  int nranks;
  float eps;
  float* partial;                 // backward: this launch's first row of partial sums, or null
  int partialCols;                // cols up to a multiple of 4
  float* rowSums;                 // backward, rows that registers do not hold: two sums a row, or null
};

// The weights' gradients of every rank receive the same sums.
struct LnSumArgs {
  void* dgamma[AR_MAX_RANKS];
  void* dbeta[AR_MAX_RANKS];
  const float* partial;           // nPartial rows of [dgamma sums, dbeta sums], partialCols floats each
  int partialCols;
  int nPartial;
  int nranks;
  int cols;
};

struct LnFewArgs {
  LnArgs rows;
  void* dgamma[kLnRanks];         // null pointers: not wanted
  void* dbeta[kLnRanks];
  int dxRows;                     // workgroups that write dx
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
// ranks of 1000 rows of 40000 bf16: 87 us (95 on another box) with 1024 threads and 8 workgroups a
// CU, 94 with 2, 106 with 512 threads, 117 with 256.  A thread adds its vectors'
// sums up in 64 bits: a row of 2^20 columns is 1024 values a thread, whose
// roundings to 32 bits moved the mean of a row of 1000.1 by 0.01.
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
    const W* beta = (const W*)a.other[r];
    double s = 0.0;
    forRow<V, BLOCK>(a.cols,
                     [&](int c) {
                       const Vec v = loadVec<T, V>(x + c);
                       float u = 0.0f;
#pragma unroll
                       for (int e = 0; e < V; ++e) u += (float)v[e];
                       s += u;
                     },
                     [&](int c) { s += (float)x[c]; });
    const float mean = blockSum((float)s, lds) / (float)a.cols;
    double q = 0.0;
    forRow<V, BLOCK>(a.cols,
                     [&](int c) {
                       const Vec v = loadVec<T, V>(x + c);
                       float u = 0.0f;
#pragma unroll
                       for (int e = 0; e < V; ++e) u = fmaf((float)v[e] - mean, (float)v[e] - mean, u);
                       q += u;
                     },
                     [&](int c) { q += ((float)x[c] - mean) * ((float)x[c] - mean); });
    const float rstd = 1.0f / sqrtf(blockSum((float)q, lds) / (float)a.cols + a.eps);
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

// v, the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// A group of THREADS threads (part of a wavefront, one, or a workgroup) owns whole
// rows and keeps them in registers: thread t holds vectors t, t + THREADS, ...
// of a row, NP of them, so memory is read once and written once.  All but the
// last of a thread's vectors lie inside the row.  The last is moved back to
// end with the row where it would pass it, so that every load is one whole
// vector without a branch: `skip` of its elements then belong to another
// thread (all V where the vector lies wholly past the end).  They count in no
// sum; what they store is what their owner stores.
template <int NP, int V>
struct RowPieces {
  uint32_t first;    // first element of the first vector
  uint32_t stride;   // elements from a vector to the next
  uint32_t last;     // first element of the last vector
  int skip;          // its elements that are another thread's
  __device__ __forceinline__ RowPieces(int t, int threads, int cols)
      : first((uint32_t)(t * V)), stride((uint32_t)(threads * V)) {
    const int at = ((NP - 1) * threads + t) * V;
    last = (uint32_t)(at > cols - V ? cols - V : at);
    skip = at - (int)last < V ? at - (int)last : V;
  }
  __device__ __forceinline__ uint32_t offset(int p) const { return p < NP - 1 ? first + (uint32_t)p * stride : last; }
  __device__ __forceinline__ bool owns(int p, int e) const { return p < NP - 1 || e >= skip; }
  // A row starts at the same address for every thread, the offset inside it
  // fits 32 bits: one scalar base and one register of offset per access.
  template <typename T>
  __device__ __forceinline__ T* at(int p, T* row) const {
    return (T*)((char*)row + (uint32_t)(offset(p) * (uint32_t)sizeof(T)));
  }
  template <typename T, bool STREAM>
  __device__ __forceinline__ void load(typename VecOf<T, V>::type (&v)[NP], const T* row) const {
#pragma unroll
    for (int p = 0; p < NP; ++p)
      v[p] = STREAM ? loadStream<T, V>(at(p, const_cast<T*>(row))) : loadVec<T, V>(at(p, const_cast<T*>(row)));
  }
  template <typename T>
  __device__ __forceinline__ void store(int p, T* row, typename VecOf<T, V>::type v) const {
    if (p < NP - 1 || skip < V) storeStream<T, V>(at(p, row), v);
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

// Sums over a group's threads.  A workgroup's wavefronts leave theirs in LDS and
// every row of 16 lanes reads the 16 slots and adds them across its lanes (slots
// of wavefronts that the workgroup does not have hold zeros, see clearSlots).
// Two LDS buffers in turn: by the time one is written again every wavefront has
// passed the barrier after it was read.
struct SumSlots {
  float v[2][2][16];   // buffer, sum, wavefront
};

// Called by every thread before the first sum; that sum's barrier publishes it.
__device__ __forceinline__ void clearSlots(SumSlots& lds) {
  if (threadIdx.x < 64 && (int)(threadIdx.x % 16) >= (int)blockDim.x / kWave)
    (&lds.v[0][0][0])[threadIdx.x] = 0.0f;
}

template <int THREADS>
__device__ __forceinline__ float groupSum(float v, SumSlots& lds, int& turn) {
  if (THREADS <= kWave) return laneSum<(THREADS < kWave ? THREADS : kWave)>(v);
  v = waveSumLast(v);
  if (threadIdx.x % kWave == kWave - 1) lds.v[turn][0][threadIdx.x / kWave] = v;
  __syncthreads();
  v = rowSum(lds.v[turn][0][threadIdx.x % 16]);
  turn ^= 1;
  return v;
}

template <int THREADS>
__device__ __forceinline__ void groupSum2(float& v, float& u, SumSlots& lds, int& turn) {
  if (THREADS <= kWave) {
    v = laneSum<(THREADS < kWave ? THREADS : kWave)>(v);
    u = laneSum<(THREADS < kWave ? THREADS : kWave)>(u);
    return;
  }
  v = waveSumLast(v);
  u = waveSumLast(u);
  if (threadIdx.x % kWave == kWave - 1) {
    lds.v[turn][0][threadIdx.x / kWave] = v;
    lds.v[turn][1][threadIdx.x / kWave] = u;
  }
  __syncthreads();
  v = rowSum(lds.v[turn][0][threadIdx.x % 16]);
  u = rowSum(lds.v[turn][1][threadIdx.x % 16]);
  turn ^= 1;
}

// DEPTH rows are in registers at once: while one is reduced the loads of the
// others are in flight.  Bound by memory.  8 ranks of 4096 rows, 16-bit: 8192
// columns 180 us (6.0 TB/s; a bare copy of as much runs at 6.2), 4096 95 us,
// 2048 49 us; 200000 rows of 256 40 us, 2 ranks of 1000 rows of 32768 52 us.
// With the launch's rows taken in turn by all groups instead of each rank's by
// its own, 1024 columns took 67 us instead of 51 (every group met every rank's
// weights); with a run of rows per group instead of turns 8192 took 208
// instead of 194 (both with the grid the GPU holds at once).
template <int DT, int WT, int THREADS, int NP, int DEPTH>
__global__ void __launch_bounds__(THREADS < kLnBlock ? kLnBlock : THREADS) layerNormInRegisters(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = kVec<DT>, GROUPS = THREADS < kLnBlock ? kLnBlock / THREADS : 1;
  typedef typename VecOf<T, V>::type Vec;
  typedef typename VecOf<W, V>::type WVec;
  __shared__ SumSlots lds;
  int turn = 0;
  if (THREADS > kWave) clearSlots(lds);
  const int t = threadIdx.x % THREADS;
  int sub = GROUPS > 1 ? (int)threadIdx.x / THREADS : 0;
  if (THREADS == kWave) sub = __builtin_amdgcn_readfirstlane(sub);
  const int r = rankOfBlock(a);
  const int64_t rows = a.rowStart[r + 1] - a.rowStart[r];
  const int64_t step = (int64_t)(a.blockStart[r + 1] - a.blockStart[r]) * GROUPS;
  int64_t row = (int64_t)((int)blockIdx.x - a.blockStart[r]) * GROUPS + sub;
  if (row >= rows) return;
  const RowPieces<NP, V> pieces(t, THREADS, a.cols);
  const T* xs = (const T*)a.x[r];
  Vec x[DEPTH][NP];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (row + d * step < rows) pieces.template load<T, true>(x[d], xs + (row + d * step) * a.xStride);
  WVec g[NP], b[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    g[p] = (WVec)(W)1.0f;
    b[p] = (WVec)(W)0.0f;
  }
  if (a.gamma[r] != nullptr) pieces.template load<W, false>(g, (const W*)a.gamma[r]);
  if (a.other[r] != nullptr) pieces.template load<W, false>(b, (const W*)a.other[r]);
  // These and the mean in scalar registers: with one vector register more the
  // 512 x 2 layout holds 5 wavefronts a SIMD instead of 6 (8192 columns 189 us
  // instead of 181).
  const float cols = uniform((float)a.cols), inv = uniform(1.0f / cols);
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
      const float quotient = groupSum<THREADS>(s, lds, turn) / cols;   // not s times 1 / cols: rounded once
      const float mean = THREADS < kWave ? quotient : uniform(quotient);
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
        pieces.template store<T>(p, y, __builtin_convertvector(o, Vec));
      }
      if (t == 0 && a.mean[r] != nullptr) {
        a.mean[r][row] = mean;
        a.rstd[r][row] = rstd;
      }
      if (row + DEPTH * step < rows) pieces.template load<T, true>(x[d], xs + (row + DEPTH * step) * a.xStride);
      row += step;
      if (row >= rows) return;
    }
  }
}

// Stores the elements of a vector of sums that its thread owns; whole ones start
// at a multiple of 16 bytes of `row`, which is as aligned itself.
template <int V, typename Pieces>
__device__ __forceinline__ void storeOwned(const Pieces& pieces, int p, float* row, FloatVec<V> v) {
  float* to = row + pieces.offset(p);
  if (pieces.owns(p, 0)) {
#pragma unroll
    for (int e = 0; e < V; e += 4) *(FloatVec<4>*)(to + e) = FloatVec<4>{v[e], v[e + 1], v[e + 2], v[e + 3]};
  } else {
#pragma unroll
    for (int e = 1; e < V; ++e)
      if (pieces.owns(p, e)) to[e] = v[e];
  }
}

// The bits of a vector that its thread owns, to be and-ed with a vector.
template <int DT>
struct OwnBits {
  typedef uint32_t words __attribute__((ext_vector_type(4)));
  typedef typename VecOf<typename Elem<DT>::type, kVec<DT>>::type Vec;
  words bits;
  __device__ __forceinline__ explicit OwnBits(int skip) {
    constexpr int PER = kVec<DT> / 4;   // elements of a word: 1 or 2
#pragma unroll
    for (int w = 0; w < 4; ++w)
      bits[w] = PER == 1 ? (w >= skip ? 0xffffffffu : 0u)
                         : (2 * w >= skip ? 0xffffu : 0u) | (2 * w + 1 >= skip ? 0xffff0000u : 0u);
  }
  __device__ __forceinline__ Vec of(Vec v) const { return __builtin_bit_cast(Vec, __builtin_bit_cast(words, v) & bits); }
};

// The backward pass with a row's x and dy in registers.  With h = (x - m) r:
//   s = sum dy g,  u = sum dy g h,  dx = r (dy g - s / C - h u / C),
//   dg += dy h,  db += dy.
// h comes first: it is a number of ordinary size whatever the rows' spread,
// where dy (x - m) and r r may pass the ends of a float.
// A thread meets the same columns in every row, so it adds their weights'
// gradients up in registers too; a workgroup's groups are joined through LDS at
// the end, and each workgroup leaves one row of partial sums.  x - m is formed
// as it stands, not as x r - m r, which would cancel where the offset is large.
// Bound by memory at 8192 columns (8 ranks of 4096 rows, bf16: 286-290 us, 5.6
// TB/s, with the 8 us of the sums' kernel); a row costs a wavefront about 200
// instructions at 8 values a thread, which shows where rows are short: 2048
// columns 85 us for 403 MB, 128 columns 60 us for 310 MB.
template <int DT, int WT, int THREADS, int NP, int DEPTH, int WAVES>
__global__ void __launch_bounds__(THREADS < kLnBlock ? kLnBlock : THREADS) __attribute__((amdgpu_waves_per_eu(WAVES)))
layerNormBackwardInRegisters(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = kVec<DT>, GROUPS = THREADS < kLnBlock ? kLnBlock / THREADS : 1;
  typedef typename VecOf<T, V>::type Vec;
  typedef typename VecOf<W, V>::type WVec;
  __shared__ SumSlots lds;
  __shared__ __align__(16) float joined[GROUPS > 1 ? GROUPS * 2 * THREADS * NP * V : 1];
  int turn = 0;
  const int threads = GROUPS > 1 ? THREADS : (int)blockDim.x;
  const int t = GROUPS > 1 ? (int)threadIdx.x % THREADS : (int)threadIdx.x;
  int sub = GROUPS > 1 ? (int)threadIdx.x / THREADS : 0;
  if (THREADS == kWave) sub = __builtin_amdgcn_readfirstlane(sub);
  if (THREADS > kWave) clearSlots(lds);
  const int r = rankOfBlock(a);
  const int64_t rows = a.rowStart[r + 1] - a.rowStart[r];
  const int64_t step = (int64_t)(a.blockStart[r + 1] - a.blockStart[r]) * GROUPS;
  int64_t row = (int64_t)((int)blockIdx.x - a.blockStart[r]) * GROUPS + sub;
  const RowPieces<NP, V> pieces(t, threads, a.cols);
  const OwnBits<DT> own(pieces.skip);
  const T* xs = (const T*)a.x[r];
  const T* dys = (const T*)a.other[r];
  T* dxs = (T*)a.y[r];
  const float* means = a.mean[r];
  const float* rstds = a.rstd[r];
  Vec x[DEPTH][NP], dy[DEPTH][NP];
  float mean[DEPTH], rstd[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    const int64_t at = row + d * step;
    if (at < rows) {
      pieces.template load<T, true>(x[d], xs + at * a.xStride);
      pieces.template load<T, true>(dy[d], dys + at * a.dyStride);
      mean[d] = means[at];
      rstd[d] = rstds[at];
    }
  }
  WVec g[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) g[p] = (WVec)(W)1.0f;
  if (a.gamma[r] != nullptr) pieces.template load<W, false>(g, (const W*)a.gamma[r]);
  FloatVec<V> dg[NP], db[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    dg[p] = (FloatVec<V>)0.0f;
    db[p] = (FloatVec<V>)0.0f;
  }
  const float inv = 1.0f / (float)a.cols;
  while (row < rows) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      float s = 0.0f, u = 0.0f;
      FloatVec<V> h[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const Vec mine = p < NP - 1 ? dy[d][p] : own.of(dy[d][p]);
        float sp = 0.0f, up = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float o = (float)mine[e], q = o * (float)g[p][e];
          h[p][e] = ((float)x[d][p][e] - mean[d]) * rstd[d];
          sp += q;
          up = fmaf(q, h[p][e], up);
          dg[p][e] = fmaf(o, h[p][e], dg[p][e]);
          db[p][e] += o;
        }
        s += sp;
        u += up;
      }
      if (dxs != nullptr) {
        groupSum2<THREADS>(s, u, lds, turn);
        s *= inv;
        u *= inv;
        T* dx = dxs + row * a.yStride;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          FloatVec<V> o;
#pragma unroll
          for (int e = 0; e < V; ++e)
            o[e] = rstd[d] * fmaf(-h[p][e], u, fmaf((float)dy[d][p][e], (float)g[p][e], -s));
          pieces.template store<T>(p, dx, __builtin_convertvector(o, Vec));
        }
      }
      const int64_t at = row + DEPTH * step;
      if (at < rows) {
        pieces.template load<T, true>(x[d], xs + at * a.xStride);
        pieces.template load<T, true>(dy[d], dys + at * a.dyStride);
        mean[d] = means[at];
        rstd[d] = rstds[at];
      }
      row += step;
      if (row >= rows) break;
    }
  }
  if (a.partial == nullptr) return;
  float* sums = a.partial + (size_t)blockIdx.x * 2 * a.partialCols;
  if (GROUPS == 1) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      storeOwned<V>(pieces, p, sums, dg[p]);
      storeOwned<V>(pieces, p, sums + a.partialCols, db[p]);
    }
    return;
  }
  constexpr int WIDTH = THREADS * NP * V;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    storeOwned<V>(pieces, p, joined + sub * 2 * WIDTH, dg[p]);
    storeOwned<V>(pieces, p, joined + (sub * 2 + 1) * WIDTH, db[p]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += kLnBlock) {
    float u = 0.0f, v = 0.0f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      u += joined[k * 2 * WIDTH + c];
      v += joined[(k * 2 + 1) * WIDTH + c];
    }
    sums[c] = u;
    sums[a.partialCols + c] = v;
  }
}

// A workgroup's row: its sums s / C and u / C, and dx from them, for which the
// row is read again, or (SUMS) the sums alone to rowSums.
template <int DT, int WT, int BLOCK, bool SUMS>
__device__ __forceinline__ void backwardRow(const LnArgs& a, int64_t row, float* lds) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = kVec<DT>;
  typedef typename VecOf<T, V>::type Vec;
  typedef typename VecOf<W, V>::type WVec;
  const int r = rankOfRow(a, row);
  const int64_t i = row - a.rowStart[r];
  const T* x = (const T*)a.x[r] + i * a.xStride;
  const T* dy = (const T*)a.other[r] + i * a.dyStride;
  T* dx = (T*)a.y[r] + i * a.yStride;
  const W* gamma = (const W*)a.gamma[r];
  const float mean = a.mean[r][i], rstd = a.rstd[r][i];
  double sums = 0.0, along = 0.0;   // as the forward pass
  forRow<V, BLOCK>(a.cols,
                   [&](int c) {
                     const Vec v = loadVec<T, V>(x + c), o = loadVec<T, V>(dy + c);
                     const WVec g = gamma ? loadVec<W, V>(gamma + c) : (WVec)(W)1.0f;
                     float s = 0.0f, u = 0.0f;
#pragma unroll
                     for (int e = 0; e < V; ++e) {
                       const float q = (float)o[e] * (float)g[e];
                       s += q;
                       u = fmaf(q, ((float)v[e] - mean) * rstd, u);
                     }
                     sums += s;
                     along += u;
                   },
                   [&](int c) {
                     const float q = (float)dy[c] * (gamma ? (float)gamma[c] : 1.0f);
                     sums += q;
                     along += q * (((float)x[c] - mean) * rstd);
                   });
  const float s = blockSum((float)sums, lds) / (float)a.cols;
  const float u = blockSum((float)along, lds) / (float)a.cols;
  if (SUMS) {
    if (threadIdx.x == 0) {
      a.rowSums[2 * row] = s;
      a.rowSums[2 * row + 1] = u;
    }
    return;
  }
  forRow<V, BLOCK>(a.cols,
                   [&](int c) {
                     const Vec v = loadVec<T, V>(x + c), o = loadVec<T, V>(dy + c);
                     const WVec g = gamma ? loadVec<W, V>(gamma + c) : (WVec)(W)1.0f;
                     FloatVec<V> d;
#pragma unroll
                     for (int e = 0; e < V; ++e)
                       d[e] = rstd * fmaf(-(((float)v[e] - mean) * rstd), u, fmaf((float)o[e], (float)g[e], -s));
                     storeVec<T, V>(dx + c, __builtin_convertvector(d, Vec));
                   },
                   [&](int c) {
                     dx[c] = (T)(rstd * fmaf(-(((float)x[c] - mean) * rstd), u,
                                             fmaf((float)dy[c], gamma ? (float)gamma[c] : 1.0f, -s)));
                   });
}

// Rows too wide for registers, or narrower than a vector.
template <int DT, int WT, int BLOCK, bool SUMS>
__global__ void __launch_bounds__(BLOCK) layerNormBackwardRows(const LnArgs a) {
  __shared__ float lds[BLOCK / kWave];
  const int64_t rows = a.rowStart[a.nranks];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) backwardRow<DT, WT, BLOCK, SUMS>(a, row, lds);
}

// The weights' sums of such rows, and dx where the rows' sums are given (so x and
// dy are read twice in all: 2 ranks of 1000 rows of 40000 bf16 174 us; 210 with
// dx from the rows' kernel and a third reading here): a thread
// per vector of columns and slice of the rows, four rows at a time; ONE takes
// single columns (rows of less than a vector and the columns behind the last
// whole one).  dx may be written over x or dy: an element is read here by the
// thread that writes it and by no other.
template <int DT, int WT, bool ONE>
__global__ void __launch_bounds__(kLnBlock) layerNormBackwardColumns(const LnArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = ONE ? 1 : kVec<DT>, UN = 4;
  typedef typename VecOf<T, V>::type Vec;
  const int first = ONE ? a.cols / kVec<DT> * kVec<DT> : 0;
  const int c = first + ((int)blockIdx.x * kLnBlock + (int)threadIdx.x) * V;
  if (c + V > a.cols) return;
  const int64_t rows = a.rowStart[a.nranks];
  const int64_t lo = rows * blockIdx.y / gridDim.y, hi = rows * (blockIdx.y + 1) / gridDim.y;
  FloatVec<V> dg = (FloatVec<V>)0.0f, db = (FloatVec<V>)0.0f;
  for (int r = 0; r < a.nranks; ++r) {
    const int64_t from = (lo > a.rowStart[r] ? lo : a.rowStart[r]) - a.rowStart[r];
    const int64_t to = (hi < a.rowStart[r + 1] ? hi : a.rowStart[r + 1]) - a.rowStart[r];
    if (from >= to) continue;
    const T* x = (const T*)a.x[r] + c;
    const T* dy = (const T*)a.other[r] + c;
    T* dx = (T*)a.y[r] + c;
    FloatVec<V> g = (FloatVec<V>)1.0f;
    if (a.gamma[r] != nullptr)
      g = __builtin_convertvector((loadVec<W, V>((const W*)a.gamma[r] + c)), FloatVec<V>);
    for (int64_t i = from; i < to; i += UN) {
      Vec v[UN], o[UN];
#pragma unroll
      for (int k = 0; k < UN; ++k)
        if (i + k < to) {
          v[k] = loadStream<T, V>(x + (i + k) * a.xStride);
          o[k] = loadStream<T, V>(dy + (i + k) * a.dyStride);
        }
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        if (i + k >= to) break;
        const float mean = a.mean[r][i + k], rstd = a.rstd[r][i + k];
        float s = 0.0f, u = 0.0f;
        if (a.rowSums != nullptr) {
          s = a.rowSums[2 * (a.rowStart[r] + i + k)];
          u = a.rowSums[2 * (a.rowStart[r] + i + k) + 1];
        }
        FloatVec<V> d;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float h = ((float)v[k][e] - mean) * rstd;
          dg[e] = fmaf((float)o[k][e], h, dg[e]);
          db[e] += (float)o[k][e];
          d[e] = rstd * fmaf(-h, u, fmaf((float)o[k][e], g[e], -s));
        }
        if (a.rowSums != nullptr)
          storeStream<T, V>(dx + (i + k) * a.yStride, __builtin_convertvector(d, Vec));
      }
    }
  }
  float* p = a.partial + (size_t)blockIdx.y * 2 * a.partialCols + c;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    p[e] = dg[e];
    p[a.partialCols + e] = db[e];
  }
}

// The sum of N slices' values in eight chains, joined in pairs: an eighth of the
// roundings of one chain.
template <int N, typename F>
__device__ __forceinline__ float joinSlices(F value) {
  static_assert(N % 8 == 0, "eight chains");
  float c[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) c[k] = value(k);
#pragma unroll
  for (int k = 8; k < N; ++k) c[k % 8] += value(k);
  return ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
}

// Few rows in one launch: the first workgroups take a row each and write dx,
// the others take 8 vectors of columns and add all rows up (32 slices of them,
// joined through LDS).  x and dy are read twice for dx (its sums first) and once
// for the weights, from the caches after the first time, but no partial sums
// leave a workgroup.  dx must not be written over x or dy.  256
// rows of 768 to 8192 columns bf16 4.3-7.1 us, 6.9-15.3 in two launches; 512
// rows 5.3-10.5 and 6.2-16.9; 1024 rows of 256 columns 8.4 and 6.6: no more
// than 512 rows come here.
constexpr int kFewRows = 512;
constexpr int kFewLanes = 8, kFewSlices = kLnBlock / kFewLanes;

template <int DT, int WT>
__global__ void __launch_bounds__(kLnBlock) layerNormBackwardFew(const LnFewArgs w) {
  const LnArgs& a = w.rows;
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  constexpr int V = kVec<DT>;
  typedef typename VecOf<T, V>::type Vec;
  struct RowAt {
    const T *x, *dy;
    const float *mean, *rstd;
  };
  __shared__ float sums[2][kFewSlices][kFewLanes * V];
  __shared__ RowAt at[kFewRows];
  if ((int)blockIdx.x < w.dxRows) {
    backwardRow<DT, WT, kLnBlock, false>(a, blockIdx.x, &sums[0][0][0]);
    return;
  }
  // where each row lies, so that rows of all ranks are read side by side
  for (int r = 0; r < a.nranks; ++r) {
    const int from = a.rowStart[r], rows = a.rowStart[r + 1] - from;
    for (int i = threadIdx.x; i < rows; i += kLnBlock)
      at[from + i] = RowAt{(const T*)a.x[r] + i * a.xStride, (const T*)a.other[r] + i * a.dyStride, a.mean[r] + i,
                           a.rstd[r] + i};
  }
  __syncthreads();
  const int rows = a.rowStart[a.nranks];
  const int lane = threadIdx.x % kFewLanes, slice = threadIdx.x / kFewLanes;
  const int step = ((int)gridDim.x - w.dxRows) * kFewLanes * V;
  for (int first = ((int)blockIdx.x - w.dxRows) * kFewLanes * V; first < a.cols; first += step) {
    // the last vector is moved back to end with the row; a column then summed
    // twice has the same sum twice
    const int c = first + lane * V > a.cols - V ? a.cols - V : first + lane * V;
    FloatVec<V> dg = (FloatVec<V>)0.0f, db = (FloatVec<V>)0.0f;
#pragma unroll 4
    for (int i = slice; i < rows; i += kFewSlices) {
      const RowAt p = at[i];
      const Vec v = loadVec<T, V>(p.x + c), o = loadVec<T, V>(p.dy + c);
      const float mean = *p.mean, rstd = *p.rstd;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        dg[e] = fmaf((float)o[e], ((float)v[e] - mean) * rstd, dg[e]);
        db[e] += (float)o[e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sums[0][slice][lane * V + e] = dg[e];
      sums[1][slice][lane * V + e] = db[e];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * kFewLanes * V; k += kLnBlock) {
      const int which = k / (kFewLanes * V), i = k % (kFewLanes * V);
      const int from = first + i / V * V;
      const int col = (from > a.cols - V ? a.cols - V : from) + i % V;
      void* const* out = which == 0 ? w.dgamma : w.dbeta;
      if (out[0] == nullptr) continue;
      const float all = joinSlices<kFewSlices>([&](int s) { return sums[which][s][i]; });
      for (int r = 0; r < a.nranks; ++r) ((W*)out[r])[col] = (W)all;
    }
    __syncthreads();   // before the next columns' sums
  }
}

// The partial sums of all workgroups and launches, 64 columns a workgroup: its
// 64 slices of 16 threads take every 64th row, then the slices are joined in
// order.  blockIdx.y: dgamma or dbeta.
constexpr int kSumBlock = 1024, kSumCols = 64, kSlices = kSumBlock / (kSumCols / 4);

template <int WT>
__global__ void __launch_bounds__(kSumBlock) layerNormWeightGrads(const LnSumArgs a) {
  typedef typename Elem<WT>::type W;
  __shared__ float lds[kSlices][kSumCols];
  void* const* out = blockIdx.y == 0 ? a.dgamma : a.dbeta;
  if (out[0] == nullptr) return;
  const int lane = threadIdx.x % (kSumCols / 4), slice = threadIdx.x / (kSumCols / 4);
  for (int first = (int)blockIdx.x * kSumCols; first < a.cols; first += (int)gridDim.x * kSumCols) {
    const int c = first + lane * 4;
    FloatVec<4> sum = (FloatVec<4>)0.0f;
    if (c < a.cols) {
      const float* p = a.partial + (size_t)blockIdx.y * a.partialCols + c;
#pragma unroll 4
      for (int k = slice; k < a.nPartial; k += kSlices) sum += *(const FloatVec<4>*)(p + (size_t)k * 2 * a.partialCols);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) lds[slice][lane * 4 + e] = sum[e];
    __syncthreads();
    const int col = first + (int)threadIdx.x;
    if (threadIdx.x < kSumCols && col < a.cols) {
      const float all = joinSlices<kSlices>([&](int k) { return lds[k][threadIdx.x]; });
      for (int r = 0; r < a.nranks; ++r) ((W*)out[r])[col] = (W)all;
    }
    __syncthreads();   // before the next columns' sums
  }
}

// A launch holds fewer than 2^32 threads along its grid: `blocks` workgroups
// of `block` threads, as many as fit into half of that.  The kernels of the
// weights' gradients step through the columns that are left over.
unsigned gridOf(int64_t blocks, int block) {
  const int64_t most = ((int64_t)1 << 31) / block;
  return (unsigned)(blocks < most ? blocks : most);
}

// How a backward launch is cut: `threads` threads hold a row, `pieces` vectors
// each (0 threads: the kernels for rows that registers do not hold), and at
// most `most` workgroups.
struct BackwardCut {
  int threads, pieces;
  int groups;   // of a workgroup
  int most;
};

BackwardCut backwardCut(int cols, int esz) {
  const int V = 16 / esz, vecs = (cols + V - 1) / V;
  if (cols < V || vecs > (esz == 4 ? 4096 : 2048)) {
    // the weights' sums alone of 2 ranks of 1000 rows of 32768: 59 us with 64
    // slices of the rows, 92 with 256
    const int wide = (vecs + kLnBlock - 1) / kLnBlock;   // workgroups across the columns
    return {0, 0, 1, wide < 64 ? 4 * kOpsCUs / wide : 16};
  }
  // One vector a thread as long as a workgroup reaches: 8192 columns 16-bit
  // 286-290 us with 1024 x 1 and three rows in flight, 292-297 with 512 x 2
  // (two rows; 160 registers a thread), 315 with one row in flight; 4096
  // columns 155 with 512 x 1, 163 with 256 x 2.  About 12 wavefronts a CU: each
  // workgroup costs a row of partial sums to write and read (2048 columns 85
  // us, 88 with 20 wavefronts; 8192 columns fill a CU with one workgroup).
  // Narrow rows, one vector a thread: 256 columns 57 us with 2 workgroups of
  // four wavefronts a CU, 73 with 1, 60 with 3, 63 with 4; two vectors: 1024
  // columns 79 with 4 (three rows in flight; 81 with two), 85 with 3.
  if (vecs <= 16) return {16, 1, 16, 2 * kOpsCUs};
  if (vecs <= 32) return {32, 1, 8, 2 * kOpsCUs};
  if (vecs <= 64) return {64, 1, 4, 2 * kOpsCUs};
  if (vecs <= 128) return {64, 2, 4, 4 * kOpsCUs};
  const int pieces = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : vecs <= 3 * 1024 ? 3 : 4;
  const int waves = ((vecs + pieces - 1) / pieces + kWave - 1) / kWave;
  return {waves * kWave, pieces, 1, (waves <= 12 ? 12 / waves : 1) * kOpsCUs};
}

// Rows of partial sums that a launch of `rows` rows of all its ranks leaves at
// most: its workgroups.  Each costs a row of partial sums to write and read, so
// few rows take few: at least 4 rows a workgroup (1024 rows x 2048 bf16 10.7
// us; 17.2 with 1 row, 12.1 with 3, 11.1 with 6, 13.9 with 12; 600 rows x 8192
// 17.6, 17.3, 17.1, 18.8, 23.8), 2 a group where it has several (4096 x 768
// 11.5, 16.6 with 1; 1024 x 768 7.9, 8.8 with 4).
int partialRows(int64_t rows, const BackwardCut& k) {
  const int each = k.groups > 1 ? 2 * k.groups : k.threads > 0 ? 4 : 1;
  const int64_t most = (rows + each - 1) / each;
  return (int)(most < 1 ? 1 : most > k.most ? k.most : most);
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
    if (rows[r] > (size_t)kLnMaxRows) return false;
    s->total += (int64_t)rows[r];
  }
  if (s->total > kLnMaxRows) return false;
  s->launches = (nranks + kLnRanks - 1) / kLnRanks;
  return true;
}

bool strideOk(size_t stride, size_t cols) { return stride >= cols && stride <= (size_t)1 << 48; }

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

// Shares `most` workgroups of `groups` rows at a time out among the ranks by
// their rows, at least one to a rank with rows (so more than `most` only where
// there are more such ranks); returns the grid.
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

// What RowPieces assumes: all of a thread's vectors but the last lie inside the
// row, and the last ones reach its end.
bool rowFits(int cols, int V, int threads, int pieces) {
  return cols >= V && cols >= (pieces - 1) * threads * V && cols <= pieces * threads * V;
}

template <int DT, int WT, int THREADS, int NP, int DEPTH>
hipError_t launchForward(LnArgs a, hipStream_t st) {
  if (!rowFits(a.cols, kVec<DT>, THREADS, NP)) return hipErrorInvalidValue;
  constexpr int BLOCK = THREADS < kLnBlock ? kLnBlock : THREADS;
  static const int resident = [] {
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, layerNormInRegisters<DT, WT, THREADS, NP, DEPTH>, BLOCK, 0) !=
        hipSuccess || n < 1)
      n = 1;
    return n;
  }();
  // Many rows take several rounds of workgroups: they start in order and each
  // as another ends, which keeps the window over memory closer than a lasting
  // grid whose workgroups drift apart does (8 ranks x 4096 rows of 8192
  // columns 194 us in one round, 189, 187, 180, 182 in 2, 4, 8, 16).  Each
  // loads the weights again, so it gets 4 rows at least, 16 where a row is
  // wider than 1024 vectors (16384 columns 98 us in one round, 97, 101, 106 in
  // 2, 4, 8); rows that do not start at 16 bytes gain nothing (12000 of 5001
  // columns 50 us, 55 in 2).
  const int64_t each = a.rowStart[a.nranks] / ((int64_t)resident * kOpsCUs * (BLOCK / THREADS)) /
                       (THREADS * NP > 1024 ? 16 : 4);
  const bool aligned16 = (a.xStride | a.yStride) % kVec<DT> == 0;
  const int rounds = !aligned16 || each < 1 ? 1 : each > 8 ? 8 : (int)each;
  const int grid = shareBlocks(&a, BLOCK / THREADS, resident * kOpsCUs * rounds);
  return launchKernel(layerNormInRegisters<DT, WT, THREADS, NP, DEPTH>, dim3(grid), dim3(BLOCK), a, st);
}

template <int DT, int WT, int BLOCK>
hipError_t launchRows(const LnArgs& a, hipStream_t st) {
  const int64_t rows = a.rowStart[a.nranks];
  const int most = (BLOCK < 128 ? 32 : 8) * kOpsCUs;
  return launchKernel(layerNormRows<DT, WT, BLOCK>, dim3((unsigned)(rows < most ? rows : most)), dim3(BLOCK), a, st);
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
    if (a.cols < kVec<DT>) return launchRows<DT, WT, 64>(a, st);
    if (vecs <= 16) return launchForward<DT, WT, 16, 1, 4>(a, st);
    if (vecs <= 32) return launchForward<DT, WT, 32, 1, 4>(a, st);
    if (vecs <= 64) return launchForward<DT, WT, 64, 1, 4>(a, st);
    if (vecs <= 128) return launchForward<DT, WT, 64, 2, 2>(a, st);
    if (vecs <= 192) return launchForward<DT, WT, 64, 3, 2>(a, st);
    if (vecs <= 256) return launchForward<DT, WT, 64, 4, 2>(a, st);
    if (vecs <= 512) return launchForward<DT, WT, 256, 2, 2>(a, st);
    if (vecs <= 768) return launchForward<DT, WT, 256, 3, 2>(a, st);
    if (vecs <= 1024) return launchForward<DT, WT, 512, 2, 2>(a, st);
    if (vecs <= 1536) return launchForward<DT, WT, 512, 3, 2>(a, st);
    if (vecs <= 2048) return launchForward<DT, WT, 512, 4, 2>(a, st);
    if (vecs <= 3 * 1024) return launchForward<DT, WT, 1024, 3, 1>(a, st);
    if (vecs <= 4096) return launchForward<DT, WT, 1024, 4, 1>(a, st);
    return launchRows<DT, WT, 1024>(a, st);
  }
};

template <int DT, int WT, int THREADS, int NP, int DEPTH, int WAVES>
hipError_t launchBackward(LnArgs a, const BackwardCut& k, int* partials, hipStream_t st) {
  if (!rowFits(a.cols, kVec<DT>, k.threads, k.pieces) || k.threads > THREADS || k.pieces != NP)
    return hipErrorInvalidValue;
  *partials = shareBlocks(&a, k.groups, partialRows(a.rowStart[a.nranks], k));
  return launchKernel(layerNormBackwardInRegisters<DT, WT, THREADS, NP, DEPTH, WAVES>, dim3(*partials),
                      dim3(THREADS < kLnBlock ? kLnBlock : k.threads), a, st);
}

// Rows that registers do not hold: dx alone, or the rows' sums and then the
// columns with dx, or the columns alone.
template <int DT, int WT>
hipError_t launchBackwardWide(const LnArgs& a, const BackwardCut& k, int* partials, hipStream_t st) {
  constexpr int V = kVec<DT>;
  const bool narrow = a.cols < V;
  const int64_t rows = a.rowStart[a.nranks];
  const int most = (narrow ? 32 : 8) * kOpsCUs;
  const dim3 grid((unsigned)(rows < most ? rows : most)), block(narrow ? 64 : 1024);
  if (a.partial == nullptr)
    return launchKernel(narrow ? layerNormBackwardRows<DT, WT, 64, false> : layerNormBackwardRows<DT, WT, 1024, false>,
                        grid, block, a, st);
  hipError_t e = hipSuccess;
  if (a.rowSums != nullptr)
    e = launchKernel(narrow ? layerNormBackwardRows<DT, WT, 64, true> : layerNormBackwardRows<DT, WT, 1024, true>,
                     grid, block, a, st);
  *partials = partialRows(rows, k);
  if (e == hipSuccess && !narrow)
    e = launchKernel(layerNormBackwardColumns<DT, WT, false>, dim3((a.cols / V + kLnBlock - 1) / kLnBlock, *partials),
                     dim3(kLnBlock), a, st);
  if (e == hipSuccess && a.cols % V != 0)
    e = launchKernel(layerNormBackwardColumns<DT, WT, true>, dim3(1, *partials), dim3(kLnBlock), a, st);
  return e;
}

// Runs the backward pass of a launch with rows; *partials receives the rows of
// partial sums it leaves.
template <int DT, int WT>
struct Backward {
  static hipError_t run(const LnArgs& a, int* partials, hipStream_t st) {
    constexpr int V = kVec<DT>;
    const BackwardCut k = backwardCut(a.cols, 16 / V);
    if (k.threads == 0) return launchBackwardWide<DT, WT>(a, k, partials, st);
    if (k.threads == 16) return launchBackward<DT, WT, 16, 1, 2, 1>(a, k, partials, st);
    if (k.threads == 32) return launchBackward<DT, WT, 32, 1, 2, 1>(a, k, partials, st);
    if (k.threads == 64 && k.pieces == 1) return launchBackward<DT, WT, 64, 1, 2, 1>(a, k, partials, st);
    if (k.threads == 64) return launchBackward<DT, WT, 64, 2, 3, 2>(a, k, partials, st);
    if (k.pieces == 1 && k.threads <= 256) return launchBackward<DT, WT, 256, 1, 3, 3>(a, k, partials, st);
    if (k.pieces == 1 && k.threads <= 512) return launchBackward<DT, WT, 512, 1, 3, 3>(a, k, partials, st);
    if (k.pieces == 1) return launchBackward<DT, WT, 1024, 1, 3, 4>(a, k, partials, st);
    if (k.pieces == 2) return launchBackward<DT, WT, 1024, 2, 1, 4>(a, k, partials, st);
    if constexpr (V == 4) {
      if (k.pieces == 3) return launchBackward<DT, WT, 1024, 3, 1, 4>(a, k, partials, st);
      return launchBackward<DT, WT, 1024, 4, 1, 4>(a, k, partials, st);
    }
    return hipErrorInvalidValue;
  }
};

template <int DT, int WT>
struct BackwardFew {
  static hipError_t run(const LnFewArgs& w, hipStream_t st) {
    constexpr int V = kVec<DT>;
    const unsigned across = gridOf((w.rows.cols + kFewLanes * V - 1) / (kFewLanes * V), kLnBlock);
    return launchKernel(layerNormBackwardFew<DT, WT>, dim3((unsigned)w.dxRows + across), dim3(kLnBlock), w, st);
  }
};

template <int DT, int WT>
struct WeightGrads {
  static hipError_t run(const LnSumArgs& a, hipStream_t st) {
    const unsigned across = gridOf((a.cols + kSumCols - 1) / kSumCols, kSumBlock);
    return launchKernel(layerNormWeightGrads<WT>, dim3(across, 2), dim3(kSumBlock), a, st);
  }
};

void fillRows(LnArgs* a, const size_t* rows, int nranks, int first) {
  a->nranks = nranks - first < kLnRanks ? nranks - first : kLnRanks;
  a->rowStart[0] = 0;
  for (int r = 0; r < a->nranks; ++r) a->rowStart[r + 1] = a->rowStart[r] + (int)rows[first + r];
}

arResult_t forward(const void* const* x, const void* const* gamma, const void* const* beta, void* const* y,
                   float* const* mean, float* const* rstd, const size_t* rows, int nranks, size_t cols,
                   size_t xStride, size_t yStride, float eps, int dtype, int wtype, hipStream_t st) {
  Shape s;
  if (!shapeOk(rows, nranks, cols, &s) || !strideOk(xStride, cols) || !strideOk(yStride, cols))
    return arInvalidArgument;
  if (!opsFloatType(dtype) || (wtype != dtype && wtype != arFloat32)) return arInvalidArgument;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return arInvalidArgument;
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
      a.other[r] = beta ? beta[first + r] : nullptr;
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

// The workspace's end: two sums for each row of the largest launch, for widths
// that are not held in registers with some element type.
size_t rowSumsBytes(const size_t* rows, int nranks, int launches, int cols) {
  if (backwardCut(cols, 2).threads != 0 && backwardCut(cols, 4).threads != 0) return 0;
  int64_t most = 0;
  for (int l = 0; l < launches; ++l) {
    const int64_t n = rowsOfLaunch(rows, nranks, l * kLnRanks);
    most = n > most ? n : most;
  }
  return ((size_t)most * 2 * sizeof(float) + 15) / 16 * 16;
}

arResult_t workspaceBytes(const size_t* rows, int nranks, size_t cols, size_t* bytes) {
  Shape s;
  if (bytes == nullptr || !shapeOk(rows, nranks, cols, &s)) return arInvalidArgument;
  // the element type is not known here: the larger of both cuts
  size_t most = 0;
  for (int esz = 2; esz <= 4; esz += 2) {
    const BackwardCut k = backwardCut((int)cols, esz);
    size_t n = 0;
    for (int l = 0; l < s.launches; ++l) {
      const int64_t launchRows = rowsOfLaunch(rows, nranks, l * kLnRanks);
      const int blocks = launchRows > 0 ? partialRows(launchRows, k) : 0;
      n += (size_t)(blocks > 0 && blocks < kLnRanks ? kLnRanks : blocks);   // one at least for each rank with rows
    }
    most = n > most ? n : most;
  }
  *bytes = (most > 0 ? most : 1) * 2 * ((cols + 3) / 4 * 4) * sizeof(float) +
           rowSumsBytes(rows, nranks, s.launches, (int)cols);
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
  bool inPlace = false;
  for (int r = 0; dx != nullptr && r < nranks; ++r)
    inPlace = inPlace || (rows[r] > 0 && (dx[r] == x[r] || dx[r] == dy[r]));
  int nPartial = 0;
  for (int l = 0; l < s.launches; ++l) {
    const int first = l * kLnRanks;
    LnFewArgs w{};
    LnArgs& a = w.rows;
    fillRows(&a, rows, nranks, first);
    const int64_t n = a.rowStart[a.nranks];
    if (n == 0) continue;
    for (int r = 0; r < a.nranks; ++r) {
      if (rows[first + r] == 0) continue;
      a.x[r] = x[first + r];
      a.other[r] = dy[first + r];
      a.y[r] = dx ? dx[first + r] : nullptr;
      a.gamma[r] = gamma ? gamma[first + r] : nullptr;
      a.mean[r] = const_cast<float*>(mean[first + r]);
      a.rstd[r] = const_cast<float*>(rstd[first + r]);
    }
    a.xStride = (int64_t)xStride;
    a.dyStride = (int64_t)dyStride;
    a.yStride = (int64_t)dxStride;
    a.cols = (int)cols;
    a.partialCols = (int)((cols + 3) / 4 * 4);
    if (weights && s.launches == 1 && !inPlace && n <= kFewRows && (int)cols >= 16 / esz) {
      for (int r = 0; r < nranks; ++r) {
        w.dgamma[r] = dgamma ? dgamma[r] : nullptr;
        w.dbeta[r] = dbeta ? dbeta[r] : nullptr;
      }
      w.dxRows = dx != nullptr ? (int)n : 0;
      return byTypes<BackwardFew, const LnFewArgs&, hipStream_t>(dtype, wtype, w, st) == hipSuccess ? arSuccess
                                                                                                  : arHipError;
    }
    if (weights) {
      a.partial = (float*)workspace + (size_t)nPartial * 2 * a.partialCols;
      // launches follow each other on the stream and share the rows' sums at the workspace's end
      if (dx != nullptr && backwardCut((int)cols, esz).threads == 0)
        a.rowSums = (float*)((char*)workspace + need - rowSumsBytes(rows, nranks, s.launches, (int)cols));
    }
    int partials = 0;
    if (byTypes<Backward, const LnArgs&, int*, hipStream_t>(dtype, wtype, a, &partials, st) != hipSuccess)
      return arHipError;
    nPartial += partials;
  }
  if (!weights) return arSuccess;
  LnSumArgs g{};
  for (int r = 0; r < nranks; ++r) {
    g.dgamma[r] = dgamma ? dgamma[r] : nullptr;
    g.dbeta[r] = dbeta ? dbeta[r] : nullptr;
  }
  g.partial = (const float*)workspace;
  g.nPartial = nPartial;
  g.partialCols = (int)((cols + 3) / 4 * 4);
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
