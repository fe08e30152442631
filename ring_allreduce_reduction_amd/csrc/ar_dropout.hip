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
//
// Times in comments are of calls in a replayed graph; a call from the host takes
// about 1 us longer where it is short.
#include <cmath>
#include <new>
#include <vector>

#include "ar_rows.h"

namespace ar {
namespace {

// Bound by memory: what it takes to draw is hidden behind it (8 ranks x 4096
// rows of 8192 bf16 forward 242 us, and 244 with the draw left out).
constexpr int kDropBlock = 256;
// Backward each workgroup leaves a row of partial sums, so it is larger: 182 us
// with 512 threads, 191 with 256, 189-198 with 1024.
constexpr int kDropBackBlock = 512;
constexpr int kDropCols = 8;    // of a thread: one block of 128 bits

// How a launch is cut.  A slice of the rows is taken `together` rows at a time
// by `tiles` workgroups: each has `across` threads side by side on every one of
// these rows, or, `flat`, they follow each other through them (across: a row's).
struct DropCut {
  int across, together, tiles;
  bool flat;
};

// Ranks of a launch at most.  Up to kOpRanks of them travel in arguments of
// that size, which take the host less time to hand over (calls from it: 4 ranks'
// 64 rows of 768 fp32 4.3 us, 4.4 with twice the size; 8 ranks' 8 rows of 8192
// backward 6.1, 6.3; 20 ranks' through the binding 6.0, 8.2 in two launches).
constexpr int kDropRanks = 2 * kOpRanks;

struct DropCall {
  int64_t xStride, residualStride, yStride;
  int cols, nranks;
  DropCut cut;
  unsigned nearBlocks;              // so many workgroups have a slice's on one XCD
  uint32_t overTiles;               // 2^32 / tiles, rounded down, at most 2^32 - 1
  float overAcross;                 // 1 / cut.across; 0 where there is one row at a time
  uint32_t threshold;               // T in the upper half; with no element kept 1,
  uint32_t mask;                    // and 0 here: what is drawn is taken for 0
  bool stream;                      // host: past the caches
  float scale;
  uint32_t key0, key1;
  uint64_t offset;
  const uint64_t* step;
  float* partial;                   // backward: this launch's first row of partial sums, or null
  int partialCols;                  // cols up to a multiple of 8
};

template <int RANKS>
struct DropArgs : DropCall {
  const void* x[RANKS];             // forward: x, backward: dy
  const void* bias[RANKS];
  const void* residual[RANKS];
  void* y[RANKS];                   // forward: y, backward: dx or null
  uint32_t firstRow[RANKS];
  int rowStart[RANKS + 1];          // rank r has rows [rowStart[r], rowStart[r + 1]) of the launch
  int sliceStart[RANKS + 1];        // and slices of rows [sliceStart[r], sliceStart[r + 1])

  // Those of another size, whose ranks fit.
  template <int OTHER>
  static DropArgs of(const DropArgs<OTHER>& a) {
    DropArgs to{};
    (DropCall&)to = a;
    for (int r = 0; r < a.nranks; ++r) {
      to.x[r] = a.x[r];
      to.bias[r] = a.bias[r];
      to.residual[r] = a.residual[r];
      to.y[r] = a.y[r];
      to.firstRow[r] = a.firstRow[r];
    }
    for (int r = 0; r <= a.nranks; ++r) {
      to.rowStart[r] = a.rowStart[r];
      to.sliceStart[r] = a.sliceStart[r];
    }
    return to;
  }
};

typedef uint32_t Words __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

__device__ __forceinline__ Words philox(Words c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t p = (uint64_t)0xD2511F53u * c[0], q = (uint64_t)0xCD9E8D57u * c[2];
    c = Words{xor3((uint32_t)(q >> 32), c[1], k0), (uint32_t)q, xor3((uint32_t)(p >> 32), c[3], k1), (uint32_t)p};
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

__device__ __forceinline__ Words wordsOf(const DropCall& a, uint64_t offset, uint32_t row, uint32_t group) {
  return philox(Words{group, row, (uint32_t)offset, (uint32_t)(offset >> 32)}, a.key0, a.key1) & a.mask;
}

// 8 elements of a row.
template <int DT, bool STREAM>
struct Eight {
  typedef typename Elem<DT>::type T;
  static constexpr int V = kVec<DT>, WORDS = 8 * sizeof(T) / 4;
  union {
    typename VecOf<T, V>::type v[8 / V];
    uint32_t words[WORDS];
  };
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) v[i] = STREAM ? loadStream<T, V>(p + i * V) : loadVec<T, V>(p + i * V);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      if (STREAM) storeStream<T, V>(p + i * V, v[i]);
      else storeVec<T, V>(p + i * V, v[i]);
    }
  }
  // The first n elements alone, where a row has fewer than 8.
  __device__ __forceinline__ void loadFew(const T* p, int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e / V][e % V] = e < n ? p[e] : (T)0.0f;
  }
  __device__ __forceinline__ void storeFew(T* p, int n) const {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) p[e] = v[e / V][e % V];
  }
  // Element e becomes what element e + k was (k < 8), 0 past the end.
  __device__ __forceinline__ void moveDown(int k) {
#pragma unroll
    for (int step = 4; step > 0; step /= 2) {
      if (!(k & step)) continue;
      const int by = step * (int)sizeof(T) / 4;   // words
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        const uint32_t low = i + by < WORDS ? words[i + by] : 0u;
        const uint32_t next = i + by + 1 < WORDS ? words[i + by + 1] : 0u;
        words[i] = step * sizeof(T) % 4 ? (next << 16 | low >> 16) : low;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) words[i] = 0;
  }
  __device__ __forceinline__ float operator[](int e) const { return (float)v[e / V][e % V]; }
  __device__ __forceinline__ void set(int e, float f) { v[e / V][e % V] = (T)f; }
};

// Where a thread works: its 8 columns and its rank's rows, every step-th from
// the first.  Threads past the columns have n <= 0.
struct DropPlace {
  int rank, column, n;
  int tile, slice, line, place;     // its line and place among the workgroup's rows
  int row, rows, step;
  uint32_t group;
};

template <int BLOCK, int RANKS>
__device__ __forceinline__ DropPlace placeOf(const DropArgs<RANKS>& a) {
  DropPlace p;
  // eight slices at a time, one an XCD (workgroups go to them in turn)
  const bool near = blockIdx.x < a.nearBlocks;
  const unsigned block = near ? blockIdx.x / 8 : blockIdx.x;
  p.slice = (int)__umulhi(block, a.overTiles);   // block / tiles, or 1 less
  p.tile = (int)block - p.slice * a.cut.tiles;
  if (p.tile >= a.cut.tiles) {
    ++p.slice;
    p.tile -= a.cut.tiles;
  }
  if (near) p.slice = p.slice * 8 + (int)(blockIdx.x % 8);
  const int item = (a.cut.flat ? p.tile * BLOCK : 0) + (int)threadIdx.x;
  p.line = (int)fmaf((float)item, a.overAcross, 0.5f * a.overAcross);   // item / across
  p.place = item - __mul24(p.line, a.cut.across);
  p.group = (uint32_t)((a.cut.flat ? 0 : p.tile * a.cut.across) + p.place);
  p.column = (int)p.group * kDropCols;
  p.rank = 0;
  while (p.slice >= a.sliceStart[p.rank + 1]) ++p.rank;
  p.n = p.line < a.cut.together ? a.cols - p.column : 0;
  const int first = a.sliceStart[p.rank];
  p.row = (p.slice - first) * a.cut.together + p.line;
  p.rows = a.rowStart[p.rank + 1] - a.rowStart[p.rank];
  p.step = (a.sliceStart[p.rank + 1] - first) * a.cut.together;
  return p;
}

// Calls f(load, settle, store), how a thread's elements of a row come and go.
// The 8 elements, or the fewer before a row's end, come with one load: at the
// end it moves back to end with the row, so that all threads' loads go out
// alike, and `settle` brings the elements to their places once they are there;
// what it reads of its neighbour's, who may be writing them in place, is not
// used.  2537 rows of 2047 fp16 backward 15.5 us with the last elements loaded
// one by one, 12.2 so.  Rows of less than 8 elements are loaded one by one.
template <typename E, typename F>
__device__ __forceinline__ void withAccess(const DropPlace& at, int cols, F f) {
  typedef typename E::T T;
  const bool tail = at.n < kDropCols;
  const auto store = [&](T* row, const E& v) {
    if (tail) v.storeFew(row, at.n);
    else v.store(row);
  };
  if (cols < kDropCols) {
    f([&](E* v, const T* row) { v->loadFew(row, at.n); }, [](E*) {}, store);
    return;
  }
  const int back = tail ? kDropCols - at.n : 0;
  f([&](E* v, const T* row) { v->load(row - back); },
    [&](E* v) {
      if (tail) v->moveDown(back);
    },
    store);
}

template <int DT, int WT, bool STREAM, bool RESIDUAL, int RANKS>
__device__ __forceinline__ void forwardRows(const DropArgs<RANKS>& a, const DropPlace& at) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  typedef Eight<DT, STREAM> E;
  const uint64_t offset = a.offset + (a.step ? *a.step : 0);
  const uint32_t first = a.firstRow[at.rank];
  const T* x = (const T*)a.x[at.rank] + at.column;
  const T* residual = RESIDUAL ? (const T*)a.residual[at.rank] + at.column : nullptr;
  T* y = (T*)a.y[at.rank] + at.column;
  Eight<WT, false> bias;
  bias.clear();
  if (a.bias[at.rank]) {
    const W* from = (const W*)a.bias[at.rank] + at.column;
    if (at.n >= kDropCols) bias.load(from);
    else bias.loadFew(from, at.n);
  }
  withAccess<E>(at, a.cols, [&](auto load, auto settle, auto store) {
    for (int64_t i = at.row; i < at.rows; i += at.step) {
      E v, z, out;
      load(&v, x + i * a.xStride);
      if (RESIDUAL) load(&z, residual + i * a.residualStride);
      const Words w = wordsOf(a, offset, first + (uint32_t)i, at.group);
      settle(&v);
      if (RESIDUAL) settle(&z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float r = RESIDUAL ? z[e] : 0.0f;
        out.set(e, kept(w, e, a.threshold) ? fmaf(v[e] + bias[e], a.scale, r) : r);
      }
      store(y + i * a.yStride, out);
    }
  });
}

template <int DT, int WT, int RANKS, bool STREAM>
__global__ void __launch_bounds__(kDropBlock) dropoutAdd(const DropArgs<RANKS> a) {
  const DropPlace at = placeOf<kDropBlock>(a);
  if (at.n <= 0) return;
  if (a.residual[at.rank]) forwardRows<DT, WT, STREAM, true>(a, at);
  else forwardRows<DT, WT, STREAM, false>(a, at);
}

template <int DT, int RANKS, bool SUMS, bool STREAM>
__global__ void __launch_bounds__(kDropBackBlock) dropoutAddBackward(const DropArgs<RANKS> a) {
  typedef typename Elem<DT>::type T;
  typedef Eight<DT, STREAM> E;
  __shared__ float lds[SUMS ? kDropBackBlock * kDropCols : 1];
  const DropPlace at = placeOf<kDropBackBlock>(a);
  FloatVec<8> sum = (FloatVec<8>)0.0f;
  if (at.n > 0) {
    const uint64_t offset = a.offset + (a.step ? *a.step : 0);
    const uint32_t first = a.firstRow[at.rank];
    const T* dy = (const T*)a.x[at.rank] + at.column;
    T* dx = a.y[at.rank] ? (T*)a.y[at.rank] + at.column : nullptr;
    withAccess<E>(at, a.cols, [&](auto load, auto settle, auto store) {
      for (int64_t i = at.row; i < at.rows; i += at.step) {
        E v, out;
        load(&v, dy + i * a.xStride);
        const Words w = wordsOf(a, offset, first + (uint32_t)i, at.group);
        settle(&v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = kept(w, e, a.threshold) ? v[e] : 0.0f;
          if (SUMS) sum[e] += d;
          out.set(e, d * a.scale);
        }
        if (dx) store(dx + i * a.yStride, out);
      }
    });
  }
  if constexpr (SUMS) {
    // a column's lines are shared out among the threads that there are to it
    const int columns = a.cut.across * kDropCols;
    int lines = a.cut.together;
    if (at.line < lines)
#pragma unroll
      for (int e = 0; e < 8; ++e) lds[at.line * columns + at.place * kDropCols + e] = sum[e];
    __syncthreads();
    const int parts = kDropBackBlock / columns;
    if (parts > 1) {
      const int part = (int)threadIdx.x / columns;
      float all = 0.0f;
      if (part < parts)
        for (int k = part; k < lines; k += parts) all += lds[k * columns + (int)threadIdx.x % columns];
      __syncthreads();
      if (part < parts) lds[threadIdx.x] = all;
      __syncthreads();
      lines = lines < parts ? lines : parts;
    }
    for (int c = threadIdx.x; c < columns; c += kDropBackBlock) {
      const int64_t column = (int64_t)at.tile * columns + c;
      if (column >= a.cols) continue;
      float all = 0.0f;
      int k = 0;
      for (; k + 8 <= lines; k += 8) all += joinSlices<8>([&](int w) { return lds[(k + w) * columns + c]; });
      for (; k < lines; ++k) all += lds[k * columns + c];
      a.partial[(size_t)at.slice * a.partialCols + column] = all;
    }
  }
}

// Few rows in one launch: a workgroup takes 64 columns of all of them, 64 rows
// at a time, and writes their sums to every rank itself.  8192 columns: one row
// 3.9 us, 5.9 in two launches; 64 rows of 8 ranks 5.7, 6.7; 256 7.3, 8.3; 512 9.8,
// 9.0, where what it takes to draw the rows one after another bounds it (two or
// four rows' loads ahead gained nothing).
constexpr int kFewAcross = 8, kFewRows = 256;

template <int RANKS>
struct DropFewArgs {
  DropArgs<RANKS> rows;
  void* dbias[RANKS];
};

template <int DT, int WT, int RANKS>
__global__ void __launch_bounds__(kDropBackBlock) dropoutAddBackwardFew(const DropFewArgs<RANKS> w) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<WT>::type W;
  typedef Eight<DT, false> E;
  constexpr int WAVES = kDropBackBlock / kWave, COLS = kFewAcross * kDropCols;
  __shared__ float lds[WAVES][COLS];
  struct RowAt {
    const T* dy;
    T* dx;
    uint32_t index;
  };
  __shared__ RowAt rows[kFewRows];
  const DropArgs<RANKS>& a = w.rows;
  for (int r = 0; r < a.nranks; ++r) {
    const int from = a.rowStart[r], n = a.rowStart[r + 1] - from;
    for (int i = threadIdx.x; i < n; i += kDropBackBlock)
      rows[from + i] = RowAt{(const T*)a.x[r] + i * a.xStride, a.y[r] ? (T*)a.y[r] + i * a.yStride : nullptr,
                             a.firstRow[r] + (uint32_t)i};
  }
  __syncthreads();
  const uint64_t offset = a.offset + (a.step ? *a.step : 0);
  const int total = a.rowStart[a.nranks];
  for (int64_t tile = blockIdx.x; tile * COLS < a.cols; tile += gridDim.x) {
    DropPlace at;
    at.rank = 0;
    at.group = (uint32_t)(tile * kFewAcross) + threadIdx.x % kFewAcross;
    at.column = (int)at.group * kDropCols;
    at.n = a.cols - at.column;
    at.row = (int)threadIdx.x / kFewAcross;
    at.rows = at.n > 0 ? total : 0;
    at.step = kDropBackBlock / kFewAcross;
    FloatVec<8> sum = (FloatVec<8>)0.0f;
    withAccess<E>(at, a.cols, [&](auto load, auto settle, auto store) {
      for (int i = at.row; i < at.rows; i += at.step) {
        const RowAt row = rows[i];
        E v, out;
        load(&v, row.dy + at.column);
        const Words words = wordsOf(a, offset, row.index, at.group);
        settle(&v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = kept(words, e, a.threshold) ? v[e] : 0.0f;
          sum[e] += d;
          out.set(e, d * a.scale);
        }
        if (row.dx) store(row.dx + at.column, out);
      }
    });
#pragma unroll
    for (int m = kFewAcross; m < kWave; m *= 2)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], m);
    const int wave = (int)threadIdx.x / kWave, lane = (int)threadIdx.x % kWave;
    if (lane < kFewAcross)
#pragma unroll
      for (int e = 0; e < 8; ++e) lds[wave][lane * kDropCols + e] = sum[e];
    __syncthreads();
    const int64_t c = tile * COLS + threadIdx.x;
    if (threadIdx.x < COLS && c < a.cols) {
      const float all = joinSlices<WAVES>([&](int k) { return lds[k][threadIdx.x]; });
      for (int r = 0; r < a.nranks; ++r) ((W*)w.dbias[r])[c] = (W)(all * a.scale);
    }
    __syncthreads();   // before the next columns' sums
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
      const float all = joinSlices<kJoinSlices>([&](int k) { return lds[k][threadIdx.x]; });
      for (int r = 0; r < a.nranks; ++r) ((W*)a.dbias[r])[col] = (W)(all * a.scale);
    }
    __syncthreads();   // before the next columns' sums
  }
}

// The share of threads that have columns.
double dropUsed(const DropCut& k, int groups, int block) {
  return (double)groups * k.together / ((double)k.tiles * block);
}

// What costs most is lines of 128 bytes that two workgroups share, then threads
// without columns.  Rows of whole lines are cut at lines, 64 threads wide where
// that comes out even (8 x 4096 x 8192 bf16 backward 180 us, 187 with 32, 190-204
// with 128).  Others forward are not cut at all: the workgroups follow each other
// through so many rows that few threads are left over (8 x 32768 x 1032 269 us,
// 509 in tiles of 16 threads; 8 x 65536 x 520 268, 518; 8 x 6500 x 5000 247, 300
// in tiles of 64).  Backward, where a thread stays with its columns, they are one
// tile up to 256 threads (x 1032 245, 299 in two of 65 threads, 423 in nine of
// 16), else even ones of 64 to 256 (8 x 16384 x 2056 in four of 65 244, in five
// of 52 263).
DropCut dropCut(int cols, int block, bool sums) {
  const int groups = (cols + kDropCols - 1) / kDropCols;
  if (groups % 32 == 0) {
    const int across = groups % 64 == 0 ? 64 : 32;
    return {across, block / across, groups / across, false};
  }
  DropCut best{};
  double used = 0.0;
  const auto offer = [&](const DropCut& k, double more) {
    const double u = dropUsed(k, groups, block);
    if (u <= used + more) return;
    used = u;
    best = k;
  };
  if (!sums) {
    const int most = groups < block / 32 ? block / groups : 32;
    for (int rows = 1; rows <= most && used < 0.97; ++rows)
      offer({groups, rows, (int)(((int64_t)rows * groups + block - 1) / block), true}, 0.0);
    return best;
  }
  if (groups % 8 == 0 && groups > 64) {   // 8 x 20000 x 1600: five tiles of 40 185 us, seven of 32 189, one of 200 202
    for (int across = 64; across >= 24; across -= 8)
      offer({across, block / across, (groups + across - 1) / across, false}, 0.02);
    return best;
  }
  if (groups <= block / 2) return {groups, block / groups, 1, false};
  for (int together = 2; together <= block / 64; ++together) {
    const int tiles = (groups + block / together - 1) / (block / together), across = (groups + tiles - 1) / tiles;
    if (across >= kWave) offer({across, block / across, tiles, false}, 0.02);
  }
  return best;
}

// Cuts the rows of a launch's ranks into slices, and returns their number.
// Workgroups that come and go keep a closer window over memory than ones that
// last: forward 245 us with 256 workgroups a CU in all, 262 with 128, 280 with
// 32, 267-271 with 512 and more; backward 181 with 32 a CU, 187 with 16, 190
// with 8, 185 with 64.  Backward a slice costs a row of partial sums to write
// and read, so it has 32 rows at least (2537 rows of 2047 11.8 us; 16 rows 11.7,
// 64 13.2; of 2048 11.0, 11.3, 11.3), but 16 or 8 where a quarter of the CUs would
// have none (3000 x 924 fp16 11.5 us, 9.2 so; 8 ranks' 84-0 x 12119 16.6, 10.7), and
// there are at most two a CU (160000 rows of 100 21 us, 23 with four, 28 with
// eight, 44 with 20; of 512 66, 69, 68, 78).
// Where up to half of the CUs would have a workgroup more than the others, its
// rows are shared out among them all (312 workgroups 11.9 us, as 256 11.1; 580
// 14.3, as 512 13.1; but 453 13.4, as 256 14.1), with tiles few enough to come near.
int sliceRows(const size_t* rows, int ranks, const DropCut& k, bool sums, int* rowStart, int* sliceStart) {
  rowStart[0] = sliceStart[0] = 0;
  for (int r = 0; r < ranks; ++r) rowStart[r + 1] = rowStart[r] + (int)rows[r];
  int least = 32;   // rows of a slice with sums
  while (least > 8 && wholeGroups(rowStart, ranks, least) * k.tiles < 3 * kOpsCUs / 4) least /= 2;
  const int each = sums && k.together < least ? (least + k.together - 1) / k.together * k.together : k.together;
  int64_t most = (sums ? 32 : 256) * kOpsCUs / k.tiles;
  if (sums && most > 2 * kOpsCUs) most = 2 * kOpsCUs;
  if (most < 1) most = 1;
  const int64_t grid = (wholeGroups(rowStart, ranks, each) < most ? wholeGroups(rowStart, ranks, each) : most) * k.tiles;
  if (sums && k.tiles <= kOpsCUs / 8 && grid > kOpsCUs && grid % kOpsCUs <= kOpsCUs / 2)
    most = grid / kOpsCUs * kOpsCUs / k.tiles;
  return giveOut(rowStart, ranks, each, k.together, (int)most, sliceStart);
}

// Calls that move more than the caches hold load and store past them: 8 x 4096
// x 8192 forward 245 us, 270 through them; backward 182 and 194; 402 MB forward
// 72 and 74.  Below that the next to read is better off: 201 MB 35.9 and 34.8,
// 134 MB backward 33.1 and 30.5.
constexpr size_t kDropStream = (size_t)256 << 20;

template <int DT, int WT>
struct DropForward {
  template <int RANKS>
  static hipError_t launch(const DropArgs<RANKS>& a, dim3 grid, hipStream_t st) {
    return launchKernel(a.stream ? dropoutAdd<DT, WT, RANKS, true> : dropoutAdd<DT, WT, RANKS, false>, grid,
                        dim3(kDropBlock), a, st);
  }
  static hipError_t run(const DropArgs<kDropRanks>& a, dim3 grid, hipStream_t st) {
    return a.nranks > kOpRanks ? launch(a, grid, st) : launch(DropArgs<kOpRanks>::of(a), grid, st);
  }
};

template <int DT>
struct DropBackward {
  template <int RANKS>
  static hipError_t launch(const DropArgs<RANKS>& a, dim3 grid, hipStream_t st) {
    const auto sums = a.stream ? dropoutAddBackward<DT, RANKS, true, true> : dropoutAddBackward<DT, RANKS, true, false>;
    const auto none = a.stream ? dropoutAddBackward<DT, RANKS, false, true> : dropoutAddBackward<DT, RANKS, false, false>;
    return launchKernel(a.partial ? sums : none, grid, dim3(kDropBackBlock), a, st);
  }
  static hipError_t run(const DropArgs<kDropRanks>& a, dim3 grid, hipStream_t st) {
    return a.nranks > kOpRanks ? launch(a, grid, st) : launch(DropArgs<kOpRanks>::of(a), grid, st);
  }
};

template <int DT, int WT>
struct DropBackwardFew {
  template <int RANKS>
  static hipError_t launch(const DropArgs<RANKS>& a, void* const* dbias, hipStream_t st) {
    constexpr int COLS = kFewAcross * kDropCols;
    DropFewArgs<RANKS> w;
    w.rows = a;
    for (int r = 0; r < RANKS; ++r) w.dbias[r] = r < a.nranks ? dbias[r] : nullptr;
    return launchKernel(dropoutAddBackwardFew<DT, WT, RANKS>,
                        dim3(gridOf(((int64_t)a.cols + COLS - 1) / COLS, kDropBackBlock)), dim3(kDropBackBlock), w, st);
  }
  static hipError_t run(const DropArgs<kDropRanks>& a, void* const* dbias, hipStream_t st) {
    return a.nranks > kOpRanks ? launch(a, dbias, st) : launch(DropArgs<kOpRanks>::of(a), dbias, st);
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

void fillDraw(DropCall* a, double p, uint64_t seed, uint64_t offset, const uint64_t* step) {
  const int t = (int)std::floor(p * 65536.0 + 0.5);
  a->threshold = (uint32_t)(t >= 65536 ? 1 : t) << 16;
  a->mask = t >= 65536 ? 0u : ~0u;
  a->scale = t >= 65536 ? 0.0f : (float)(65536.0 / (65536 - t));
  a->key0 = (uint32_t)seed;
  a->key1 = (uint32_t)(seed >> 32);
  a->offset = offset;
  a->step = step;
}

// Ranks of a launch: its workgroups, one at least to a tile of each rank's
// columns, have fewer than 2^32 threads.
int dropRanks(size_t cols) { return cols <= (size_t)1 << 26 ? kDropRanks : 1; }

// This launch's rows and their slices; returns the grid's slices.
int fillDropRows(DropArgs<kDropRanks>* a, const size_t* rows, const uint64_t* firstRow, int nranks, int first,
                 size_t cols, bool sums) {
  const int most = dropRanks(cols);
  a->nranks = nranks - first < most ? nranks - first : most;
  uint64_t next = 0;
  for (int r = 0; r < first; ++r) next += rows[r];
  for (int r = 0; r < a->nranks; ++r) {
    a->firstRow[r] = (uint32_t)(firstRow ? firstRow[first + r] : next);
    next += rows[first + r];
  }
  a->cols = (int)cols;
  a->partialCols = (int)((cols + 7) / 8 * 8);
  a->cut = dropCut((int)cols, sums ? kDropBackBlock : kDropBlock, sums);
  a->overAcross = a->cut.together > 1 ? 1.0f / (float)a->cut.across : 0.0f;
  return sliceRows(rows + first, a->nranks, a->cut, sums, a->rowStart, a->sliceStart);
}

// The grid.  Tiles whose ends are not those of 128-byte lines share lines with
// their neighbours, and go to the same XCD with them, whose cache puts the lines
// together (8 x 4096 x 8191 bf16 forward 273 us, 335 without; backward 219, 264;
// of whole lines, 8192, 247, 247 and 184, 181).
dim3 dropGrid(DropArgs<kDropRanks>* a, int slices, int esz) {
  const unsigned tiles = (unsigned)a->cut.tiles, grid = (unsigned)slices * tiles;
  uintptr_t bits = (uintptr_t)(a->xStride | a->yStride | a->residualStride | a->cut.across * kDropCols) * (uintptr_t)esz;
  for (int r = 0; r < a->nranks; ++r) bits |= (uintptr_t)a->x[r] | (uintptr_t)a->y[r] | (uintptr_t)a->residual[r];
  const bool near = !a->cut.flat && tiles > 1 && bits % 128 != 0;
  a->nearBlocks = near ? grid / (8 * tiles) * (8 * tiles) : 0;
  a->overTiles = tiles == 1 ? ~0u : (uint32_t)(((uint64_t)1 << 32) / tiles);
  return dim3(grid);
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
  DropArgs<kDropRanks> a{};
  fillDraw(&a, p, seed, offset, step);
  const size_t bytes = (size_t)s.total * cols * (size_t)esz * (residual ? 3 : 2);
  for (int first = 0; first < nranks; first += dropRanks(cols)) {
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
    a.stream = bytes > kDropStream;
    const dim3 grid = dropGrid(&a, slices, esz);
    if (byTypes<DropForward, const DropArgs<kDropRanks>&, dim3, hipStream_t>(dtype, wtype, a, grid, st) != hipSuccess)
      return arHipError;
  }
  return arSuccess;
}

arResult_t dropWorkspace(const size_t* rows, int nranks, size_t cols, size_t* bytes) {
  Shape s;
  if (bytes == nullptr || !shapeOk(rows, nranks, cols, &s)) return arInvalidArgument;
  const DropCut k = dropCut((int)cols, kDropBackBlock, true);
  size_t slices = 0;
  const int ranks = dropRanks(cols);
  int rowStart[kDropRanks + 1], sliceStart[kDropRanks + 1];
  for (int first = 0; first < nranks; first += ranks)
    slices += (size_t)sliceRows(rows + first, nranks - first < ranks ? nranks - first : ranks, k, true, rowStart, sliceStart);
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
  DropArgs<kDropRanks> a{};
  fillDraw(&a, p, seed, offset, step);
  int partials = 0;
  const size_t bytes = (size_t)s.total * cols * (size_t)esz * (dx ? 2 : 1);
  for (int first = 0; first < nranks; first += dropRanks(cols)) {
    const int slices = fillDropRows(&a, rows, firstRow, nranks, first, cols, true);
    if (slices == 0) continue;
    for (int r = 0; r < a.nranks; ++r) {
      const bool any = rows[first + r] > 0;
      a.x[r] = any ? dy[first + r] : nullptr;
      a.y[r] = any && dx ? dx[first + r] : nullptr;
    }
    a.xStride = (int64_t)dyStride;
    a.yStride = (int64_t)dxStride;
    a.stream = bytes > kDropStream;
    if (dbias != nullptr && nranks <= dropRanks(cols) && s.total <= kFewRows) {
      const hipError_t e = byTypes<DropBackwardFew, const DropArgs<kDropRanks>&, void* const*, hipStream_t>(
          dtype, wtype, a, dbias, st);
      return e == hipSuccess ? arSuccess : arHipError;
    }
    if (dbias != nullptr) a.partial = (float*)workspace + (size_t)partials * a.partialCols;
    const dim3 grid = dropGrid(&a, slices, esz);
    if (byType<DropBackward, const DropArgs<kDropRanks>&, dim3, hipStream_t>(dtype, a, grid, st) != hipSuccess)
      return arHipError;
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
