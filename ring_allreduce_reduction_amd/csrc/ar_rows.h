// ar_rows.h -- the host side that operators over the ranks' rows share: their
// limits, argument checks, and the choice of a kernel by element types.
#pragma once

#include <vector>

#include "ar_api.h"
#include "ar_internal.h"
#include "ar_ops.h"

namespace ar {

// Ranks per launch: their pointers travel in the kernel arguments, which every
// launch copies (1 KB; with 32 ranks' a one-row call took 0.4-1 us longer).
constexpr int kOpRanks = 16;
constexpr size_t kRowsMaxCols = (size_t)1 << 30;
constexpr int64_t kRowsMax = 0x7fffffff;   // of all ranks

// A launch holds fewer than 2^32 threads along its grid: `blocks` workgroups
// of `block` threads, as many as fit into half of that.  Kernels launched with
// it step through what is left over.
inline unsigned gridOf(int64_t blocks, int block) {
  const int64_t most = ((int64_t)1 << 31) / block;
  return (unsigned)(blocks < most ? blocks : most);
}

struct Shape {
  int64_t total = 0;
  int launches = 0;
};

// Row counts every entry checks alike.
inline bool rowsOk(const size_t* rows, int nranks, Shape* s) {
  if (rows == nullptr || nranks < 1 || nranks > AR_MAX_RANKS) return false;
  s->total = 0;
  for (int r = 0; r < nranks; ++r) {
    if (rows[r] > (size_t)kRowsMax) return false;
    s->total += (int64_t)rows[r];
  }
  if (s->total > kRowsMax) return false;
  s->launches = (nranks + kOpRanks - 1) / kOpRanks;
  return true;
}

// Row counts and widths.
inline bool shapeOk(const size_t* rows, int nranks, size_t cols, Shape* s) {
  return cols >= 1 && cols <= kRowsMaxCols && rowsOk(rows, nranks, s);
}

inline bool strideOk(size_t stride, size_t cols) { return stride >= cols && stride <= (size_t)1 << 48; }

inline bool aligned(const void* p, int esz) { return p != nullptr && (uintptr_t)p % (uintptr_t)esz == 0; }

inline int64_t rowsOfLaunch(const size_t* rows, int nranks, int first) {
  int64_t n = 0;
  for (int r = first; r < nranks && r < first + kOpRanks; ++r) n += (int64_t)rows[r];
  return n;
}

// Adds a rank's row buffer to the overlap check; false for a bad pointer.
inline bool addRows(std::vector<Extent>& v, const void* p, size_t rows, size_t cols, size_t stride, int esz,
                    bool output, int pair) {
  if (rows == 0) return true;
  if (!aligned(p, esz) || rows > ((size_t)1 << 48) / stride) return false;
  v.push_back(Extent{(uintptr_t)p, cols * (size_t)esz, rows, stride * (size_t)esz, output, pair});
  return true;
}

inline bool addFlat(std::vector<Extent>& v, const void* p, size_t count, int esz, bool output) {
  return addRows(v, p, count ? 1 : 0, count, count, esz, output, -1);
}

// Shares `most` workgroups of `groups` rows at a time out among the ranks by
// their rows, at least one to a rank with rows (so more than `most` only where
// there are more such ranks): rank r takes [blockStart[r], blockStart[r + 1]).
// Returns the grid.
inline int shareOut(const int* rowStart, int nranks, int groups, int most, int* blockStart) {
  const int64_t rows = rowStart[nranks];
  int ranks = 0;
  for (int r = 0; r < nranks; ++r) ranks += rowStart[r + 1] > rowStart[r];
  const double share = most > ranks ? (double)(most - ranks) / (double)rows : 0.0;
  blockStart[0] = 0;
  for (int r = 0; r < nranks; ++r) {
    const int64_t n = rowStart[r + 1] - rowStart[r];
    const int64_t full = (n + groups - 1) / groups;
    const int64_t mine = n == 0 ? 0 : (int64_t)((double)n * share) + 1;
    blockStart[r + 1] = blockStart[r] + (int)(mine < full ? mine : full);
  }
  return blockStart[nranks];
}

// Groups of `groups` rows that all ranks' rows make, none of two ranks'.
inline int64_t wholeGroups(const int* rowStart, int nranks, int groups) {
  int64_t n = 0;
  for (int r = 0; r < nranks; ++r) n += ((int64_t)rowStart[r + 1] - rowStart[r] + groups - 1) / groups;
  return n;
}

// As shareOut, but where `most` are enough each rank has a workgroup for every
// `each` of its rows.
inline int giveOut(const int* rowStart, int nranks, int each, int groups, int most, int* blockStart) {
  if (wholeGroups(rowStart, nranks, each) > most) return shareOut(rowStart, nranks, groups, most, blockStart);
  blockStart[0] = 0;
  for (int r = 0; r < nranks; ++r)
    blockStart[r + 1] = blockStart[r] + (int)(((int64_t)rowStart[r + 1] - rowStart[r] + each - 1) / each);
  return blockStart[nranks];
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

template <template <int> class F, typename... A>
hipError_t byType(int dtype, A... args) {
  if (dtype == arFloat32) return F<arFloat32>::run(args...);
  if (dtype == arFloat16) return F<arFloat16>::run(args...);
  return F<arBfloat16>::run(args...);
}

}  // namespace ar
