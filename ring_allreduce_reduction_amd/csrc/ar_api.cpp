// ar_api.cpp -- the overlap check shared by the C entry points.
#include "ar_api.h"

#include <algorithm>

namespace ar {
namespace {

uintptr_t endOf(const Extent& e) { return e.begin + (e.rows - 1) * e.stride + e.width; }

bool sameMemory(const Extent& a, const Extent& b) {
  return a.begin == b.begin && a.width == b.width && a.rows == b.rows && (a.rows == 1 || a.stride == b.stride);
}

bool touches(const Extent& a, const Extent& b) {
  if (a.begin >= endOf(b) || b.begin >= endOf(a)) return false;
  // Same stride: row starts differ by d modulo the stride, so the rows stay
  // apart when each fits the gap the other leaves.
  const size_t s = a.rows > 1 ? a.stride : b.stride;
  const bool sameStride = (a.rows == 1 || a.stride == s) && (b.rows == 1 || b.stride == s);
  if (sameStride && (a.rows > 1 || b.rows > 1) && a.width <= s && b.width <= s) {
    const size_t d = b.begin >= a.begin ? (b.begin - a.begin) % s : (s - (a.begin - b.begin) % s) % s;
    if (d >= a.width && d + b.width <= s) return false;
  }
  return true;
}

}  // namespace

bool outputsOverlap(std::vector<Extent>& v) {
  std::sort(v.begin(), v.end(), [](const Extent& a, const Extent& b) { return a.begin < b.begin; });
  // Only pairs with an output are looked at: any number of inputs may share
  // memory (one tensor listed 2^20 times), and dense buffers then end the search
  // at their first pair that is not in place.
  std::vector<size_t> nextOutput(v.size() + 1, v.size());   // the first output from here on
  for (size_t i = v.size(); i-- > 0;) nextOutput[i] = v[i].output ? i : nextOutput[i + 1];
  for (size_t i = 0; i < v.size(); ++i) {
    const uintptr_t end = endOf(v[i]);
    for (size_t j = i + 1; j < v.size(); ++j) {
      if (!v[i].output) j = nextOutput[j];
      if (j == v.size() || v[j].begin >= end) break;
      if (v[i].pair >= 0 && v[i].pair == v[j].pair && sameMemory(v[i], v[j])) continue;
      if (touches(v[i], v[j])) return true;
    }
  }
  return false;
}

}  // namespace ar
