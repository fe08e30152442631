// The operators' overlap check (ar_api.cpp) against a byte-by-byte answer, on
// random buffers of a small address range, under the sanitizers.
#include <stdint.h>
#include <stdio.h>

#include <random>
#include <vector>

#include "ar_api.h"

static bool same(const ar::Extent& a, const ar::Extent& b) {
  return a.pair >= 0 && a.pair == b.pair && a.begin == b.begin && a.width == b.width && a.rows == b.rows &&
         (a.rows == 1 || a.stride == b.stride);
}

static bool touch(const ar::Extent& a, const ar::Extent& b) {
  std::vector<char> used(4096, 0);
  for (size_t i = 0; i < a.rows; ++i)
    for (size_t k = 0; k < a.width; ++k) used[a.begin + i * a.stride + k] = 1;
  for (size_t i = 0; i < b.rows; ++i)
    for (size_t k = 0; k < b.width; ++k)
      if (used[b.begin + i * b.stride + k]) return true;
  return false;
}

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int missed = 0, over = 0, refused = 0, allowed = 0;
  for (int round = 0; round < 200000; ++round) {
    std::vector<ar::Extent> v;
    const size_t shared = (size_t)pick(4, 24);
    const int n = pick(2, 5);
    for (int i = 0; i < n; ++i) {
      ar::Extent e;
      e.width = (size_t)pick(1, 10);
      e.rows = (size_t)pick(1, 6);
      e.stride = pick(0, 2) ? shared : (size_t)pick(1, 24);
      if (e.stride < e.width) e.stride = e.width;
      e.begin = (uintptr_t)pick(1, 220);
      e.output = pick(0, 1) != 0;
      e.pair = pick(-1, 1);
      if (i > 0 && pick(0, 3) == 0) {   // a likely in-place pair
        e = v.back();
        e.output = !e.output;
      }
      v.push_back(e);
    }
    bool want = false, interleaved = false;
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j) {
        if ((!v[(size_t)i].output && !v[(size_t)j].output) || same(v[(size_t)i], v[(size_t)j])) continue;
        want = want || touch(v[(size_t)i], v[(size_t)j]);
        interleaved = interleaved || v[(size_t)i].stride != v[(size_t)j].stride;
      }
    const bool got = ar::outputsOverlap(v);
    if (want && !got) ++missed;                  // never
    if (!want && got && !interleaved) ++over;    // only rows of different strides may be refused without a shared byte
    refused += got;
    allowed += !got;
  }
  printf("missed %d, refused needlessly %d (of %d refused, %d allowed)\n", missed, over, refused, allowed);
  return missed || over || refused < 1000 || allowed < 1000;
}
