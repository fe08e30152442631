// ar_api.h -- what every C entry point of libar.so shares on the host side:
// its ROCTx range, the state of this thread's open group, and the check that
// a call's outputs overlap nothing they must not.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <vector>

#include <rocprofiler-sdk-roctx/roctx.h>

#include "ar.h"

// A ROCTx range around an API call, as the pages mark each API entry with an
// NVTX range ["NCCL 原始碼解讀：一個 AllReduce 的 GPU 旅程", ch.3 §3.1, ch.6, the
// ncclAllReduce call chain]: rocprofv3 --marker-trace records one per call
// (host time of the call: argument checks, planning and the enqueue).
struct ApiRange {
  explicit ApiRange(const char* name) { roctxRangePushA(name); }
  ~ApiRange() { roctxRangePop(); }
  ApiRange(const ApiRange&) = delete;
  ApiRange& operator=(const ApiRange&) = delete;
};

namespace ar {

// Whether this host thread is between arGroupStart and its arGroupEnd.
bool groupOpen();
// Keeps the first error of the open group (arGroupEnd reports it); returns r.
arResult_t noteGroupError(arResult_t r);

// One buffer of a call: `rows` rows of `width` bytes, `stride` bytes apart
// (dense memory is one row).  `pair` names the buffer an output may share
// its memory with exactly (same start, width, rows and stride): buffers with
// the same non-negative pair value.
struct Extent {
  uintptr_t begin;
  size_t width, rows, stride;
  bool output;
  int pair;
};

// True if an output overlaps another buffer it is not exactly in place with.
// Rows that interleave without touching (column slices of one wider buffer,
// the same stride) do not overlap.  Sorts `v`.
bool outputsOverlap(std::vector<Extent>& v);

}  // namespace ar
