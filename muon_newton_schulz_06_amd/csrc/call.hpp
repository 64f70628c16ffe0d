// What the layer entry points share on the host: argument checks, launch
// status, exceptions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdlib>
#include <string>
#include <vector>

#include "../../include/muon_layers.h"
#include "launch.hpp"

namespace muon {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxLd = int64_t(1) << 32;

// Collects a call's argument errors and address ranges; the first error is
// kept.  Everything here runs before any HIP call.
struct Args {
  struct Range {
    uintptr_t lo, hi;
    const char* name;
    int64_t ld;
    bool written;
  };
  muon_status_t status = MUON_OK;
  std::string msg;
  std::vector<Range> ranges;

  bool ok() const { return status == MUON_OK; }
  void fail(muon_status_t s, const std::string& m) {
    if (ok()) {
      status = s;
      msg = m;
    }
  }
  void size(const char* name, int64_t v, int64_t lo, int64_t hi) {
    if (v < lo) fail(MUON_ERR_INVALID_ARG, std::string(name) + " below " + std::to_string(lo));
    else if (v > hi) fail(MUON_ERR_UNSUPPORTED, std::string(name) + " above " + std::to_string(hi));
  }
  void dtype(const char* name, int32_t d) {
    if (d != MUON_DTYPE_F32 && d != MUON_DTYPE_BF16)
      fail(MUON_ERR_INVALID_ARG, std::string("unknown ") + name);
  }
  // rows × cols of esz-byte elements; a matrix without rows may be NULL
  void matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t esz,
              bool written) {
    if (!ok() || rows == 0) return;
    if (!p) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if ((uintptr_t)p % esz) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is not aligned to its type");
    if (ld < cols) return fail(MUON_ERR_INVALID_ARG, std::string(name) + ": row stride below the row length");
    if (ld > kMaxLd) return fail(MUON_ERR_UNSUPPORTED, std::string(name) + ": row stride above 2^32");
    const uintptr_t lo = (uintptr_t)p;
    ranges.push_back({lo, lo + (uintptr_t)(((rows - 1) * ld + cols) * (int64_t)esz), name, ld, written});
  }
  void buffer(const char* name, const void* p, size_t have, size_t need, bool written) {
    if (!ok() || need == 0) return;
    if (!p) return fail(MUON_ERR_WORKSPACE, std::string(name) + " is NULL");
    if ((uintptr_t)p & 255) return fail(MUON_ERR_WORKSPACE, std::string(name) + " not 256-byte aligned");
    if (have < need)
      return fail(MUON_ERR_WORKSPACE, std::string(name) + " too small: need " + std::to_string(need) +
                                          " bytes, got " + std::to_string(have));
    const uintptr_t lo = (uintptr_t)p;
    ranges.push_back({lo, lo + need, name, 0, written});
  }
  // Written ranges overlap nothing, but for the pairs `same` allows (an
  // output that is the same matrix as an input).
  template <typename F>
  void aliases(F&& same) {
    for (size_t i = 0; ok() && i < ranges.size(); ++i)
      for (size_t j = 0; ok() && j < ranges.size(); ++j) {
        const Range &a = ranges[i], &b = ranges[j];
        if (i == j || !a.written || !(a.lo < b.hi && b.lo < a.hi)) continue;
        if (!b.written && a.lo == b.lo && a.hi == b.hi && a.ld == b.ld && same(a.name, b.name)) continue;
        fail(MUON_ERR_ALIAS, std::string(a.name) + " overlaps " + b.name);
      }
  }
  void aliases() {
    aliases([](const char*, const char*) { return false; });
  }
  muon_status_t report() const {
    if (!ok()) set_last_error(msg);
    return status;
  }
};

inline muon_status_t check_device() {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) {
    set_last_error("no HIP device visible");
    return MUON_ERR_NO_DEVICE;
  }
  return MUON_OK;
}

// Status of a launch; with MUON_DEBUG_SYNC=1 (and no capture) it waits for
// the stream, so that a failing kernel is named.
inline muon_status_t launched(const char* what, hipError_t e, hipStream_t st) {
  if (e == hipSuccess) {
    const char* dbg = std::getenv("MUON_DEBUG_SYNC");
    if (dbg && dbg[0] == '1') {
      hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
      if (hipStreamIsCapturing(st, &cs) == hipSuccess && cs == hipStreamCaptureStatusNone) {
        e = hipStreamSynchronize(st);
        if (e == hipSuccess) e = hipGetLastError();
      }
    }
  }
  if (e == hipSuccess) return MUON_OK;
  set_last_error(std::string(what) + ": " + hipGetErrorString(e));
  return MUON_ERR_HIP;
}

// No exception leaves an entry point.
template <typename F>
muon_status_t guarded(F&& f) {
  try {
    set_last_error("");
    return f();
  } catch (const std::exception& e) {
    try {
      set_last_error(e.what());
    } catch (...) {
    }
    return MUON_ERR_INVALID_ARG;
  } catch (...) {
    return MUON_ERR_INVALID_ARG;
  }
}

inline size_t esize(int32_t dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

// Rows of whole 16-byte chunks at 16-byte aligned addresses.
inline bool whole_chunks(const void* p, int64_t ld, int64_t cols, size_t esz) {
  const int64_t v = 16 / (int64_t)esz;
  return ((uintptr_t)p & 15) == 0 && ld % v == 0 && cols % v == 0;
}

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace muon
