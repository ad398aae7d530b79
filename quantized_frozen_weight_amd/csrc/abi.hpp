// What the entry points of the C ABI share on the host: argument checks,
// workspace arithmetic, and the status of their launches.
#pragma once
#include <hip/hip_runtime.h>

#include "qlora.h"

namespace qlora {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

inline bool fits_int(long long a, long long b) {
  return a > 0 && b > 0 && a * b < (1LL << 31);
}

inline int check_dtype(int dtype) {
  return (dtype == QLORA_F32 || dtype == QLORA_BF16) ? QLORA_OK : QLORA_EINVAL;
}

inline char* at(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

// Before a call enqueues anything: a HIP error that earlier work of the
// caller left pending is not ours to clear, and launching on top of it would
// blame it on this call. The call returns QLORA_EHIP, enqueues nothing and
// leaves the error in place for the caller.
inline int pending_error() {
  return hipPeekAtLastError() == hipSuccess ? QLORA_OK : QLORA_EHIP;
}

// After a call's launches: nothing was pending before them (pending_error),
// so an error now is one of this call's launches; it is reported and
// cleared.
inline int launch_status() {
  hipError_t e = hipGetLastError();
  return e == hipSuccess ? QLORA_OK : QLORA_EHIP;
}

inline size_t dtype_bytes(int dtype) { return dtype == QLORA_F32 ? 4 : 2; }

// A pointer that may be NULL and must be aligned where it is not.
inline bool opt16(const void* p) { return p == nullptr || aligned16(p); }

// Byte ranges of a call's arguments; NULL ranges are left out.
struct Ranges {
  struct { const char* p; size_t n; } r[24];
  int count = 0;
  void add(const void* p, size_t n) {
    if (p != nullptr && n > 0) { r[count].p = static_cast<const char*>(p); r[count].n = n; ++count; }
  }
  bool hits(const void* p, size_t n) const {
    const char* q = static_cast<const char*>(p);
    for (int i = 0; i < count; ++i)
      if (q < r[i].p + r[i].n && r[i].p < q + n) return true;
    return false;
  }
};

// Outputs against inputs and against each other.
inline bool disjoint(const Ranges& outs, const Ranges& ins) {
  Ranges seen = ins;
  for (int i = 0; i < outs.count; ++i) {
    if (seen.hits(outs.r[i].p, outs.r[i].n)) return false;
    seen.add(outs.r[i].p, outs.r[i].n);
  }
  return true;
}

}  // namespace qlora
