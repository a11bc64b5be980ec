// host_checks.h -- what the host sides of libecho's calls share: the launch
// helper and the checks of addresses and byte ranges.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo.h"
#include "launch_shape.h"

namespace echo {

// Launch `kernel` with its one by-value argument struct.  The status is the
// launch's own (hipLaunchKernel's return value), so an error an earlier,
// unrelated HIP call left in the thread's last-error slot is neither
// reported as this call's nor cleared.
template <typename A>
inline int launch(void (*kernel)(A), dim3 grid, dim3 block, hipStream_t s, A arg) {
  void* argv[] = {&arg};
  const hipError_t e =
      hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, argv, 0, s);
  return e == hipSuccess ? ECHO_SUCCESS : ECHO_ERR_HIP;
}

template <typename A>
inline int launch(void (*kernel)(A), dim3 grid, hipStream_t s, A arg) {
  return launch(kernel, grid, dim3(kBlock), s, arg);
}

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A check that passed with nothing to do: zero elements.  The entry point
// then returns ECHO_SUCCESS without looking at its pointers or launching.
constexpr int kEmpty = 1;

// the status an entry point returns for a check result that is not SUCCESS
inline int finished(int rc) { return rc < 0 ? rc : ECHO_SUCCESS; }

// Byte ranges written (outputs, including read-modify-write state) and read
// (inputs).  Outputs must be pairwise disjoint and disjoint from every
// input, except one explicitly allowed identical pair (y == x in place).
class Aliases {
 public:
  void out(const void* p, int64_t bytes) { add(outs_, no_, p, bytes); }
  void in(const void* p, int64_t bytes) { add(ins_, ni_, p, bytes); }
  void allow_identical(const void* a, const void* b) { allow_a_ = a; allow_b_ = b; }
  bool ok() const {
    for (int i = 0; i < no_; ++i) {
      for (int j = i + 1; j < no_; ++j)
        if (overlap(outs_[i], outs_[j])) return false;
      for (int j = 0; j < ni_; ++j)
        if (overlap(outs_[i], ins_[j]) && !allowed(outs_[i], ins_[j])) return false;
    }
    return true;
  }

 private:
  struct Span { uintptr_t lo, hi; };
  static constexpr int kCap = 4 * ECHO_MAX_RANKS + 16;
  static void add(Span* s, int& k, const void* p, int64_t bytes) {
    if (!p || bytes <= 0 || k >= kCap) return;
    s[k].lo = (uintptr_t)p;
    s[k].hi = (uintptr_t)p + (uintptr_t)bytes;
    ++k;
  }
  static bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
  bool allowed(const Span& o, const Span& i) const {
    if (!allow_a_) return false;
    const uintptr_t a = (uintptr_t)allow_a_, b = (uintptr_t)allow_b_;
    return o.lo == i.lo && o.hi == i.hi && ((o.lo == a && i.lo == b) || (o.lo == b && i.lo == a));
  }
  Span outs_[kCap], ins_[kCap];
  int no_ = 0, ni_ = 0;
  const void* allow_a_ = nullptr;
  const void* allow_b_ = nullptr;
};

}  // namespace echo
