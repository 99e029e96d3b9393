// What a kernel says about itself in the status word: a bounded wait that gave up, and the
// index checks of the bounds-checked build.  The word behind it has the site, a number of
// one place in the sources: waits 1.. tc_fwd, 21.. tc_bwd_q128, 31.. gemm_bf16, 41..
// ffn_tokens, 51.. gemm_split; indexes 101.. tc_fwd, 201.. tc_bwd_q128, 301.. gemm_bf16,
// 303 ffn_tokens, 311.. gemm_split.
//
// Device-side index checks of the bounds-checked build (compiled with
// -DCPATTN_BOUNDS_CHECK into libcpattn_checked.so; the normal build compiles
// them away).  A failing check records the first failure in the workspace
// status word (kStatusBounds and a site code naming the access) and tells the
// caller to skip the access; it never traps.  A skipped tensor load leaves its
// barrier incomplete, so the waiting role gives up through the kernel's
// bounded waits and the CTA leaves normally.
#pragma once
#include <stdint.h>

namespace cpattn {

constexpr int32_t kStatusTimeout = 1;  // status word: a bounded wait gave up
constexpr int32_t kStatusBounds = 3;   // status word: a device-side index check failed

// Polling rounds that a kernel which gives up waits for what it has in flight.
constexpr long long kDrainLimit = 1LL << 24;
constexpr long long kLandLimit = 1LL << 16;   // milliseconds: a load lands within microseconds

// The first site to give up is kept; the CTA's other waits give up too.
__device__ __forceinline__ void record_timeout(int32_t* status, volatile int* abort, int site) {
  if (atomicCAS(&status[0], 0, kStatusTimeout) == 0) status[1] = site;
  *abort = 1;
}

#ifdef CPATTN_BOUNDS_CHECK
__device__ __forceinline__ bool in_range_checked(long long v, long long lo, long long hi,
                                                 int32_t* status, int site) {
  if (v >= lo && v < hi) return true;
  if (status && atomicCAS(&status[0], 0, kStatusBounds) == 0) status[1] = site;
  return false;
}
#define CP_IN_RANGE(v, lo, hi, status, site) \
  ::cpattn::in_range_checked((long long)(v), (long long)(lo), (long long)(hi), (status), (site))
#else
#define CP_IN_RANGE(v, lo, hi, status, site) true
#endif

}  // namespace cpattn
