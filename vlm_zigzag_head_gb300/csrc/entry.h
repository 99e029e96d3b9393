// Helpers of the C entry points that live outside api.cu: the thread-local
// error message and the guard that keeps C++ exceptions inside the library.
#pragma once
#include <cuda_runtime.h>

#include <exception>
#include <string>

#include "../../include/cpattn.h"

namespace cpattn {

void set_last_error(const std::string& msg);   // api.cu
long long device_wait_limit();                 // api.cu

inline cp_status_t entry_fail(cp_status_t s, const std::string& msg) {
  set_last_error(msg);
  return s;
}

// Records CUDA events around the launches of a scope while profiling is on
// (cp_profile_begin; kinds as documented there).
struct ProfileScope {
  ProfileScope(int kind, cudaStream_t st, int launches = 1);
  ~ProfileScope();
  ProfileScope(const ProfileScope&) = delete;
  ProfileScope& operator=(const ProfileScope&) = delete;

 private:
  int kind;
  cudaStream_t st;
  cudaEvent_t a = nullptr, b = nullptr;
  int count;
};

#define ENTRY_CUDA(call, what)                                                                   \
  do {                                                                                           \
    cudaError_t e_ = (call);                                                                     \
    if (e_ != cudaSuccess)                                                                       \
      return ::cpattn::entry_fail(CP_ERR_CUDA,                                                   \
                                  std::string(what) + ": " + cudaGetErrorString(e_));            \
  } while (0)

#define ENTRY_TRY try {
#define ENTRY_CATCH                                                        \
  }                                                                        \
  catch (const std::exception& ex) {                                       \
    return ::cpattn::entry_fail(CP_ERR_INVALID_ARG, ex.what());            \
  }                                                                        \
  catch (...) {                                                            \
    return ::cpattn::entry_fail(CP_ERR_INVALID_ARG, "unknown exception");  \
  }

}  // namespace cpattn
