// Host-side helpers shared by the C entry points: the error text of a failed
// launch and the per-kernel timing around each launch (defined in
// kda_host.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Records the HIP error for kda_status_string and returns KDA_ERR_HIP.
int hip_fail(hipError_t e);

// Brackets one launch of the calling thread with events between
// kda_profile_begin and kda_profile_end; otherwise does nothing.
struct ProfScope {
  int kind;
  int64_t units;
  hipStream_t s;
  hipEvent_t a = nullptr;
  ProfScope(int k, int64_t u, hipStream_t st);
  void done();
};

}  // namespace kda

#define KDA_TRY(kind, units, expr)                   \
  do {                                               \
    kda::ProfScope ps_(kind, units, s);              \
    const hipError_t e_ = (expr);                    \
    ps_.done();                                      \
    if (e_ != hipSuccess) return kda::hip_fail(e_);  \
  } while (0)
