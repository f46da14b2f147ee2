// Shared by the files that implement C entry points (defined in sffn_api.cpp): the calling
// thread's error message, and launches timed by name while profiling is on.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sparse_ffn.h"

namespace sffn {

sffn_status_t api_fail(sffn_status_t s, const char* msg) noexcept;
sffn_status_t api_launch(const char* name, hipStream_t s, hipError_t (*f)(void*), void* ctx) noexcept;
template <typename Fn>
inline sffn_status_t api_run(const char* name, hipStream_t s, Fn& f) noexcept {
  return api_launch(name, s, [](void* c) -> hipError_t { return (*static_cast<Fn*>(c))(); }, &f);
}

}  // namespace sffn
