// Helpers shared by the files that hold the C ABI's entry points.
#pragma once

#include <exception>
#include <string>

#include "common.cuh"

namespace gptq {

// Runs an entry point's body; no C++ exception leaves it.
template <typename F>
gptq_status guarded(F&& f) {
  const size_t mark = trace_mark();
  try {
    f();
    set_last_error("");
    return GPTQ_OK;
  } catch (const Error& e) {
    trace_discard(mark);
    set_last_error(e.msg);
    return e.status;
  } catch (const std::exception& e) {
    trace_discard(mark);
    set_last_error(std::string("internal error: ") + e.what());
    return GPTQ_ERR_CUDA;
  } catch (...) {
    trace_discard(mark);
    set_last_error("internal error");
    return GPTQ_ERR_CUDA;
  }
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline void require(bool ok, gptq_status s, const char* msg) {
  if (!ok) fail(s, "%s", msg);
}

}  // namespace gptq
