// guard.cuh -- exceptions end at the C boundary. Plain C++ (no CUDA types).
#pragma once
#include <new>
#include <string>

#include "gpt2.h"

namespace g2 {

// f(), or an error code with a message in *msg when it throws. The messages are short enough for a
// string to hold them without memory of its own.
template <class F>
int guarded(std::string* msg, F&& f) noexcept {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    *msg = "no host memory";
    return GPT2_ERR_OOM;
  } catch (...) {
    *msg = "internal error";
    return GPT2_ERR_CUDA;
  }
}

}  // namespace g2
