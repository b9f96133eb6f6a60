// abi.hpp -- what the files of the C ABI share.
#pragma once
#include <hip/hip_runtime.h>

namespace oba {

// Runs fn(ctx), which launches kernels on st, bracketed by timing events
// under `name` when timing is enabled; OBA_EHIP (with its text) if a launch
// failed.
int abi_launch(const char* name, hipStream_t st, void (*fn)(void*), void* ctx);

}  // namespace oba
