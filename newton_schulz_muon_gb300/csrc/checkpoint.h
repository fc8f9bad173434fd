// What checkpoint.cu offers the library's other entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "muon.h"

namespace muon {

// x [rows][ld] bf16 <- the checkpoint's values (of a device and arguments that are checked).
// A kernel launched with programmatic dependence may begin while this one runs.
cudaError_t launch_checkpoint_load(const muon_checkpoint* checkpoint, void* x, int64_t ld, cudaStream_t stream);

}  // namespace muon
