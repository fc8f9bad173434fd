// TMA tensor maps for entry points that take no plan (runtime.cu has the encoder).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace muon {

// Map of a [count][rows][ld] array of bf16, logical (cols, rows, count), box box_x x box_y x 1
// with the 128-byte swizzle.
bool encode_tensor_map(CUtensorMap* map, void* base, int64_t cols, int64_t rows, int64_t count, int64_t ld, uint32_t box_x,
                       uint32_t box_y);

}  // namespace muon
