// tensor_map.h -- TMA descriptors of arrays of rows.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace sd {

// [rows][heads][128] of bf16 (or of bytes), with a box of {x values, y heads, z rows} and, with `swizzle`, the 128-byte
// swizzle.
cudaError_t encode_rows_map(CUtensorMap* m, const void* base, bool bytes, long heads, long rows, int x, int y, int z,
                            bool swizzle);

}  // namespace sd
