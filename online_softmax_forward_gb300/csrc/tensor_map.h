// tensor_map.h -- TMA maps of the 16-bit tensors the tcgen05 kernels read.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace attn {

// The first `rows` rows of each slice of a [slices, S, d] 16-bit tensor as a 3-D TMA map, box
// 64 (d) x 128 (rows) x 1, 128-byte swizzle; rows outside read as zeros.  False if the driver
// refuses it.
bool make_tile_map(CUtensorMap *m, const void *base, bool bf16, int d, int S, int rows, int64_t slices);

}  // namespace attn
