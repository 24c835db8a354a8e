// Tensor map for TMA loads of 8-bit page rows (tma_maps.cu).
#pragma once

#include <cuda.h>

namespace sas {

// TMA map of [rows, 128] bytes: 128 x 1 x box_rows boxes, 128-byte swizzle.
bool make_byte_map(CUtensorMap* map, const void* base, long long rows, int box_rows);

}  // namespace sas
