// Host-side helpers of the 8-bit integer kernels.
#pragma once

#include "sge_host.h"

namespace sge {

// 2-D int8 tensor map over a row-major [rows][cols] matrix with row pitch
// `pitch` bytes (a multiple of 16), box [box_rows][128], 128-byte swizzle,
// out-of-bounds elements read as zero.
int make_tmap_i8(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t pitch,
                 uint32_t box_rows);

}  // namespace sge
