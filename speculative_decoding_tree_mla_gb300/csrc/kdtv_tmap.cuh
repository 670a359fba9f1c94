// TMA tensor-map helper shared by the tensor-core translation units.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace kdtv {

// 2-D bf16 tensor map: a rows x cols view with a row stride of
// row_stride_elems elements (0 = cols), boxes of box_rows x box_cols, 128-byte
// swizzle (or 64-byte with swizzle_bytes = 64, for 32-column boxes).
CUresult encode_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                   uint32_t box_cols, uint32_t box_rows, uint64_t row_stride_elems = 0,
                   int swizzle_bytes = 128);

// Tensor map of `rank` (3..4) dimensions, innermost first, of 2-byte (bf16) or
// 1-byte elements; strides in bytes, of all but the innermost dimension.  128-,
// 64- or 32-byte swizzle, or none (0).
CUresult encode_nd(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
                   const uint64_t* strides, const uint32_t* box, int elem_bytes, int swizzle_bytes);

}  // namespace kdtv
