// tma_host.h -- host-side TMA tensor-map encoding used by the tensor-core kernels.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace gca {

// Tensor map over a row-major bf16 matrix [rows, row_elems] (row stride
// row_elems * 2 bytes, a multiple of 16), box of 64 columns x box_rows rows,
// 128-byte swizzle.  Returns false if the driver entry point is missing or
// rejects the arguments.
bool encode_bf16_rows(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_elems,
                      uint32_t box_rows);

// The same view with a box of box_cols (64 or 32) columns: 64 columns use the
// 128-byte swizzle, 32 columns the 64-byte swizzle (one box row per swizzle span).
bool encode_bf16_rows_box(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_elems,
                          uint32_t box_cols, uint32_t box_rows);

// Tensor map over bf16 sequences [B, L, row_elems] (row stride row_elems * 2
// bytes, a multiple of 16), box of 64 columns x box_rows rows x 1 sequence,
// 128-byte swizzle.  Rows outside [0, L) of a sequence are out of bounds:
// loads fill them with zeros, stores skip them.
bool encode_bf16_seq(CUtensorMap* map, const void* base, uint64_t B, uint64_t L, uint64_t row_elems,
                     uint32_t box_rows);

// Tensor map over a bf16 tensor of three dimensions (innermost first) whose two
// outer strides are given in elements (multiples of 8), with a 128-byte swizzle
// and a box whose innermost extent is 64 elements.  Elements outside the tensor
// read as zeros and are not written.  wide: L2 fetches 256 bytes around what a load
// touches, else 128.
bool encode_bf16_3d(CUtensorMap* map, const void* base, uint64_t n0, uint64_t n1, uint64_t n2,
                    uint64_t stride1, uint64_t stride2, uint32_t box1, uint32_t box2, bool wide = true);

// The same over four dimensions.
bool encode_bf16_4d(CUtensorMap* map, const void* base, const uint64_t (&n)[4], const uint64_t (&stride)[3],
                    const uint32_t (&box)[3], bool wide = true);

// Tensor map over a row-major fp32 matrix [rows, row_elems] (row stride
// row_elems * 4 bytes, a multiple of 16), box of box_cols x box_rows (box_cols
// * 4 a multiple of 16), no swizzle: the box lands in shared memory as
// box_rows dense rows of box_cols floats.
bool encode_f32_box(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_elems,
                    uint32_t box_cols, uint32_t box_rows);

}  // namespace gca
