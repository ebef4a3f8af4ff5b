// Host-side encoding of the TMA tensor maps that the GEMM kernels read their bf16 operands through.
// Every map has 128-byte swizzled boxes (inner extent at most 64 elements) and fills with zeros past
// its extents. false: the driver refused the map (or has no encoder).
#pragma once

#include <cuda.h>

#include <cstdint>

namespace tpx {

// 2-D bf16 view [outer, inner] with row stride `ld` elements.
bool encode_bf16_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                    uint32_t box_inner, uint32_t box_outer);
// 3-D bf16 view [count, rows, inner], row stride `ld` elements, matrices rows * ld elements apart;
// boxes of one matrix. A box that runs past a matrix's last row is filled with zeros there, and does
// not reach into the next matrix.
bool encode_bf16_3d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t count, uint64_t ld,
                    uint32_t box_inner, uint32_t box_rows);

// 3-D view [count, rows, cols] of a contiguous fp32 or bf16 output for stores of 32 x 32 boxes, whose rows of 128 (64)
// bytes lie swizzled in shared memory with the pattern of that width.
bool encode_out_3d(CUtensorMap* m, void* base, bool f32, uint64_t cols, uint64_t rows, uint64_t count);

}  // namespace tpx
