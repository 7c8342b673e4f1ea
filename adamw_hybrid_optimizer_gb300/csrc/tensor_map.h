// Tensor maps of matrices for TMA (ns_gemm.cu).
#pragma once

#include <cuda.h>

namespace muon {

// 3-D bf16 map (inner, rows, batch) with a box of (64, box_rows, 1) and 128-byte swizzle; elements past the inner or row
// extent load as zeros and are not stored. ld and mstride in elements, multiples of 8; base 16-byte aligned.
bool make_bf16_map(CUtensorMap *map, const void *base, long long inner, long long rows, long long batch, long long ld,
                   long long mstride, int box_rows);
// As above for fp32, with a box of (32, box_rows, 1); ld and mstride multiples of 4.
bool make_f32_map(CUtensorMap *map, const void *base, long long inner, long long rows, long long batch, long long ld,
                  long long mstride, int box_rows);

}  // namespace muon
