// outer.hpp -- segred_outer for other translation units.
#pragma once

#include "internal.hpp"

namespace segred {

// out[vc, m] = *scale * (left[n, vc])^T right, one segment of n rows: left's rows
// are `width` >= vc elements apart, row r of the right side is right[right_rows[r]]
// of its n rows, offsets = {0, n} on the device, `scale` on the device or null.
// Pointers are those of segred_outer, checked by the caller.
int outer_scaled(const void *left, int64_t width, int64_t vc, const void *right, const int64_t *right_rows, int64_t n,
                 int64_t m, int32_t dtype, const int64_t *offsets, void *out, int32_t out_dtype, const float *scale,
                 void *workspace, hipStream_t stream);

}  // namespace segred
