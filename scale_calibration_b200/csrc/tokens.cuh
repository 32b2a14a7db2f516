// The quantisation of tokens as the products use it (internal header).
#pragma once

#include "common.cuh"

namespace lh {

// Refusals of lh_quantize_tokens.
lh_status check_tokens(const void* X, lh_dtype x_dtype, int64_t n_src, int64_t c_in, int64_t ld_x, const int32_t* rows,
                       int64_t row_div, int64_t n_rows, const int64_t* offsets, int64_t n_groups, const uint8_t* packed,
                       const uint8_t* scale_tiles, const float* token_scale, const void* X_out, lh_dtype out_dtype);

}  // namespace lh
