// prefix_tc.h -- launcher of the tensor-core kernel for the shared part of a shared-prefix decode.
#pragma once

#include "saw_internal.h"

namespace saw {

// How the prefix's work is cut: pairs of 128-row tiles per kv head, and runs of split_blocks 128-token
// blocks.  The kernel writes hkv * row_blocks * splits pieces of 8 rows.
struct PrefixTcShape {
    int32_t row_blocks, row_pairs, splits, split_blocks;
};
PrefixTcShape prefix_tc_shape(int32_t num_kv_heads, int64_t rows, int32_t prefix_len, int32_t sms);

cudaError_t launch_prefix_tc(const DecodeArgs &a, const int32_t *prefix_table, int32_t prefix_len,
                             const PrefixTcShape &s, float *slots, cudaStream_t stream);

}  // namespace saw
