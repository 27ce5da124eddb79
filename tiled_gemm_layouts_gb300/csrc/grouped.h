// grouped.h -- what the host entry points of the grouped products share
// (grouped.cu, adapters.cu).
#pragma once

#include "grouped_params.h"
#include "host_common.h"

namespace tg {

constexpr int64_t kMaxRowGroups = 4096;

// `groups` matrices of `outer` rows of `inner` elements, ld and stride elements
// apart, in boxes of 64 x box_outer x 1 with the 128-byte swizzle.
bool encode_stack(CUtensorMap* map, int dtype, const void* base, int64_t inner, int64_t outer, int64_t groups,
                  int64_t ld, int64_t stride, uint32_t box_outer);

// Rows of a matrix: `row` (a list, or null), divided by per_row, and the maps of
// boxes of 64 columns x box_rows rows and of gathered rows.
bool encode_rows(GroupedRows* rows, int dtype, const void* base, int64_t count, int64_t cols, int64_t ld,
                 const int32_t* row, int64_t per_row, uint32_t box_rows);

}  // namespace tg
