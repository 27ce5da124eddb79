// grouped.h -- what the host entry points of the grouped products share
// (grouped.cu, adapters.cu).
#pragma once

#include "grouped_params.h"
#include "host_common.h"

namespace tg {

constexpr int64_t kMaxRowGroups = 4096;

// Products of few rows per group, B by rows of its transpose (grouped_few.cu).
constexpr int kFewTileRows = 16;
struct FewRowsParams {
    const int* offset;
    int groups, rows, x_rows, per_row, n, k;
    const uint16_t* x;
    long long ldx;
    const int* row;
    const uint16_t* b;
    long long ldb, stride_b;
    uint16_t* y;
    long long ldy;
    const uint16_t* bias;
    long long ld_bias;
    int relu;
    const uint16_t* relu_of;
    long long ld_relu;
};
cudaError_t launch_few_rows(const FewRowsParams& p, bool bf16, long long tiles, int sms, cudaStream_t stream);

}  // namespace tg
