// grouped_params.h -- what the host side hands to the grouped product kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// The launches of rows that choose their weights.
enum GroupedMode : int {
    GROUPED_ROWS = 0,    // Y[i] = epilogue(X[source(i)] B[g]): tiles of a group's rows
    GROUPED_WEIGHT = 1,  // dB[g] = X^T dY over a group's rows, or its transpose
};

// Rows of a 16-bit matrix, one after another or by a list of rows.
struct GroupedRows {
    CUtensorMap box;     // 64 columns of consecutive rows (no list)
    CUtensorMap box2;    // GROUPED_ROWS: the same of two K-blocks, among the first `pairs`
    CUtensorMap gather;  // GROUPED_WEIGHT: four rows of 64 columns, by their numbers
    int pairs;
    const int* row;      // [R] or null: row i itself
    uint32_t magic;      // source row: row[i] / per_row = row[i] * magic >> shift
    int shift;
    int count;           // source rows; a row outside reads as zeros
    const void* base;    // for the list's copies
    long long ld;
    int cols;
};

struct alignas(128) GroupedParams {
    // GROUPED_WEIGHT: P holds the product's rows, Q its columns, both along their rows' columns.
    // Else: P is X, and map_q the matrices: {K, N, G} or {N, K, G}.
    GroupedRows p, q;
    CUtensorMap map_q, map_q2;  // map_q2: two K-blocks at once, among the first q_pairs (K-major matrices)
    int q_pairs;
    const int* offset;    // [groups + 1]
    int groups, rows;     // rows: R
    int num_kb;           // 64-deep K-blocks (not GROUPED_WEIGHT, whose rows are the depth)
    int tiles_m, tiles_n; // tiles_m: GROUPED_WEIGHT only
    int group_m;          // raster: tile rows that share their columns' operand in turn
    int m, n;             // m: rows of a dB (GROUPED_WEIGHT); n: columns of the output
    int q_mn;             // Q's columns contiguous in memory
    uint32_t idesc;
    int bf16;
    void* out;
    long long ldo, out_stride;  // out_stride: from one dB to the next
    const void* bias;           // [groups] rows
    long long ld_bias;
    int relu;
    const void* relu_of;        // [R] rows
    long long ld_relu;
    // watchdog
    long long timeout_cycles;
    int* status;
};

// Tile of a launch: `bn` columns; 256 rows on a CTA pair or 128 on one CTA.
// `list`: rows by a list, fetched by warps of their own.
struct GroupedTile {
    int bn, pair, list;
    int rows() const { return pair ? 256 : 128; }
    int blocks_rows() const { return pair && list ? 1 : 2; }  // K-blocks per transaction of GROUPED_ROWS
};

// `tiles`: the most tiles there can be.
cudaError_t launch_grouped(int mode, const GroupedParams& p, GroupedTile tile, long long tiles, int sms, cudaStream_t stream);

}  // namespace tg
