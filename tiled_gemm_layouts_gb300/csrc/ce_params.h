// ce_params.h -- what the host side hands to the linear cross entropy kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// The launches of linear cross entropy (l: logits, G: gradient of the logits).
enum CeMode : int {
    CE_LSE = 0,       // l = H W^T, reduced to (max, sum of exponentials) per row and tile
    CE_GRAD = 1,      // l again, turned into a piece of G
    CE_PRODUCTS = 2,  // from a piece of G: dH += G W (side 0) and dW = G^T H (side 1)
};

// One tiled product P * Q^T or P * Q and where its tiles go.
struct CeSide {
    // One 64-deep K-block per box (MN-major Q: 64 of its columns, and all the
    // columns of a tile in map_q3), and two K-blocks per box.  Every copy has
    // a fixed cost, so the wide boxes are used wherever they hold whole
    // blocks: the first p_pairs / q_pairs K-blocks, the first q_whole columns.
    CUtensorMap map_p, map_q, map_q3, map_p2, map_q2;
    CUtensorMap map_c;           // tensor stores of the output
    int p_pairs, q_pairs, q_whole;
    int num_kb;              // K-blocks of the contraction (or of one split of it)
    int tiles_m, tiles_n;    // 0: this side has no work
    int group_m;             // raster: tile rows per group
    uint32_t idesc;
    uint32_t p_bytes;        // bytes one K-block of P lands in a CTA
    int out_rows, out_cols;  // of dH's planes, or of this piece of dW
};

struct alignas(128) CeParams {
    CeSide side[2];
    int bf16;
    // Rows that count, on the device (null: all): only tile rows of logits and
    // of dH, and K-blocks of dW's contraction, that hold one are worked on.
    const int* live;
    // CE_LSE and CE_GRAD
    int rows;                // T
    int cols;                // columns of the logits in this launch (a piece of V)
    long long col0;          // first of them in the vocabulary
    const long long* target; // CE_LSE: [T] as the caller gave it
    float2* part;            // CE_LSE: [T][tiles_n][2 halves] (max in log2 units, sum of powers of two)
    float* hit;              // CE_LSE: [T] logit of the target, in log2 units
    const int* row_target;   // CE_GRAD: per compacted row, its target
    const float2* row_scale; // CE_GRAD: per compacted row, lse in log2 units and factor of G
    // CE_PRODUCTS
    int splits, all_kb;      // dH: splits of the contraction, each side[0].num_kb deep, and all of it
    int accumulate;          // dH: add to what the planes hold
    void* out;               // dW: first row of this piece
    long long ldo;
    int n_tma;               // dW: columns the tensor map holds; the kernel stores the others itself
    const float* alpha;      // dW: factor of the product, on the device
    // watchdog
    long long timeout_cycles;
    int* status;
};

// Tile of a launch: `bn` columns; 256 rows on a CTA pair or 128 on one CTA.
struct CeTile {
    int bn, pair;
    int rows() const { return pair ? 256 : 128; }
};

// `chained`: the launch may be scheduled while the kernel before it in the
// stream still runs (every kernel here waits for that one's end by itself).
cudaError_t launch_ce(int mode, const CeParams& p, CeTile tile, int sms, bool chained,
                      cudaStream_t stream);

}  // namespace tg
