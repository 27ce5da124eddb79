// ce_params.h -- what the host side hands to the linear cross entropy kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// The four products of linear cross entropy, each a tiled GEMM P * Q^T or
// P * Q with its own epilogue (l: logits, G: gradient of the logits).
enum CeMode : int {
    CE_LSE = 0,   // l = H W^T, reduced to (max, sum of exponentials) per row and tile
    CE_GRAD = 1,  // l again, turned into a piece of G
    CE_DH = 2,    // G W, added into fp32 planes
    CE_DW = 3,    // G^T H, a piece of dW
};

struct alignas(128) CeParams {
    CUtensorMap map_p, map_q;    // one 64-deep K-block of each operand per box
    CUtensorMap map_p2, map_q2;  // two K-blocks per box, where p_2k / q_2k
    CUtensorMap map_c;           // stores: G (CE_GRAD), fp32 planes (CE_DH), dW (CE_DW)
    int p_2k, q_2k;
    int q_3d;             // MN-major Q: one 3-D box per K-block (else 64-column boxes)
    uint32_t p_bytes;     // bytes one K-block of P lands in a CTA
    int num_kb;           // K-blocks of the whole contraction
    int kb_per_split;     // K-blocks of one split of it (num_kb when there is one)
    int tiles_m, tiles_n, splits;
    int group_m;          // raster: tile rows per group
    uint32_t idesc;
    int bf16;
    // Rows that count, on the device: CE_GRAD and CE_DH then run only the tile
    // rows that hold one, CE_DW only the K-blocks (null: all).
    const int* live;
    // CE_LSE and CE_GRAD
    int rows;             // T
    int cols;             // columns of the logits in this launch (a piece of V)
    long long col0;       // first of them in the vocabulary
    const long long* target;  // CE_LSE: [T] as the caller gave it
    float2* part;         // CE_LSE: [T][tiles_n] (max in log2 units, sum of powers of two)
    float* hit;           // CE_LSE: [T] logit of the target
    const int* row_target;    // CE_GRAD: per compacted row, its target
    const float2* row_scale;  // CE_GRAD: per compacted row, lse in log2 units and factor of G
    int out_rows, out_cols;  // CE_DH: of a plane; CE_DW: of this piece of dW
    // CE_DH
    int accumulate;       // add to what the planes hold
    // CE_DW
    void* out;            // first row of this piece of dW
    long long ldo;
    int n_tma;            // columns the tensor map holds; the kernel stores the others itself
    const float* alpha;   // factor of the product, on the device
    // watchdog
    long long timeout_cycles;
    int* status;
};

// Tile of a launch: `bn` columns; 256 rows on a CTA pair or 128 on one CTA.
struct CeTile {
    int bn, pair;
};

cudaError_t launch_ce(int mode, const CeParams& p, CeTile tile, int sms, cudaStream_t stream);

}  // namespace tg
