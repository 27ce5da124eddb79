// grouped_few.cu -- grouped products of few rows per group (a decoder's tokens):
// Y[i] = epilogue(X[source(i)] B[g]) with B[g]'s transpose stored by rows.
//
// Bound by reading the matrices of the groups that have rows.  A block takes 16
// rows of a group and 16 of its matrix's N rows; its eight warps split the
// contraction 128 columns at a time, and every lane keeps eight 16-byte loads of
// the matrix in flight, 64 KB per SM; the sums are joined in shared memory, always
// in the same order.  The matrix fragments are loaded as they are used: nothing is
// gained by staging what is read once.  One row through 8 matrices of 2048 x 4096
// (134 MB): 27 us, 5.0 TB/s; the tiles of 128 rows take 46, waiting for one
// 8 KB copy after another.
#include "direct.cuh"
#include "grouped.h"

namespace tg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;
constexpr int kCols = 16;   // two fragments of 8
constexpr int kStep = 128;  // of the contraction, per warp

template <bool BF>
__global__ void __launch_bounds__(kThreads, 2) few_rows_kernel(const __grid_constant__ FewRowsParams p) {
    __shared__ float joined[kWarps / 2][8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const RowTile tile = find_tile<kRows>(p.offset, p.groups, p.rows, blockIdx.y, lane);
    if (tile.g < 0) return;
    const uint16_t* x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = g + 8 * j;
        long long from = -1;
        if (i < tile.rows) from = p.row ? p.row[tile.lo + i] : tile.lo + i;
        if (p.row && from >= 0) from /= p.per_row;
        x[j] = from >= 0 && from < p.x_rows ? p.x + from * p.ldx : nullptr;
    }
    for (int n0 = blockIdx.x * kCols; n0 < p.n; n0 += gridDim.x * kCols) {
        const uint16_t* b[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int n = n0 + 8 * f + g;
            b[f] = n < p.n ? p.b + tile.g * p.stride_b + n * p.ldb : nullptr;
        }
        float c[2][4] = {};
        const uint4 none = make_uint4(0, 0, 0, 0);
        const bool second = tile.rows > 8;
        for (int k = warp * kStep; k < p.k; k += kWarps * kStep) {
            uint4 bv[2][4], xv[2][4];
            if (k + kStep <= p.k) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int f = 0; f < 2; ++f) bv[f][h] = b[f] ? __ldcs(reinterpret_cast<const uint4*>(b[f] + k + 32 * h + 8 * q)) : none;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        xv[j][h] = x[j] && (j == 0 || second) ? *reinterpret_cast<const uint4*>(x[j] + k + 32 * h + 8 * q) : none;
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        bv[f][h] = b[f] ? load8(b[f], k + 32 * h + 8 * q, p.k) : none;
                        xv[f][h] = x[f] ? load8(x[f], k + 32 * h + 8 * q, p.k) : none;
                    }
            }
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    mma<BF>(c[f], xv[0][h].x, xv[1][h].x, xv[0][h].y, xv[1][h].y, bv[f][h].x, bv[f][h].y);
                    mma<BF>(c[f], xv[0][h].z, xv[1][h].z, xv[0][h].w, xv[1][h].w, bv[f][h].z, bv[f][h].w);
                }
        }
        // the warps' sums, half of them to the other half, three times
#pragma unroll
        for (int half = kWarps / 2; half; half /= 2) {
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int j = 0; j < 8; ++j) joined[warp - half][j][lane] = c[j / 4][j % 4];
            }
            __syncthreads();
            if (warp < half) {
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j / 4][j % 4] += joined[warp][j][lane];
            }
            __syncthreads();
        }
        if (warp) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = g + 8 * j;
            if (i >= tile.rows) continue;
            const long long r = tile.lo + i;
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = n0 + 8 * f + 2 * q + h;
                    if (n >= p.n) continue;
                    float y = c[f][2 * j + h];
                    if (p.bias) y += wide<BF>(p.bias[tile.g * p.ld_bias + n]);
                    if (p.relu) y = y < 0.0f ? 0.0f : y;  // (a NaN stays one)
                    if (p.relu_of && !(wide<BF>(p.relu_of[r * p.ld_relu + n]) > 0.0f)) y = 0.0f;
                    p.y[r * p.ldy + n] = narrow<BF>(y);
                }
        }
    }
}

}  // namespace

cudaError_t launch_few_rows(const FewRowsParams& p, bool bf16, long long tiles, int sms, cudaStream_t stream) {
    // Blocks of several tiles of columns pay once for finding their rows: as many as
    // make one round of two blocks per SM, where that is up to four (one row through 8
    // matrices of 2048 x 4096: 1024 tiles 35 us, in 256 blocks 31); else two (16 rows
    // through 8 of 64 such matrices each: 119 us with two, 128 with one, 138 with eight).
    const long long columns = (p.n + kCols - 1) / kCols, round = 2LL * sms;
    const long long each = columns * tiles <= 4 * round ? (columns * tiles + round - 1) / round : 2;
    const dim3 grid((unsigned)((columns + each - 1) / each), (unsigned)tiles, 1);
    if (bf16)
        few_rows_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else
        few_rows_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace tg
