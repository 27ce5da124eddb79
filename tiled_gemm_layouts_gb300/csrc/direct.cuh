// direct.cuh -- products whose operands go from global memory into matrix
// fragments without a stop in shared memory, for kernels that wait for memory.
//
// A lane (g, q) of a warp (g = lane / 4, q = lane % 4) holds of mma.sync's operands
// two neighbouring elements of the contraction at a time.  The contraction's order
// is free, so it loads 8 neighbouring ones of a row at once and hands them to two
// instructions, the same way for both operands.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace tg {

template <bool BF>
__device__ __forceinline__ float wide(uint16_t h) {
    if constexpr (BF) return __uint_as_float((uint32_t)h << 16);
    return __half2float(__ushort_as_half(h));
}
template <bool BF>
__device__ __forceinline__ uint16_t narrow(float x) {
    if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    return __half_as_ushort(__float2half_rn(x));
}
template <bool BF>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    return (uint32_t)narrow<BF>(a) | (uint32_t)narrow<BF>(b) << 16;
}

// c += a b, 16 x 8 x 16: lane (g, q) holds of a rows g and g + 8, of b column g,
// of c rows g and g + 8, columns 2q and 2q + 1.
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Columns c .. c+7 of a row, zeros from `end` on.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int end) {
    if (c >= end) return make_uint4(0, 0, 0, 0);
    uint4 v = *reinterpret_cast<const uint4*>(row + c);
    if (c + 8 > end) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (c + 2 * j >= end) w[j] = 0;
            if (c + 2 * j + 1 >= end) w[j] &= 0xFFFFu;
        }
    }
    return v;
}
// And c .. c+3.
__device__ __forceinline__ uint2 load4(const uint16_t* row, int c, int end) {
    if (c >= end) return make_uint2(0, 0);
    uint2 v = *reinterpret_cast<const uint2*>(row + c);
    if (c + 4 > end) {
        if (c + 1 >= end) v.x &= 0xFFFFu;
        if (c + 2 >= end) v.y = 0;
        if (c + 3 >= end) v.y &= 0xFFFFu;
    }
    return v;
}

// The group, and the first and number of its rows, of tile t, when every
// group's rows are cut into tiles of kRows; g < 0 if there are fewer tiles.  Offsets
// outside 0..rows are taken for the nearest of them.
// By a whole warp, 128 groups at a time.
struct RowTile {
    int g, lo, rows;
};
template <int kRows>
__device__ __forceinline__ RowTile find_tile(const int* offset, int groups, int all_rows, int t, int lane) {
    for (int window = 0; window < groups; window += 128) {
        int end[5], tiles[4], incl = 0;
#pragma unroll
        for (int k = 0; k < 5; ++k) end[k] = max(0, min(offset[min(window + 4 * lane + k, groups)], all_rows));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            tiles[k] = (max(0, end[k + 1] - end[k]) + kRows - 1) / kRows;
            incl += tiles[k];
        }
        const int own = incl;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const unsigned later = __ballot_sync(0xffffffffu, t < incl);
        if (later) {
            const int owner = __ffs(later) - 1;
            int i = t - (incl - own), k = 0, lo = end[0], hi = end[1];
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (k == j && i >= tiles[j]) {
                    i -= tiles[j];
                    k = j + 1;
                    lo = end[j + 1];
                    hi = end[j + 2];
                }
            RowTile r;
            r.g = window + 4 * owner + __shfl_sync(0xffffffffu, k, owner);
            r.lo = __shfl_sync(0xffffffffu, lo + i * kRows, owner);
            r.rows = min(kRows, __shfl_sync(0xffffffffu, hi, owner) - r.lo);
            return r;
        }
        t -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return {-1, 0, 0};
}

}  // namespace tg
