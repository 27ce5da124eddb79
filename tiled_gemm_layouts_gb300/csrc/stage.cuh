// stage.cuh -- row copies for operands the tensor maps cannot describe, as
// part of a kernel (stage.cu has the kernel that only copies).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// The 8 elements that start `s` elements (0 to 7) into two 16-byte units.
__device__ __forceinline__ uint4 funnel(uint4 a, uint4 b, int s) {
    const bool four = s & 4, two = s & 2;
    const uint32_t w0 = four ? a.z : a.x, w1 = four ? a.w : a.y, w2 = four ? b.x : a.z,
                   w3 = four ? b.y : a.w, w4 = four ? b.z : b.x, w5 = four ? b.w : b.y;
    const uint32_t v0 = two ? w1 : w0, v1 = two ? w2 : w1, v2 = two ? w3 : w2, v3 = two ? w4 : w3,
                   v4 = two ? w5 : w4;
    const uint32_t bits = (uint32_t)(s & 1) * 16;
    return make_uint4(__funnelshift_r(v0, v1, bits), __funnelshift_r(v1, v2, bits),
                      __funnelshift_r(v2, v3, bits), __funnelshift_r(v3, v4, bits));
}

// Elements between the 16-byte boundary before `p` and `p`.
__device__ __forceinline__ int shift_of(const uint16_t* p) {
    return (int)(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;
}

// 16 bytes from an even address, out of the aligned 16-byte units around it.
__device__ __forceinline__ uint4 load_shifted(const uint16_t* p) {
    const uint4* base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
    return funnel(__ldg(base), __ldg(base + 1), shift_of(p));
}

// i / d for 0 <= i, 0 < d: in 32 bits where both fit (a 64-bit division is a
// routine of a hundred instructions, most of a copied run's time).
__device__ __forceinline__ long long row_of(long long i, long long d) {
    if ((unsigned long long)(i | d) >> 32 == 0) return (uint32_t)i / (uint32_t)d;
    return i / d;
}

// rows x cols 16-bit elements from (src, lds) to (dst, ldd).
struct CopyJob {
    const uint16_t* src;
    long long lds;
    uint16_t* dst;
    long long ldd;
    long long rows, cols;  // rows 0: nothing to copy
};

// This thread's share of a copy by `threads` threads: every `threads`-th run
// of 8 elements.  (Four runs in flight per thread, or whole warps that load
// every word once and shuffle, need twice the registers and were slower.)
__device__ __forceinline__ void copy_rows(const CopyJob& job, long long thread, long long threads) {
    const uintptr_t end = reinterpret_cast<uintptr_t>(job.src + (job.rows - 1) * job.lds + job.cols);
    const long long vecs = (job.cols + 7) / 8;
    const long long total = job.rows * vecs;
    for (long long i = thread; i < total; i += threads) {
        const long long r = row_of(i, vecs), c0 = (i - r * vecs) * 8;
        const uint16_t* s = job.src + r * job.lds + c0;
        uint16_t* d = job.dst + r * job.ldd + c0;
        const int n = (int)(job.cols - c0 < 8 ? job.cols - c0 : 8);
        alignas(16) uint16_t v[8];
        if (n == 8 && (reinterpret_cast<uintptr_t>(s) & 15u) == 0) {
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(s);
        } else if (n == 8 && (reinterpret_cast<uintptr_t>(s) & ~uintptr_t(15)) + 32 <= end) {
            *reinterpret_cast<uint4*>(v) = load_shifted(s);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) v[j] = s[j];
        }
        if (n == 8 && (reinterpret_cast<uintptr_t>(d) & 15u) == 0) {
            *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) d[j] = v[j];
        }
    }
}

}  // namespace tg
