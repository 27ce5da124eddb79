// stage.cuh -- row copies for operands the tensor maps cannot describe, as
// part of a kernel (stage.cu has the kernel that only copies).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// 16 bytes from an even address, out of the aligned 16-byte words around it.
__device__ __forceinline__ uint4 load_shifted(const uint16_t* s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(s);
    const uint4* base = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
    const uint4 a = __ldg(base), b = __ldg(base + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int word = (int)(at & 15u) >> 2;
    uint32_t v[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {  // w[word + k] by selects
        v[k] = w[k];
#pragma unroll
        for (int j = 1; j < 4; ++j)
            if (k + j < 8) v[k] = word == j ? w[k + j] : v[k];
    }
    const uint32_t bits = (uint32_t)(at & 2u) * 8u;
    return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                      __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
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
