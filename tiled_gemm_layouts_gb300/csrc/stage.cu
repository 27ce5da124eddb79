// stage.cu -- row copies for operands the tensor maps cannot describe.
//
// A TMA tensor map needs a 16-byte-aligned base and row strides that are whole
// 16-byte units.  Positive strides of any size are valid arguments all the
// same (ninetoothed.org "Named layouts", section "Runtime and compilation"),
// so tg_gemm_ws copies such an operand into an aligned dense buffer in the
// caller's workspace first, and copies an unaligned C out of one afterwards.
// The copy is a plain bandwidth-bound kernel: one thread moves 8 consecutive
// elements of a row.  The store is one 16-byte access where its side is
// aligned.  So is the load; a load that is not takes the two aligned 16-byte
// words that hold its elements (the neighbour reads one of them too, from L1)
// and shifts them together, except where the second would end past the
// source's last byte.
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

namespace {

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

__global__ void copy_rows_kernel(const uint16_t* __restrict__ src, long long lds,
                                 uint16_t* __restrict__ dst, long long ldd, long long rows,
                                 long long cols) {
    const uintptr_t end = reinterpret_cast<uintptr_t>(src + (rows - 1) * lds + cols);
    const long long vecs = (cols + 7) / 8;
    const long long total = rows * vecs;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const long long r = i / vecs, c0 = (i - r * vecs) * 8;
        const uint16_t* s = src + r * lds + c0;
        uint16_t* d = dst + r * ldd + c0;
        const int n = (int)(cols - c0 < 8 ? cols - c0 : 8);
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

}  // namespace

// Copies rows x cols 16-bit elements from (src, lds) to (dst, ldd), both
// strides in elements, asynchronously on `stream`.
cudaError_t launch_copy_rows(const void* src, long long lds, void* dst, long long ldd,
                             long long rows, long long cols, cudaStream_t stream) {
    if (rows <= 0 || cols <= 0) return cudaSuccess;
    const long long work = rows * ((cols + 7) / 8);
    const long long blocks = (work + 255) / 256;
    copy_rows_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(
        static_cast<const uint16_t*>(src), lds, static_cast<uint16_t*>(dst), ldd, rows, cols);
    return cudaGetLastError();
}

}  // namespace tg
