// stage.cu -- row copies for operands the tensor maps cannot describe.
//
// A TMA tensor map needs a 16-byte-aligned base and row strides that are whole
// 16-byte units.  Positive strides of any size are valid arguments all the
// same (ninetoothed.org "Named layouts", section "Runtime and compilation"),
// so tg_gemm_ws copies such an operand into an aligned dense buffer in the
// caller's workspace first, and copies an unaligned C out of one afterwards.
// The copy is a plain bandwidth-bound kernel: one thread moves 8 consecutive
// elements of a row (stage.cuh).  The store is one 16-byte access where its
// side is aligned.  So is the load; a load that is not takes the two aligned
// 16-byte words that hold its elements (the neighbour reads one of them too,
// from L1) and shifts them together, except where the second would end past
// the source's last byte.
#include "stage.cuh"

namespace tg {

namespace {

__global__ void copy_rows_kernel(const CopyJob job) {
    copy_rows(job, blockIdx.x * (long long)blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}

}  // namespace

// Copies rows x cols 16-bit elements from (src, lds) to (dst, ldd), both
// strides in elements, asynchronously on `stream`.
cudaError_t launch_copy_rows(const void* src, long long lds, void* dst, long long ldd,
                             long long rows, long long cols, cudaStream_t stream) {
    if (rows <= 0 || cols <= 0) return cudaSuccess;
    const long long work = rows * ((cols + 7) / 8);
    const long long blocks = (work + 255) / 256;
    copy_rows_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(CopyJob{
        static_cast<const uint16_t*>(src), lds, static_cast<uint16_t*>(dst), ldd, rows, cols});
    return cudaGetLastError();
}

}  // namespace tg
