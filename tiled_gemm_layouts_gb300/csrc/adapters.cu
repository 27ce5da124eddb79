// adapters.cu -- low-rank adapters of many requests beside a shared projection
// (tg_adapters).
//
//   u_i = x_t A_g^T   (rank values, fp32)        y_t += s_g (u_i B_g^T)
//
// for each grouped row i, its token t = row[i] and its group (adapter) g.
//
// Few rows (a decoder's batch).  Bound by latency and by reading A and B: at
// 64 rows, each with an adapter of its own of rank 16 between 4096 columns, they
// are 16.8 MB.  The first kernel cuts a row's columns into pieces, one per
// block; a warp sums a piece's products for some of the rank, 16 bytes per lane
// and load, and writes the sums by piece.  The second adds the pieces up (in
// their order) and gives every column of y to one thread, whose row of B lies
// beside its neighbours' in memory.  It is launched behind the first one's tail.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "../../include/tilegemm.h"
#include "chained.cuh"
#include "grouped.h"

namespace tg {
namespace {

constexpr int kLowThreads = 256;
constexpr int64_t kMaxRank = 128;
constexpr int kMaxPieces = 32;

struct AdapterParams {
    int T, G, rank, K, N;
    const uint16_t* x;
    long long ldx;
    const int* row;
    const int* offset;
    const uint16_t* a;
    long long lda;
    const uint16_t* b;
    long long ldb;
    const float* scale;
    uint16_t* y;
    long long ldy;
    int pieces, piece;  // of K, and columns (a multiple of 256) of one
    float* part;        // [T][pieces][rank]
};

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
// sum += a . b over 8 columns, those from `left` on left out
template <bool BF>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, int left, float sum) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int s = (j & 1) * 16;
        const float x = wide<BF>((uint16_t)(aw[j / 2] >> s)), y = wide<BF>((uint16_t)(bw[j / 2] >> s));
        if (j < left) sum = fmaf(x, y, sum);
    }
    return sum;
}

// The group of grouped row i by the whole warp, or -1: the last whose rows start
// at or before i, if i is before its end.  32 offsets at a time.
__device__ __forceinline__ int group_of(const AdapterParams& p, int i, int lane) {
    int lo = 0, span = p.G + 1;  // the answer is among lo .. lo + span - 1
    while (span > 1) {
        const int step = (span + 31) / 32;
        const int at = lo + lane * step;
        const bool starts = lane * step < span && p.offset[at] <= i;
        const unsigned mask = __ballot_sync(0xffffffffu, starts);
        if (mask == 0) return -1;
        const int top = 31 - __clz(mask);
        lo += top * step;
        span = min(step, span - top * step);
    }
    return p.offset[lo] <= i && lo < p.G ? lo : -1;
}

template <bool BF>
__global__ void __launch_bounds__(kLowThreads) low_kernel(const AdapterParams p) {
    allow_next_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.y;
    const int g = group_of(p, i, lane);
    const int t = p.row[i];
    if (g < 0 || t < 0 || t >= p.T) return;
    const int k0 = blockIdx.x * p.piece, k1 = min(p.K, k0 + p.piece);
    const uint16_t* x = p.x + (long long)t * p.ldx;
    const uint16_t* a = p.a + (long long)g * p.rank * p.lda;
    constexpr int kTogether = 4;  // of the rank, so that their loads are in flight together
    for (int r0 = warp * kTogether; r0 < p.rank; r0 += kLowThreads / 32 * kTogether) {
        float sum[kTogether] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = k0 + 8 * lane; k < k1; k += 256) {
            const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
                if (r0 + j < p.rank)
                    sum[j] = dot8<BF>(xv, *reinterpret_cast<const uint4*>(a + (long long)(r0 + j) * p.lda + k), k1 - k, sum[j]);
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
#pragma unroll
            for (int d = 16; d; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
            if (lane == 0 && r0 + j < p.rank)
                p.part[((long long)i * p.pieces + blockIdx.x) * p.rank + r0 + j] = sum[j];
        }
    }
}

template <bool BF>
__global__ void __launch_bounds__(kLowThreads) add_kernel(const AdapterParams p) {
    __shared__ float low[kMaxRank];
    const int i = blockIdx.y;
    const int g = group_of(p, i, threadIdx.x & 31);
    const int t = p.row[i];
    if (g < 0 || t < 0 || t >= p.T) return;
    wait_for_previous_kernel();
    const float* part = p.part + (long long)i * p.pieces * p.rank;
    for (int r = threadIdx.x; r < (int)kMaxRank; r += kLowThreads) {
        float sum = 0.0f;
        if (r < p.rank)
            for (int k = 0; k < p.pieces; ++k) sum += part[k * p.rank + r];
        low[r] = sum;
    }
    __syncthreads();
    const float s = p.scale ? p.scale[g] : 1.0f;
    for (int n = blockIdx.x * kLowThreads + threadIdx.x; n < p.N; n += gridDim.x * kLowThreads) {
        const uint16_t* b = p.b + ((long long)g * p.N + n) * p.ldb;
        uint16_t* y = p.y + (long long)t * p.ldy + n;
        float sum = 0.0f;
        for (int r = 0; r < p.rank; r += 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(b + r);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = wide<BF>((uint16_t)(w[j / 2] >> ((j & 1) * 16)));
                if (r + j < p.rank) sum = fmaf(x, low[r + j], sum);
            }
        }
        *y = narrow<BF>(fmaf(s, sum, wide<BF>(*y)));
    }
}

// Pieces of K: enough blocks for every SM, a multiple of 256 columns each.
int pieces_of(int64_t T, int64_t K) {
    const int64_t most = (K + 255) / 256, wanted = (1024 + T - 1) / T;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(most, wanted), kMaxPieces));
}

int check_sizes(int64_t T, int64_t N, int64_t K, int64_t rank, int64_t G, int dtype) {
    if (T <= 0 || N <= 0 || K <= 0 || rank <= 0 || G <= 0 || T > kMaxSize || N > kMaxSize || K > kMaxSize ||
        rank > kMaxRank || G > kMaxRowGroups)
        return TG_ERR_INVALID_ARG;
    if (dtype != TG_F16 && dtype != TG_BF16) return TG_ERR_DTYPE;
    return TG_OK;
}

size_t workspace_of(int64_t T, int64_t K, int64_t rank) {
    return (size_t)T * (size_t)pieces_of(T, K) * (size_t)rank * sizeof(float);
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_adapters_workspace_size(int64_t T, int64_t N, int64_t K, int64_t rank, int64_t G, tg_dtype dtype,
                                          size_t* bytes) {
    const int rc = check_sizes(T, N, K, rank, G, (int)dtype);
    if (rc) return rc;
    if (!bytes) return TG_ERR_INVALID_ARG;
    *bytes = workspace_of(T, K, rank);
    return TG_OK;
}

extern "C" int tg_adapters(int64_t T, int64_t N, int64_t K, int64_t rank, int64_t G, const void* X, int64_t ldx,
                           const int32_t* row, const int32_t* offset, const void* A, int64_t lda, const void* B,
                           int64_t ldb, const float* scale, void* Y, int64_t ldy, tg_dtype dtype, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    int rc = check_sizes(T, N, K, rank, G, (int)dtype);
    if (rc) return rc;
    if (!X || !row || !offset || !A || !B || !Y || !workspace) return TG_ERR_INVALID_ARG;
    if (ldx < K || lda < K || ldb < rank || ldy < N || ldx > kMaxLd || lda > kMaxLd || ldb > kMaxLd || ldy > kMaxLd)
        return TG_ERR_STRIDE;
    auto off = [](const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; };
    if (!aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(Y) || ldx % 8 || lda % 8 || ldb % 8 || ldy % 8 ||
        off(row, 4) || off(offset, 4) || off(scale, 4) || off(workspace, 256))
        return TG_ERR_ALIGN;
    const size_t need = workspace_of(T, K, rank);
    if (workspace_bytes < need) return TG_ERR_BUFFER;
    // (G * rank rows of A and G * N of B, one after another)
    const void* ptrs[8] = {Y, workspace, X, A, B, row, offset, scale};
    const Span spans[8] = {span_of(Y, T, N, ldy), span_bytes(workspace, need), span_of(X, T, K, ldx),
                           span_of(A, G * rank, K, lda), span_of(B, G * N, rank, ldb), span_bytes(row, (u128)T * 4),
                           span_bytes(offset, (u128)(G + 1) * 4), span_bytes(scale, (u128)G * 4)};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 8; ++j)
            if (intersects(spans[i], spans[j])) return TG_ERR_OVERLAP;
    if (T > 65535) return TG_ERR_INVALID_ARG;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (!load_driver_entry_points()) return TG_ERR_CUDA;
    PointerChecks check{dev};
    for (int i = 0; i < 8; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    AdapterParams p = {};
    p.T = (int)T;
    p.G = (int)G;
    p.rank = (int)rank;
    p.K = (int)K;
    p.N = (int)N;
    p.x = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.row = row;
    p.offset = offset;
    p.a = static_cast<const uint16_t*>(A);
    p.lda = lda;
    p.b = static_cast<const uint16_t*>(B);
    p.ldb = ldb;
    p.scale = scale;
    p.y = static_cast<uint16_t*>(Y);
    p.ldy = ldy;
    const int pieces = pieces_of(T, K);
    p.piece = (int)((K + pieces * 256LL - 1) / (pieces * 256LL) * 256);
    p.pieces = (int)((K + p.piece - 1) / p.piece);
    p.part = static_cast<float*>(workspace);
    const dim3 low((unsigned)p.pieces, (unsigned)T, 1);
    const dim3 add((unsigned)std::min<int64_t>((N + kLowThreads - 1) / kLowThreads, 1024), (unsigned)T, 1);
    if (dtype == TG_BF16)
        low_kernel<true><<<low, kLowThreads, 0, stream>>>(p);
    else
        low_kernel<false><<<low, kLowThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = dtype == TG_BF16 ? launch_chained(add_kernel<true>, add, kLowThreads, stream, p)
                             : launch_chained(add_kernel<false>, add, kLowThreads, stream, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
