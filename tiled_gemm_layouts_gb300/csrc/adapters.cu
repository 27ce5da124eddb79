// adapters.cu -- low-rank adapters of many requests beside a shared projection
// (tg_adapters).
//
//   u_i = x_t A_g^T   (rank values)        y_t += s_g (u_i B_g^T)
//
// for each grouped row i, its token t = row[i] and its group (adapter) g.
//
// Bound by memory: x is read once, y read and written; A and B are small and
// come out of L2 for all rows but an adapter's first.  At rank 32 and 4096
// columns there are 170 operations per byte of x and y, a third of what the
// legacy matrix instructions do in that time, and nothing is worth staging: an
// mma.sync fragment is loaded from global memory as it is used.  The order of
// the contraction is free, so lane (g, q) of a warp takes columns 8q..8q+7 of
// rows g, g + 8, ... as one 16-byte load, and the columns of both operands meet
// two by two in the fragments of two instructions.  Likewise the second
// product's columns are dealt out so that a lane ends up with 8 consecutive ones
// of y.  So every access is 16 bytes per lane, 64 consecutive ones per row.
//
// The first kernel takes 32 rows per block; its warps, and several blocks if
// there are few rows, split the columns of x, and the sums are joined in shared
// memory and (blocks) in the second kernel, always in the same order.  The
// second kernel's operand u is split into two 16-bit parts (their sum keeps 16
// bits of bf16, 22 of fp16), after a power of two that brings the largest of a
// row's values near 1, so that fp16 neither overflows nor underflows; sums are
// fp32, and y is rounded once.
//
// 6677 rows with one of 8 adapters of rank 32, 4096 columns: 51 us, 3.3 TB/s; the
// second kernel takes half of it.  64 rows, each with an adapter of its own of
// rank 16: 10 us, most of it two launches.  (There, a block or a cluster of blocks
// per row, without matrix instructions, took 10 to 17 us and for fewer adapters more.)
#include <algorithm>
#include <cstring>

#include "../../include/tilegemm.h"
#include "chained.cuh"
#include "direct.cuh"
#include "grouped.h"

namespace tg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 32;             // per block: two fragments of 16
constexpr int64_t kMaxRank = 128;
constexpr int kRankPass = 64;         // of the rank, per block of the first kernel
constexpr int kStepK = 64;            // columns of x per warp and step
constexpr int kMaxSplits = 16;
// Blocks of the first kernel beyond which splits gain nothing: two on each of a GB300's 152
// SMs.  A constant, since the workspace, whose size follows from it, is asked for without a device.
constexpr int kLowBlocks = 2 * 152;

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
    int splits, split;  // of K, and columns of one (a multiple of kStepK)
    int pitch;          // rank rounded up to 16
    float* low;         // [splits][T][pitch]
    int chunk;          // columns of y per block (a multiple of 256)
};

// u: grid (tiles, splits of K, passes over the rank).  NT fragments of 8 of the rank.
template <bool BF, int NT>
__global__ void __launch_bounds__(kThreads) low_kernel(const AdapterParams p) {
    __shared__ float joined[kWarps / 2][2][NT][4][32];
    allow_next_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const RowTile tile = find_tile<kRows>(p.offset, p.G, p.T, blockIdx.x, lane);
    if (tile.g < 0) return;
    const int r0 = blockIdx.z * kRankPass;
    // rows g, g + 8, g + 16, g + 24 of the tile; what stands in for a row that is not
    // there goes nowhere, and neither does what stands in for one of the rank
    const uint16_t* x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = g + 8 * j;
        const int t = i < tile.rows ? p.row[tile.lo + i] : -1;
        x[j] = p.x + (t >= 0 && t < p.T ? (long long)t * p.ldx : 0) + 8 * q;
    }
    const uint16_t* a[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r0 + 8 * n + g;
        a[n] = p.a + ((long long)tile.g * p.rank + (r < p.rank ? r : 0)) * p.lda + 8 * q;
    }
    float c[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[m][n][j] = 0.0f;
    const int k1 = min(p.K, (int)(blockIdx.y + 1) * p.split);
    auto products = [&](int m, const uint4& x0, const uint4& x1, const uint4 (&av)[NT]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma<BF>(c[m][n], x0.x, x1.x, x0.y, x1.y, av[n].x, av[n].y);
            mma<BF>(c[m][n], x0.z, x1.z, x0.w, x1.w, av[n].z, av[n].w);
        }
    };
    const bool second = tile.rows > 16;  // else its rows 16..31 are none
    for (int k = blockIdx.y * p.split + warp * kStepK; k < k1; k += kWarps * kStepK) {
        uint4 xv[2][4], av[2][NT];
        if (k + kStepK <= k1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[h][j] = *reinterpret_cast<const uint4*>(x[j] + k + 32 * h);
#pragma unroll
                for (int n = 0; n < NT; ++n) av[h][n] = *reinterpret_cast<const uint4*>(a[n] + k + 32 * h);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = k + 32 * h;
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[h][j] = load8(x[j] - 8 * q, at + 8 * q, k1);
#pragma unroll
                for (int n = 0; n < NT; ++n) av[h][n] = load8(a[n] - 8 * q, at + 8 * q, k1);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            products(0, xv[h][0], xv[h][1], av[h]);
            if (second) products(1, xv[h][2], xv[h][3], av[h]);
        }
    }
    // the warps' sums, half of them to the other half, three times
#pragma unroll
    for (int half = kWarps / 2; half; half /= 2) {
        if (warp >= half && warp < 2 * half) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) joined[warp - half][m][n][j][lane] = c[m][n][j];
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[m][n][j] += joined[warp][m][n][j][lane];
        }
        __syncthreads();
    }
    if (warp) return;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * m + 8 * h + g;
            if (i >= tile.rows) continue;
            float* out = p.low + ((long long)blockIdx.y * p.T + tile.lo + i) * p.pitch + r0 + 2 * q;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (r0 + 8 * n < p.pitch) {
                    const int r = r0 + 8 * n + 2 * q;  // (0 from the rank on)
                    *reinterpret_cast<float2*>(out + 8 * n) =
                        make_float2(r < p.rank ? c[m][n][2 * h] : 0.0f, r + 1 < p.rank ? c[m][n][2 * h + 1] : 0.0f);
                }
        }
}

// y: grid (tiles, chunks of N).  KC: fragments of 16 of the rank.  TAIL: the last
// of them is not whole.  Four warps make u's fragments, one for each eight rows;
// they stay in shared memory, so that registers leave room for three blocks on an SM.
template <bool BF, int KC, bool TAIL>
__global__ void __launch_bounds__(kThreads, KC <= 2 ? 3 : 2) add_kernel(const __grid_constant__ AdapterParams p) {
    __shared__ uint4 low[4][KC][32];  // of rows g + 8j, columns 16c + 4q .. + 3: two words each of the large and the small parts
    __shared__ float factors[4][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const RowTile tile = find_tile<kRows>(p.offset, p.G, p.T, blockIdx.x, lane);
    if (tile.g < 0) return;
    uint16_t* y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = g + 8 * j;
        const int t = i < tile.rows ? p.row[tile.lo + i] : -1;
        y[j] = t >= 0 && t < p.T ? p.y + (long long)t * p.ldy : nullptr;
    }
    // y's columns are brought to L2 ahead, the first ones before the wait and each pass's
    // next ones in the loop below, but not for ranks up to 16, whose passes are too short
    // for it.  (30000 rows, us without and with: rank 16 158 and 163, 32 211 and 178,
    // 128 518 and 468.)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = blockIdx.y * p.chunk + warp * 32 + 8 * q;
        if (KC > 1 && y[j] && n < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(y[j] + n));
    }
    wait_for_previous_kernel();
    if (warp < 4) {
        const bool there = g + 8 * warp < tile.rows;
        const float* from = p.low + ((long long)tile.lo + g + 8 * warp) * p.pitch + 4 * q;
        float u[KC][4], top = 0.0f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (there && 16 * c < p.pitch)
                for (int k = 0; k < p.splits; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(from + (long long)k * p.T * p.pitch + 16 * c);
                    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
            u[c][0] = sum.x, u[c][1] = sum.y, u[c][2] = sum.z, u[c][3] = sum.w;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(u[c][k]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with 2^e <= top < 2^(e+1); rows of zeros, or with an infinity, as they are
        float down = 1.0f, factor = p.scale ? p.scale[tile.g] : 1.0f;
        if (top > 0x1p-100f && top < 0x1p100f) {
            const uint32_t e = __float_as_uint(top) & 0x7F800000u;
            down = __uint_as_float(0x7F000000u - e);
            factor *= __uint_as_float(e);
        }
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint32_t part[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float rest[2];
                uint16_t h[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float v = u[c][2 * k + x] * down;
                    h[x] = narrow<BF>(v);
                    rest[x] = v - wide<BF>(h[x]);
                    if (!(fabsf(rest[x]) < 1.0f)) rest[x] = 0.0f;  // of an infinity
                }
                part[k] = (uint32_t)h[0] | (uint32_t)h[1] << 16;
                part[2 + k] = narrow2<BF>(rest[0], rest[1]);
            }
            low[warp][c][lane] = make_uint4(part[0], part[1], part[2], part[3]);
        }
        if (q == 0) factors[warp][g] = factor;
    }
    __syncthreads();
    const bool second = tile.rows > 16;
    const int end = min(p.N, (int)(blockIdx.y + 1) * p.chunk);
    const uint16_t* bg = p.b + (long long)tile.g * p.N * p.ldb + 4 * q;
    // 32 columns of y from n0 on: fragment f's column c is n0 + 8 (c / 2) + 2 f + c % 2,
    // so that this lane's are n0 + 8q .. n0 + 8q + 7
    for (int n0 = blockIdx.y * p.chunk + warp * 32; n0 < end; n0 += kWarps * 32) {
        const int n = n0 + 8 * q;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (KC > 1 && y[j] && n + kWarps * 32 < end) asm volatile("prefetch.global.L2 [%0];" ::"l"(y[j] + n + kWarps * 32));
        uint4 old[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            old[j] = !y[j] ? make_uint4(0, 0, 0, 0) : n + 8 <= p.N ? *reinterpret_cast<const uint4*>(y[j] + n) : load8(y[j], n, p.N);
        uint2 b[4][KC];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            // (a column behind the last goes nowhere)
            const uint16_t* row = bg + (long long)min(p.N - 1, n0 + 8 * (g >> 1) + 2 * f + (g & 1)) * p.ldb;
#pragma unroll
            for (int c = 0; c < KC; ++c)
                b[f][c] = TAIL ? load4(row - 4 * q, 16 * c + 4 * q, p.rank) : *reinterpret_cast<const uint2*>(row + 16 * c);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {  // rows g + 16 m and 8 more
            if (m && !second) break;
            float acc[4][4] = {};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 u0 = low[2 * m][c][lane], u1 = low[2 * m + 1][c][lane];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    mma<BF>(acc[f], u0.z, u1.z, u0.w, u1.w, b[f][c].x, b[f][c].y);
                    mma<BF>(acc[f], u0.x, u1.x, u0.y, u1.y, b[f][c].x, b[f][c].y);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 2 * m + h;
                const float factor = factors[j][g];
                const uint32_t w[4] = {old[j].x, old[j].y, old[j].z, old[j].w};
                uint32_t o[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    o[f] = narrow2<BF>(fmaf(factor, acc[f][2 * h], wide<BF>((uint16_t)(w[f] & 0xFFFFu))),
                                       fmaf(factor, acc[f][2 * h + 1], wide<BF>((uint16_t)(w[f] >> 16))));
                if (!y[j] || n >= p.N) continue;
                if (n + 8 <= p.N) {
                    *reinterpret_cast<uint4*>(y[j] + n) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (n + x < p.N) y[j][n + x] = (uint16_t)(o[x / 2] >> (x & 1) * 16);
                }
            }
        }
    }
}

int64_t tiles_of(int64_t T, int64_t G) { return std::min(T, G) + T / kRows; }

// Splits of K: no more blocks than two on every SM, of at least one step of all
// warps (7777 rows of rank 32, 4096 columns: 68 us with 753 blocks in three splits, 62
// with 251).
int splits_of(int64_t T, int64_t G, int64_t K) {
    const int64_t most = (K + kWarps * kStepK - 1) / (kWarps * kStepK);
    const int64_t wanted = kLowBlocks / tiles_of(T, G);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(most, wanted), kMaxSplits));
}
int64_t pitch_of(int64_t rank) { return (rank + 15) / 16 * 16; }

template <bool BF>
cudaError_t launch_low(const AdapterParams& p, dim3 grid, cudaStream_t stream) {
    if (p.rank <= 16)
        low_kernel<BF, 2><<<grid, kThreads, 0, stream>>>(p);
    else if (p.rank <= 32)
        low_kernel<BF, 4><<<grid, kThreads, 0, stream>>>(p);
    else
        low_kernel<BF, 8><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}
template <bool BF>
cudaError_t launch_add(const AdapterParams& p, dim3 grid, cudaStream_t stream) {
    // (fragments that the rank does not reach have no elements of B)
    const bool whole = p.rank == 16 || p.rank == 32 || p.rank == 64 || p.rank == 128;
    auto pick = [&](auto full, auto tail) { return launch_chained(whole ? full : tail, grid, kThreads, stream, p); };
    if (p.rank <= 16) return pick(add_kernel<BF, 1, false>, add_kernel<BF, 1, true>);
    if (p.rank <= 32) return pick(add_kernel<BF, 2, false>, add_kernel<BF, 2, true>);
    if (p.rank <= 64) return pick(add_kernel<BF, 4, false>, add_kernel<BF, 4, true>);
    return pick(add_kernel<BF, 8, false>, add_kernel<BF, 8, true>);
}

int check_sizes(int64_t T, int64_t N, int64_t K, int64_t rank, int64_t G, int dtype) {
    if (T <= 0 || N <= 0 || K <= 0 || rank <= 0 || G <= 0 || T > kMaxSize || N > kMaxSize || K > kMaxSize ||
        rank > kMaxRank || G > kMaxRowGroups)
        return TG_ERR_INVALID_ARG;
    if (dtype != TG_F16 && dtype != TG_BF16) return TG_ERR_DTYPE;
    return TG_OK;
}

size_t workspace_of(int64_t T, int64_t G, int64_t K, int64_t rank) {
    return (size_t)T * (size_t)splits_of(T, G, K) * (size_t)pitch_of(rank) * sizeof(float);
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_adapters_workspace_size(int64_t T, int64_t N, int64_t K, int64_t rank, int64_t G, tg_dtype dtype,
                                          size_t* bytes) {
    const int rc = check_sizes(T, N, K, rank, G, (int)dtype);
    if (rc) return rc;
    if (!bytes) return TG_ERR_INVALID_ARG;
    *bytes = workspace_of(T, G, K, rank);
    return TG_OK;
}

extern "C" int tg_adapters(int64_t T, int64_t N, int64_t K, int64_t rank, int64_t G, const void* X, int64_t ldx,
                           const int32_t* row, const int32_t* offset, const void* A, int64_t lda, const void* B,
                           int64_t ldb, const float* scale, void* Y, int64_t ldy, tg_dtype dtype, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    int rc = check_sizes(T, N, K, rank, G, (int)dtype);
    if (rc) return rc;
    if (!X || !row || !offset || !A || !B || !Y || !workspace) return TG_ERR_INVALID_ARG;
    const size_t need = workspace_of(T, G, K, rank);
    if (ldx < K || lda < K || ldb < rank || ldy < N || ldx > kMaxLd || lda > kMaxLd || ldb > kMaxLd || ldy > kMaxLd)
        return TG_ERR_STRIDE;
    auto off = [](const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; };
    if (!aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(Y) || ldx % 8 || lda % 8 || ldb % 8 || ldy % 8 ||
        off(row, 4) || off(offset, 4) || off(scale, 4) || off(workspace, 256))
        return TG_ERR_ALIGN;
    if (workspace_bytes < need) return TG_ERR_BUFFER;
    // (G * rank rows of A and G * N of B, one after another)
    const void* ptrs[8] = {Y, workspace, X, A, B, row, offset, scale};
    const Span spans[8] = {span_of(Y, T, N, ldy), span_bytes(workspace, need), span_of(X, T, K, ldx),
                           span_of(A, G * rank, K, lda), span_of(B, G * N, rank, ldb), span_bytes(row, (u128)T * 4),
                           span_bytes(offset, (u128)(G + 1) * 4), span_bytes(scale, (u128)G * 4)};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 8; ++j)
            if (intersects(spans[i], spans[j])) return TG_ERR_OVERLAP;
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
    p.splits = splits_of(T, G, K);
    p.split = (int)((K + (int64_t)p.splits * kStepK - 1) / ((int64_t)p.splits * kStepK) * kStepK);
    p.splits = (int)((K + p.split - 1) / p.split);
    p.pitch = (int)pitch_of(rank);
    p.low = static_cast<float*>(workspace);
    // Columns of y per block: few enough for three blocks per SM, at most 1024, or 2048
    // where u's fragments are many (7777 rows, us, 1024 to 2048: rank 32 62 to 70, rank 64 93 to 89).
    const int64_t most = rank <= 32 ? 1024 : 2048;
    const int64_t tiles = tiles_of(T, G);
    int64_t chunks = std::max<int64_t>((N + most - 1) / most, std::min<int64_t>((N + 255) / 256, (3LL * info->sms + tiles - 1) / tiles));
    chunks = std::min<int64_t>(chunks, 65535);
    p.chunk = (int)((N + chunks * 256 - 1) / (chunks * 256) * 256);
    chunks = (N + p.chunk - 1) / p.chunk;
    const dim3 low((unsigned)tiles, (unsigned)p.splits, (unsigned)((rank + kRankPass - 1) / kRankPass));
    const dim3 add((unsigned)tiles, (unsigned)chunks, 1);
    cudaError_t e = dtype == TG_BF16 ? launch_low<true>(p, low, stream) : launch_low<false>(p, low, stream);
    if (e == cudaSuccess) e = dtype == TG_BF16 ? launch_add<true>(p, add, stream) : launch_add<false>(p, add, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
