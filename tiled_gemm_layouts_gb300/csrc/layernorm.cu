// layernorm.cu -- layer norm and its gradient (tg_layernorm,
// tg_layernorm_grad).
//
//   xh = (x - mean) rstd      y = xh w + b
//   g = dy w;  dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh;  db = sum over rows of dy
//
// Both are bound by memory: every element is read once and written once.  A
// row stays in registers between its two reductions (mean, then squared
// differences from it: no cancellation), held by one warp up to 1024 columns
// and by a block beyond.  The gradient's blocks walk over rows and keep their
// columns' dw and db in fp32 registers; one partial row per block goes to the
// workspace and a second kernel adds them in a fixed order, so results repeat
// bit for bit.  Statistics and sums are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <initializer_list>

#include "../../include/tilegemm.h"
#include "host_common.h"

namespace tg {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool BF>
__device__ __forceinline__ float widen(uint16_t h) {
    return BF ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}
template <bool BF>
__device__ __forceinline__ uint16_t narrow(float x) {
    return BF ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// VEC consecutive 16-bit elements, moved with one access.
template <int VEC>
struct Pack {
    uint16_t e[VEC];
};
template <>
struct alignas(16) Pack<8> {
    uint16_t e[8];
};
template <>
struct alignas(4) Pack<2> {
    uint16_t e[2];
};

template <int VEC>
__device__ __forceinline__ Pack<VEC> load(const uint16_t* p) {
    Pack<VEC> v;
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4*>(&v) = __ldg(reinterpret_cast<const uint4*>(p));
    else if constexpr (VEC == 2)
        *reinterpret_cast<uint32_t*>(&v) = __ldg(reinterpret_cast<const uint32_t*>(p));
    else
        v.e[0] = __ldg(p);
    return v;
}

// Sums of N values over the WARPS warps that share a row; every thread gets
// them.  `buf` has room for N * WARPS floats and alternates between calls, so
// one barrier per call is enough.
template <int N, int WARPS>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (WARPS > 1) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) buf[k * WARPS + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float x = lane < WARPS ? buf[k * WARPS + lane] : 0.0f;
#pragma unroll
            for (int o = WARPS / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            v[k] = __shfl_sync(0xffffffffu, x, 0);
        }
    }
}

struct LnParams {
    long long rows;
    int cols;
    const uint16_t *x, *dy;
    long long ldx, lddy;
    const uint16_t *weight, *bias;
    float eps;
    uint16_t* out;  // y, or dx
    long long ldo;
    float *mean, *rstd;
    float* part;  // gradient: [blocks][2][cols]
};

// WARPS warps per row, NV packs of VEC elements per thread.  Rows wider than
// that (WIDE) are read again from memory, which finds most of them in L2.
constexpr int kRowsPerBlock = 4;  // rows of a block whose rows take one warp each

template <bool BF, int VEC, int WARPS, int NV, bool WIDE>
__global__ void __launch_bounds__(WARPS == 1 ? 32 * kRowsPerBlock : 32 * WARPS)
ln_forward_kernel(const LnParams p) {
    __shared__ float buf[2][WARPS == 1 ? 1 : WARPS];
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    constexpr int kThreads = 32 * WARPS, kStep = kThreads * VEC;
    const long long row = WARPS == 1 ? (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5)
                                     : (long long)blockIdx.x;
    if (row >= p.rows) return;
    const uint16_t* x = p.x + row * p.ldx;
    uint16_t* y = p.out + row * p.ldo;
    const int chunks = WIDE ? (p.cols + kStep * NV - 1) / (kStep * NV) : 1;
    Pack<VEC> v[NV];
    auto fetch = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (chunk * NV + i) * kStep + tid * VEC;
            if (c < p.cols) v[i] = load<VEC>(x + c);
        }
    };
    float sum[1] = {0.0f};
    for (int k = 0; k < chunks; ++k) {
        fetch(k);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((k * NV + i) * kStep + tid * VEC < p.cols)
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[0] += widen<BF>(v[i].e[j]);
    }
    row_sum<1, WARPS>(sum, buf[0]);
    const float mean = sum[0] / (float)p.cols;
    float sq[1] = {0.0f};
    for (int k = 0; k < chunks; ++k) {
        if (WIDE) fetch(k);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((k * NV + i) * kStep + tid * VEC < p.cols)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = widen<BF>(v[i].e[j]) - mean;
                    sq[0] = fmaf(d, d, sq[0]);
                }
    }
    row_sum<1, WARPS>(sq, buf[1]);
    const float rstd = 1.0f / sqrtf(sq[0] / (float)p.cols + p.eps);
    if (tid == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
    }
    for (int k = 0; k < chunks; ++k) {
        if (WIDE) fetch(k);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (k * NV + i) * kStep + tid * VEC;
            if (c >= p.cols) continue;
            const Pack<VEC> w = load<VEC>(p.weight + c);
            Pack<VEC> b = {}, o;
            if (p.bias) b = load<VEC>(p.bias + c);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xh = (widen<BF>(v[i].e[j]) - mean) * rstd;
                o.e[j] = narrow<BF>(fmaf(xh, widen<BF>(w.e[j]), widen<BF>(b.e[j])));
            }
            *reinterpret_cast<Pack<VEC>*>(y + c) = o;
        }
    }
}

// dx, and this block's partial sums of dw and db.
template <bool BF, int VEC, int WARPS, int NV>
__global__ void __launch_bounds__(WARPS == 1 ? 32 * kRowsPerBlock : 32 * WARPS)
ln_backward_kernel(const LnParams p) {
    constexpr int kThreads = 32 * WARPS, kStep = kThreads * VEC;
    constexpr int kGroups = WARPS == 1 ? kRowsPerBlock : 1;  // rows in work at once
    __shared__ float buf[2][WARPS == 1 ? 1 : 2 * WARPS];
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int group = WARPS == 1 ? threadIdx.x >> 5 : 0;
    float dw[NV][VEC], db[NV][VEC];
    Pack<VEC> w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kStep + tid * VEC;
        w[i] = Pack<VEC>{};
        if (c < p.cols) w[i] = load<VEC>(p.weight + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
    }
    const float inv = 1.0f / (float)p.cols;
    int flip = 0;
    for (long long row = (long long)blockIdx.x * kGroups + group; row < p.rows;
         row += (long long)gridDim.x * kGroups) {
        const uint16_t* x = p.x + row * p.ldx;
        const uint16_t* dy = p.dy + row * p.lddy;
        Pack<VEC> vx[NV], vd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * kStep + tid * VEC;
            if (c < p.cols) {
                vx[i] = load<VEC>(x + c);
                vd[i] = load<VEC>(dy + c);
            }
        }
        const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
        float s[2] = {0.0f, 0.0f};  // sums of g and of g xh
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * kStep + tid * VEC < p.cols)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xh = (widen<BF>(vx[i].e[j]) - mean) * rstd;
                    const float d = widen<BF>(vd[i].e[j]), g = d * widen<BF>(w[i].e[j]);
                    s[0] += g;
                    s[1] = fmaf(g, xh, s[1]);
                    dw[i][j] = fmaf(d, xh, dw[i][j]);
                    db[i][j] += d;
                }
        row_sum<2, WARPS>(s, buf[flip]);
        flip ^= 1;
        const float c1 = s[0] * inv, c2 = s[1] * inv;
        uint16_t* dx = p.out + row * p.ldo;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * kStep + tid * VEC;
            if (c >= p.cols) continue;
            Pack<VEC> o;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xh = (widen<BF>(vx[i].e[j]) - mean) * rstd;
                const float g = widen<BF>(vd[i].e[j]) * widen<BF>(w[i].e[j]);
                o.e[j] = narrow<BF>(rstd * (g - c1 - xh * c2));
            }
            *reinterpret_cast<Pack<VEC>*>(dx + c) = o;
        }
    }
    // one partial row per row group: [block * kGroups + group][2][cols]
    float* part = p.part + ((long long)blockIdx.x * kGroups + group) * 2 * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kStep + tid * VEC;
        if (c < p.cols)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                part[c + j] = dw[i][j];
                part[p.cols + c + j] = db[i][j];
            }
    }
}

// Rows too wide for registers: dx alone, one block per row.
template <bool BF>
__global__ void __launch_bounds__(1024) ln_backward_wide_kernel(const LnParams p) {
    __shared__ float buf[2 * 32];
    const long long row = blockIdx.x;
    const uint16_t* x = p.x + row * p.ldx;
    const uint16_t* dy = p.dy + row * p.lddy;
    uint16_t* dx = p.out + row * p.ldo;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
        const float xh = (widen<BF>(x[c]) - mean) * rstd, g = widen<BF>(dy[c]) * widen<BF>(p.weight[c]);
        s[0] += g;
        s[1] = fmaf(g, xh, s[1]);
    }
    row_sum<2, 32>(s, buf);
    const float c1 = s[0] / (float)p.cols, c2 = s[1] / (float)p.cols;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
        const float xh = (widen<BF>(x[c]) - mean) * rstd, g = widen<BF>(dy[c]) * widen<BF>(p.weight[c]);
        dx[c] = narrow<BF>(rstd * (g - c1 - xh * c2));
    }
}

// Their partial dw and db: block (column group, row group), thread = column.
template <bool BF>
__global__ void __launch_bounds__(256) ln_backward_wide_columns_kernel(const LnParams p) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float d = widen<BF>(p.dy[row * p.lddy + c]);
        const float xh = (widen<BF>(p.x[row * p.ldx + c]) - p.mean[row]) * p.rstd[row];
        dw = fmaf(d, xh, dw);
        db += d;
    }
    float* part = p.part + (long long)blockIdx.y * 2 * p.cols;
    part[c] = dw;
    part[p.cols + c] = db;
}

// Adds the partial rows: 32 columns per block, 32 threads along the rows of
// each, then across those in a fixed order.
template <bool BF>
__global__ void __launch_bounds__(1024)
ln_reduce_kernel(const float* __restrict__ part, int parts, int cols, uint16_t* __restrict__ dw,
                 uint16_t* __restrict__ db) {
    __shared__ float s[2][32][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.0f, b = 0.0f;
    if (c < cols)
#pragma unroll 4
        for (int r = y; r < parts; r += 32) {
            a += part[(long long)r * 2 * cols + c];
            b += part[((long long)r * 2 + 1) * cols + c];
        }
    s[0][y][lane] = a;
    s[1][y][lane] = b;
    __syncthreads();
    a = s[0][lane][y];
    b = s[1][lane][y];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    const int out = blockIdx.x * 32 + y;
    if (lane == 0 && out < cols) {
        dw[out] = narrow<BF>(a);
        if (db) db[out] = narrow<BF>(b);
    }
}

// Widest pack that every row, weight and output allows: whole packs per row
// and aligned row starts.
int pack_of(int64_t cols, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
    for (int vec : {8, 2}) {
        bool ok = cols % vec == 0;
        for (const void* q : ptrs) ok = ok && (reinterpret_cast<uintptr_t>(q) % (2 * vec)) == 0;
        for (int64_t ld : lds) ok = ok && ld % vec == 0;
        if (ok) return vec;
    }
    return 1;
}

// Calls f with the row shape (warps per row, packs per thread) for `cols`;
// packs in registers up to the last one's width.
#define TG_LN_SHAPES(F, VEC)          \
    if (cols <= 32 * 1 * VEC) F(1, 1) \
    if (cols <= 32 * 2 * VEC) F(1, 2) \
    if (cols <= 32 * 4 * VEC) F(1, 4) \
    if (cols <= 128 * 2 * VEC) F(4, 2) \
    if (cols <= 128 * 4 * VEC) F(4, 4) \
    if (cols <= 256 * 4 * VEC) F(8, 4) \
    if (cols <= 512 * 4 * VEC) F(16, 4)
// Narrow packs (rows of odd addresses): more of them per thread.
#define TG_LN_NARROW_SHAPES(F, VEC)   \
    if (cols <= 32 * 4 * VEC) F(1, 4) \
    if (cols <= 32 * 8 * VEC) F(1, 8) \
    if (cols <= 128 * 8 * VEC) F(4, 8) \
    if (cols <= 256 * 8 * VEC) F(8, 8) \
    if (cols <= 512 * 8 * VEC) F(16, 8) \
    if (cols <= 1024 * 8 * VEC) F(32, 8)

template <bool BF>
cudaError_t launch_forward(const LnParams& p, int vec, cudaStream_t stream) {
    const int cols = p.cols;
#define TG_LAUNCH(WARPS, NV, VEC, WIDE)                                                            \
    {                                                                                              \
        const long long blocks = WARPS == 1 ? cdiv(p.rows, kRowsPerBlock) : p.rows;                \
        ln_forward_kernel<BF, VEC, WARPS, NV, WIDE>                                                \
            <<<(unsigned)blocks, WARPS == 1 ? 32 * kRowsPerBlock : 32 * WARPS, 0, stream>>>(p);    \
        return cudaGetLastError();                                                                 \
    }
#define TG_F8(WARPS, NV) TG_LAUNCH(WARPS, NV, 8, false)
#define TG_F2(WARPS, NV) TG_LAUNCH(WARPS, NV, 2, false)
#define TG_F1(WARPS, NV) TG_LAUNCH(WARPS, NV, 1, false)
    if (vec == 8) {
        TG_LN_SHAPES(TG_F8, 8)
        TG_LAUNCH(16, 4, 8, true)
    }
    if (vec == 2) {
        TG_LN_NARROW_SHAPES(TG_F2, 2)
        TG_LAUNCH(32, 8, 2, true)
    }
    TG_LN_NARROW_SHAPES(TG_F1, 1)
    TG_LAUNCH(32, 8, 1, true)
#undef TG_F8
#undef TG_F2
#undef TG_F1
#undef TG_LAUNCH
}

// Partial rows of dw and db for a row shape: enough blocks to fill the GPU.
struct GradShape {
    int warps, packs, vec;  // warps 0: the wide kernels
    int blocks, parts;
};

GradShape grad_shape(int64_t rows, int64_t cols, int vec, int sms) {
    GradShape s{0, 0, vec, 0, 0};
#define TG_SET(WARPS, NV)                  \
    {                                      \
        if (!s.warps) s.warps = WARPS, s.packs = NV; \
    }
    if (vec == 8) {
        TG_LN_SHAPES(TG_SET, 8)
    } else if (vec == 2) {
        TG_LN_NARROW_SHAPES(TG_SET, 2)
    } else {
        TG_LN_NARROW_SHAPES(TG_SET, 1)
    }
#undef TG_SET
    const int groups = s.warps == 1 ? kRowsPerBlock : 1;
    const int threads = s.warps == 1 ? 32 * kRowsPerBlock : 32 * s.warps;
    int64_t most;
    if (s.warps) {
        most = (int64_t)sms * (threads >= 1024 ? 1 : threads >= 512 ? 1 : threads >= 256 ? 2 : 4);
        const int64_t need = cdiv(rows, groups);
        s.blocks = (int)(need < most ? need : most);
        s.parts = s.blocks * groups;
    } else {
        s.blocks = s.parts = (int)(rows < 64 ? rows : 64);
    }
    return s;
}

template <bool BF>
cudaError_t launch_backward(const LnParams& p, const GradShape& s, cudaStream_t stream) {
#define TG_LAUNCH(WARPS, NV, VEC)                                                                     \
    if (s.warps == WARPS && s.packs == NV) {                                                          \
        ln_backward_kernel<BF, VEC, WARPS, NV>                                                        \
            <<<s.blocks, WARPS == 1 ? 32 * kRowsPerBlock : 32 * WARPS, 0, stream>>>(p);               \
        return cudaGetLastError();                                                                    \
    }
    if (s.warps == 0) {
        ln_backward_wide_kernel<BF><<<(unsigned)p.rows, 1024, 0, stream>>>(p);
        ln_backward_wide_columns_kernel<BF>
            <<<dim3((unsigned)cdiv(p.cols, 256), s.blocks), 256, 0, stream>>>(p);
        return cudaGetLastError();
    }
    if (s.vec == 8) {
        TG_LAUNCH(1, 1, 8) TG_LAUNCH(1, 2, 8) TG_LAUNCH(1, 4, 8) TG_LAUNCH(4, 2, 8)
        TG_LAUNCH(4, 4, 8) TG_LAUNCH(8, 4, 8) TG_LAUNCH(16, 4, 8)
    } else if (s.vec == 2) {
        TG_LAUNCH(1, 4, 2) TG_LAUNCH(1, 8, 2) TG_LAUNCH(4, 8, 2) TG_LAUNCH(8, 8, 2)
        TG_LAUNCH(16, 8, 2) TG_LAUNCH(32, 8, 2)
    } else {
        TG_LAUNCH(1, 4, 1) TG_LAUNCH(1, 8, 1) TG_LAUNCH(4, 8, 1) TG_LAUNCH(8, 8, 1)
        TG_LAUNCH(16, 8, 1) TG_LAUNCH(32, 8, 1)
    }
#undef TG_LAUNCH
    return cudaErrorInvalidValue;
}

int check_sizes(int64_t rows, int64_t cols, int dtype) {
    if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim) return TG_ERR_INVALID_ARG;
    if (dtype != TG_F16 && dtype != TG_BF16) return TG_ERR_DTYPE;
    return TG_OK;
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_layernorm(int64_t rows, int64_t cols, const void* X, int64_t ldx,
                            const void* weight, const void* bias, float eps, void* Y, int64_t ldy,
                            float* mean, float* rstd, tg_dtype dtype, cudaStream_t stream) {
    int rc = check_sizes(rows, cols, (int)dtype);
    if (rc) return rc;
    if (!X || !weight || !Y || !mean || !rstd || !(eps >= 0.0f)) return TG_ERR_INVALID_ARG;
    if (ldx < cols || ldy < cols || ldx > kMaxLd || ldy > kMaxLd) return TG_ERR_STRIDE;
    if (off(X, 2) || off(weight, 2) || off(bias, 2) || off(Y, 2) || off(mean, 4) || off(rstd, 4))
        return TG_ERR_ALIGN;
    const Span spans[6] = {span_of(Y, rows, cols, ldy), span_bytes(mean, (u128)rows * 4),
                           span_bytes(rstd, (u128)rows * 4), span_of(X, rows, cols, ldx),
                           span_of(weight, 1, cols, cols), span_of(bias, 1, cols, cols)};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (intersects(spans[i], spans[j])) return TG_ERR_OVERLAP;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();  // the allocation-range query of check_pointer
    const void* ptrs[6] = {Y, mean, rstd, X, weight, bias};
    for (int i = 0; i < 6; ++i)
        if ((rc = check_pointer(ptrs[i], spans[i], dev))) return rc;
    LnParams p;
    std::memset(&p, 0, sizeof(p));
    p.rows = rows;
    p.cols = (int)cols;
    p.x = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.weight = static_cast<const uint16_t*>(weight);
    p.bias = static_cast<const uint16_t*>(bias);
    p.eps = eps;
    p.out = static_cast<uint16_t*>(Y);
    p.ldo = ldy;
    p.mean = mean;
    p.rstd = rstd;
    const int vec = pack_of(cols, {X, weight, bias, Y}, {ldx, ldy});
    if ((dtype == TG_BF16 ? launch_forward<true>(p, vec, stream)
                          : launch_forward<false>(p, vec, stream)) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}

// The workspace holds the partial rows of the shape with the most of them.
extern "C" int tg_layernorm_grad_workspace_size(int64_t rows, int64_t cols, tg_dtype dtype,
                                                size_t* bytes) {
    int rc = check_sizes(rows, cols, (int)dtype);
    if (rc) return rc;
    if (!bytes) return TG_ERR_INVALID_ARG;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    int64_t parts = 0;
    for (int vec : {8, 2, 1}) {
        const GradShape s = grad_shape(rows, cols, vec, info->sms);
        if (s.parts > parts) parts = s.parts;
    }
    *bytes = (size_t)parts * 2 * (size_t)cols * sizeof(float);
    return TG_OK;
}

extern "C" int tg_layernorm_grad(int64_t rows, int64_t cols, const void* dY, int64_t lddy,
                                 const void* X, int64_t ldx, const void* weight, const float* mean,
                                 const float* rstd, void* dX, int64_t lddx, void* dweight,
                                 void* dbias, tg_dtype dtype, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    int rc = check_sizes(rows, cols, (int)dtype);
    if (rc) return rc;
    if (!dY || !X || !weight || !mean || !rstd || !dX || !dweight || !workspace)
        return TG_ERR_INVALID_ARG;
    if (lddy < cols || ldx < cols || lddx < cols || lddy > kMaxLd || ldx > kMaxLd || lddx > kMaxLd)
        return TG_ERR_STRIDE;
    if (off(dY, 2) || off(X, 2) || off(weight, 2) || off(dX, 2) || off(dweight, 2) || off(dbias, 2) ||
        off(mean, 4) || off(rstd, 4) || off(workspace, 256))
        return TG_ERR_ALIGN;
    int dev;
    DeviceInfo* info;
    const Span outs[3] = {span_of(dX, rows, cols, lddx), span_of(dweight, 1, cols, cols),
                          span_of(dbias, 1, cols, cols)};
    const Span ins[5] = {span_of(dY, rows, cols, lddy), span_of(X, rows, cols, ldx),
                         span_of(weight, 1, cols, cols), span_bytes(mean, (u128)rows * 4),
                         span_bytes(rstd, (u128)rows * 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (intersects(outs[i], outs[j])) return TG_ERR_OVERLAP;
        for (const Span& s : ins)
            if (intersects(outs[i], s)) return TG_ERR_OVERLAP;
    }
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();
    const int vec = pack_of(cols, {dY, X, weight, dX}, {lddy, ldx, lddx});
    const GradShape s = grad_shape(rows, cols, vec, info->sms);
    const size_t need = (size_t)s.parts * 2 * (size_t)cols * sizeof(float);
    if (workspace_bytes < need) return TG_ERR_BUFFER;
    const Span work = span_bytes(workspace, need);
    for (const Span& o : outs)
        if (intersects(work, o)) return TG_ERR_OVERLAP;
    for (const Span& o : ins)
        if (intersects(work, o)) return TG_ERR_OVERLAP;
    const void* outp[3] = {dX, dweight, dbias};
    const void* inp[5] = {dY, X, weight, mean, rstd};
    for (int i = 0; i < 3; ++i)
        if ((rc = check_pointer(outp[i], outs[i], dev))) return rc;
    for (int i = 0; i < 5; ++i)
        if ((rc = check_pointer(inp[i], ins[i], dev))) return rc;
    if ((rc = check_pointer(workspace, work, dev))) return rc;
    LnParams p;
    std::memset(&p, 0, sizeof(p));
    p.rows = rows;
    p.cols = (int)cols;
    p.x = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.dy = static_cast<const uint16_t*>(dY);
    p.lddy = lddy;
    p.weight = static_cast<const uint16_t*>(weight);
    p.out = static_cast<uint16_t*>(dX);
    p.ldo = lddx;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.part = static_cast<float*>(workspace);
    cudaError_t e = dtype == TG_BF16 ? launch_backward<true>(p, s, stream)
                                     : launch_backward<false>(p, s, stream);
    if (e == cudaSuccess) {
        auto reduce = dtype == TG_BF16 ? ln_reduce_kernel<true> : ln_reduce_kernel<false>;
        reduce<<<(unsigned)cdiv(cols, 32), 1024, 0, stream>>>(p.part, s.parts, p.cols,
                                                              static_cast<uint16_t*>(dweight),
                                                              static_cast<uint16_t*>(dbias));
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
