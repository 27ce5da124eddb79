// combine.cu -- the weighted sum of the rows that belong to a token
// (tg_combine) and its gradient (tg_combine_grad).
//
//   out_t = sum_j w_tj Y[place_tj]
//   dY[place_tj] = w_tj dout_t        dw_tj = dout_t . Y[place_tj]
//
// Bound by memory: every row of Y is read once (and one of dY written), out or
// dout once.  The sum: a thread owns 8 columns of a token (16 bytes), loads
// them from up to 8 of its rows before it adds any, and a block's threads
// cover neighbouring columns.  The gradient: a warp per (token, j), the j of a
// token in one block, so that dout comes out of L1 for all but the first; the
// dot product is summed in fp32 by lane and joined by the warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <initializer_list>

#include "../../include/tilegemm.h"
#include "host_common.h"
#include "packed.cuh"

namespace tg {
namespace {

constexpr int kSumThreads = 256;
constexpr int kGradWarps = 8;
constexpr int64_t kMaxRows = 1024;  // of one token

struct CombineParams {
    long long T;
    int k;
    long long D, y_rows;
    const uint16_t* y;
    long long ldy;
    const int* place;
    const float* weight;
    uint16_t* out;  // combine: [T]; gradient: dY
    long long ldo;
    const uint16_t* dout;
    long long lddo;
    float* dweight;
    unsigned units;  // of VEC columns per row
    bool narrow;     // fewer than 2^32 of them in all
};

template <bool BF>
__device__ __forceinline__ float2 wide2(uint32_t w) {
    if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
}
template <bool BF>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// VEC columns of 16 bits as VEC / 2 words (one word, its upper half 0, for 1)
template <int VEC>
struct Unit {
    uint32_t w[VEC == 8 ? 4 : 1];
};
template <int VEC>
__device__ __forceinline__ Unit<VEC> load_unit(const uint16_t* p) {
    Unit<VEC> u;
    if constexpr (VEC == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        u.w[0] = v.x, u.w[1] = v.y, u.w[2] = v.z, u.w[3] = v.w;
    } else {
        u.w[0] = *p;
    }
    return u;
}
template <int VEC>
__device__ __forceinline__ void store_unit(uint16_t* p, const Unit<VEC>& u) {
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
    else
        *p = (uint16_t)u.w[0];
}

template <bool BF, int VEC>
__global__ void __launch_bounds__(kSumThreads) combine_kernel(const CombineParams p) {
    constexpr int W = VEC == 8 ? 4 : 1;
    const long long u = (long long)blockIdx.x * kSumThreads + threadIdx.x;
    // (most often in 32 bits: a 64-bit division takes as long as the rest)
    const long long t = p.narrow ? (long long)((unsigned)u / p.units) : u / p.units;
    if (t >= p.T) return;
    const long long c = (u - t * p.units) * VEC;
    const int* place = p.place + t * p.k;
    const float* weight = p.weight ? p.weight + t * p.k : nullptr;
    f2 sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = pair(0.0f, 0.0f);
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        Unit<VEC> v[8];
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = 0.0f;
            int at = -1;
            if (j0 + j < p.k) at = place[j0 + j];
            const bool there = at >= 0 && at < p.y_rows;
            if (there) {
                w[j] = weight ? weight[j0 + j] : 1.0f;
                v[j] = load_unit<VEC>(p.y + at * p.ldy + c);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v[j].w[i] = 0;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 x = wide2<BF>(v[j].w[i]);
                sum[i] = fma(pair(x.x, x.y), pair(w[j], w[j]), sum[i]);
            }
    }
    Unit<VEC> o;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float2 x = split(sum[i]);
        o.w[i] = narrow2<BF>(x.x, x.y);
    }
    store_unit<VEC>(p.out + t * p.ldo + c, o);
}

template <bool BF, int VEC>
__global__ void __launch_bounds__(32 * kGradWarps) combine_grad_kernel(const CombineParams p) {
    constexpr int W = VEC == 8 ? 4 : 1;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    if (item >= p.T * p.k) return;
    const long long t = (unsigned)item / (unsigned)p.k;  // (T k < 2^31)
    const int at = p.place[item];
    if (at < 0 || at >= p.y_rows) {
        if (p.dweight && lane == 0) p.dweight[item] = 0.0f;
        return;
    }
    const float w = p.weight ? p.weight[item] : 1.0f;
    const uint16_t* dout = p.dout + t * p.lddo;
    const uint16_t* y = p.y + at * p.ldy;
    uint16_t* dy = p.out + at * p.ldo;
    f2 dot = pair(0.0f, 0.0f);
#pragma unroll 4
    for (unsigned u = lane; u < p.units; u += 32) {
        const Unit<VEC> g = load_unit<VEC>(dout + (long long)u * VEC);
        Unit<VEC> x, o;
        if (p.dweight) x = load_unit<VEC>(y + (long long)u * VEC);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 gg = wide2<BF>(g.w[i]);
            if (p.dweight) {
                const float2 yy = wide2<BF>(x.w[i]);
                dot = fma(pair(gg.x, gg.y), pair(yy.x, yy.y), dot);
            }
            o.w[i] = narrow2<BF>(gg.x * w, gg.y * w);
        }
        if (p.out) store_unit<VEC>(dy + (long long)u * VEC, o);
    }
    if (!p.dweight) return;
    const float2 both = split(dot);
    float sum = both.x + both.y;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) p.dweight[item] = sum;
}

// 16-byte units where every row starts on one and is a whole number of them
int columns_per_unit(int64_t D, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
    bool whole = D % 8 == 0;
    for (const void* q : ptrs) whole = whole && aligned16(q);
    for (int64_t ld : lds) whole = whole && ld % 8 == 0;
    return whole ? 8 : 1;
}

int check_sizes(int64_t T, int64_t k, int64_t D, int64_t y_rows, int dtype) {
    if (T <= 0 || k <= 0 || D <= 0 || y_rows <= 0 || T > kMaxSize || k > kMaxRows || D > kMaxSize || y_rows > kMaxDim ||
        T * k > kMaxDim)
        return TG_ERR_INVALID_ARG;
    if (dtype != TG_F16 && dtype != TG_BF16) return TG_ERR_DTYPE;
    return TG_OK;
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
bool bad_ld(int64_t ld, int64_t D) { return ld < D || ld > kMaxLd; }

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_combine(int64_t T, int64_t k, int64_t D, const void* Y, int64_t y_rows, int64_t ldy,
                          const int32_t* place, const float* weight, void* out, int64_t ldo, tg_dtype dtype,
                          cudaStream_t stream) {
    int rc = check_sizes(T, k, D, y_rows, (int)dtype);
    if (rc) return rc;
    if (!Y || !place || !out) return TG_ERR_INVALID_ARG;
    if (bad_ld(ldy, D) || bad_ld(ldo, D)) return TG_ERR_STRIDE;
    if (off(Y, 2) || off(out, 2) || off(place, 4) || off(weight, 4)) return TG_ERR_ALIGN;
    const void* ptrs[4] = {out, Y, place, weight};
    const Span spans[4] = {span_of(out, T, D, ldo), span_of(Y, y_rows, D, ldy), span_bytes(place, (u128)T * k * 4),
                           span_bytes(weight, (u128)T * k * 4)};
    for (int j = 1; j < 4; ++j)
        if (intersects(spans[0], spans[j])) return TG_ERR_OVERLAP;
    CombineParams p = {};
    const int vec = columns_per_unit(D, {Y, out}, {ldy, ldo});
    p.units = (unsigned)(D / vec);
    const int64_t blocks = (T * (int64_t)p.units + kSumThreads - 1) / kSumThreads;
    if (blocks > kMaxDim) return TG_ERR_INVALID_ARG;
    p.narrow = blocks < (1LL << 32) / kSumThreads;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();  // the allocation-range query of check_pointer
    PointerChecks check{dev};
    for (int i = 0; i < 4; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    p.T = T;
    p.k = (int)k;
    p.D = D;
    p.y_rows = y_rows;
    p.y = static_cast<const uint16_t*>(Y);
    p.ldy = ldy;
    p.place = place;
    p.weight = weight;
    p.out = static_cast<uint16_t*>(out);
    p.ldo = ldo;
    auto kern = dtype == TG_BF16 ? (vec == 8 ? combine_kernel<true, 8> : combine_kernel<true, 1>)
                                 : (vec == 8 ? combine_kernel<false, 8> : combine_kernel<false, 1>);
    kern<<<(unsigned)blocks, kSumThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return TG_ERR_CUDA;
    return TG_OK;
}

extern "C" int tg_combine_grad(int64_t T, int64_t k, int64_t D, const void* dout, int64_t lddo, const void* Y,
                               int64_t y_rows, int64_t ldy, const int32_t* place, const float* weight, void* dY,
                               int64_t lddy, float* dweight, tg_dtype dtype, cudaStream_t stream) {
    int rc = check_sizes(T, k, D, y_rows, (int)dtype);
    if (rc) return rc;
    if (!dout || !place || (!dY && !dweight) || (dweight && !Y)) return TG_ERR_INVALID_ARG;
    if (!dweight) Y = nullptr;  // not read
    if (bad_ld(lddo, D) || (Y && bad_ld(ldy, D)) || (dY && bad_ld(lddy, D))) return TG_ERR_STRIDE;
    if (off(dout, 2) || off(Y, 2) || off(dY, 2) || off(place, 4) || off(weight, 4) || off(dweight, 4)) return TG_ERR_ALIGN;
    const void* ptrs[6] = {dY, dweight, dout, Y, place, weight};
    const Span spans[6] = {span_of(dY, y_rows, D, lddy), span_bytes(dweight, (u128)T * k * 4), span_of(dout, T, D, lddo),
                           span_of(Y, y_rows, D, ldy),   span_bytes(place, (u128)T * k * 4),   span_bytes(weight, (u128)T * k * 4)};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (intersects(spans[i], spans[j])) return TG_ERR_OVERLAP;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();
    PointerChecks check{dev};
    for (int i = 0; i < 6; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    CombineParams p = {};
    const int vec = columns_per_unit(D, {dout, Y, dY}, {lddo, Y ? ldy : 8, dY ? lddy : 8});
    p.units = (unsigned)(D / vec);
    p.T = T;
    p.k = (int)k;
    p.D = D;
    p.y_rows = y_rows;
    p.y = static_cast<const uint16_t*>(Y);
    p.ldy = Y ? ldy : 0;
    p.place = place;
    p.weight = weight;
    p.out = static_cast<uint16_t*>(dY);
    p.ldo = dY ? lddy : 0;
    p.dout = static_cast<const uint16_t*>(dout);
    p.lddo = lddo;
    p.dweight = dweight;
    const unsigned blocks = (unsigned)((T * k + kGradWarps - 1) / kGradWarps);
    auto kern = dtype == TG_BF16 ? (vec == 8 ? combine_grad_kernel<true, 8> : combine_grad_kernel<true, 1>)
                                 : (vec == 8 ? combine_grad_kernel<false, 8> : combine_grad_kernel<false, 1>);
    kern<<<blocks, 32 * kGradWarps, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return TG_ERR_CUDA;
    return TG_OK;
}
