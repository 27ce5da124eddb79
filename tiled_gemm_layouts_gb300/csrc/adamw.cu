// adamw.cu -- one AdamW step over many tensors (tg_adamw).
//
//   g' = s g;  m = b1 m + (1-b1) g';  v = b2 v + (1-b2) g'^2
//   p = p (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v) / sqrt(1-b2^t) + eps)
//
// in fp32, on the fp32 master copy where there is one; the 16-bit parameter is
// then its rounded copy.  Bound by memory: every element of p, g, m and v is
// read once and written once.  With 8-bit states an element is 16 bytes and
// leaves room for about 110 instructions at the memory's rate.  The step's
// quotient is the hardware's approximation (within 2 ulp, far below eps's and
// lr's meaning).  What the states are rounded from is kept as exact as the
// formula, without contraction, because a last bit more or less decides some
// roundings to 8 bits: sqrt(v) and the quotients by a block's scales are an
// approximation and one correction by its fused remainder (Markstein 1990).
// (Library quotients and roots, one byte converted at a time: 819 us for 2e8
// elements; as it is now 519 to 523, 6.1 TB/s, with 78 % of the issue slots
// taken.  32-bit states move 28 bytes per element at 7.0 TB/s.  Tensors that
// start between 16-byte boundaries are accessed by element: 5e7 elements 467 us
// with 32-bit states, aligned 203, and 292 with 8-bit ones, aligned 133.)
//
// 32-bit states are two floats per element.  8-bit states are two e4m3 bytes
// per element and, for each block of 256 elements, one fp32 scale each (a
// 448th of the block's largest magnitude): m itself, rounded to nearest even,
// and r = sqrt(v).  The root halves the exponent range that e4m3's 18
// octaves have to hold.  r is rounded up with the probability of what is cut
// off: with b2 = 0.999 a step moves r by 0.05 %, far below e4m3's spacing of
// 6 to 12 %, and rounding to nearest would never let it decay.  A root above
// zero stays above zero, so that a small v next to a large one does not turn
// its m into an unbounded step.  A gradient that is no finite number makes its
// block's scales infinite or NaN, as the formula for the scales has it: a caller
// that may have such gradients looks at them before the step.
//
// Tensors are dealt out in chunks of 2048 elements; their descriptors travel
// as kernel arguments, up to kMaxTensors per launch, and a block finds its
// tensor by bisection, so the step allocates nothing and can be captured.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "../../include/tilegemm.h"
#include "host_common.h"
#include "packed.cuh"

namespace tg {
namespace {

constexpr int kBlock8 = 256;      // elements that share a scale
constexpr int kChunk = 2048;      // elements of one block of threads: 8 per thread
constexpr int kMaxTensors = 256;  // descriptors per launch
constexpr int kFewTensors = 32;   // and of the launch with small arguments

struct AdamTensor {
    void* p;
    float* master;
    const void* g;
    void *m, *v;
    float *m_scale, *v_scale;
    long long n;
};
template <int CAP>
struct AdamParams {
    float beta1, rest1, beta2, rest2, keep, step_size, root, eps;
    const float* grad_scale;
    uint32_t seed;
    int count;
    int first[CAP + 1];  // first chunk of each tensor
    AdamTensor t[CAP];
};
static_assert(sizeof(AdamParams<kMaxTensors>) <= 32000, "kernel arguments");

// 20 pseudo-random bits from an element's index and the seed, the same for every
// tensor of a step: a 32-bit integer mixer by xor-shifts and multiplications, with
// shifts and multipliers from the search that C. Wellons published ("hash
// prospector", 2018).
__device__ __forceinline__ uint32_t mixed_bits(uint32_t i, uint32_t seed) {
    uint32_t x = i + seed * 0x9E3779B9u;
    x = (x ^ (x >> 16)) * 0x21F0AAADu;
    x = (x ^ (x >> 15)) * 0x735A2D97u;
    return (x ^ (x >> 15)) & 0xFFFFFu;
}

// Two e4m3 bytes of a word to fp32, and two values to a word's low half.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Largest magnitude; a NaN stays a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 1 / x within an ulp.  Only a denominator below fp32's normal range would be
// taken for zero; sqrt of the smallest fp32 is 3e-23.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// r = sqrt(x) for 8 values between `low` and `high`: with y near 1/sqrt(x),
// s = x y is off by (x - s^2) / (2 sqrt(x)).
__device__ __forceinline__ void roots(const float (&x)[8], float low, float high, float (&r)[8]) {
    if (low >= 0x1p-100f && high <= 0x1p100f) {
        const f2 half = pair(0.5f, 0.5f);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            float y0, y1;
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(x[k]));
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(x[k + 1]));
            const f2 v = pair(x[k], x[k + 1]), y = pair(y0, y1), s = mul(v, y);
            const f2 root = fma(fma(mul(s, pair(-1.0f, -1.0f)), s, v), mul(y, half), s);
            r[k] = split(root).x;
            r[k + 1] = split(root).y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = __fsqrt_rn(x[k]);
    }
}

// q from 0 to (but for a rounding) 448, or NaN, to a value that e4m3 holds, up
// with the probability of what is cut off; the conversion saturates.  Its 3 mantissa bits are the upper ones of fp32's 23;
// below 2^-6, where e4m3's steps stay 2^-9, so are those of q + 2^-6.
__device__ __forceinline__ float stochastic(float q, uint32_t bits) {
    const float off = q < 0x1p-6f ? 0x1p-6f : 0.0f;
    const float cut = __uint_as_float((__float_as_uint(q + off) + bits) & ~0xFFFFFu) - off;
    return max_nan(cut, q > 0.0f ? 0x1p-9f : q);
}

// Element types of p and of g: 0 fp16, 1 bf16, 2 fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* base, long long i, int n, float (&x)[8]) {
    if constexpr (DT == TG_F32) {
        const float* s = static_cast<const float*>(base) + i;
        if (n == 8 && (reinterpret_cast<uintptr_t>(s) & 15u) == 0) {
            *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(s);
            *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(s + 4);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = k < n ? s[k] : 0.0f;
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(base) + i;
        uint16_t e[8];
        if (n == 8 && (reinterpret_cast<uintptr_t>(s) & 15u) == 0) {
            *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(s);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = k < n ? s[k] : (uint16_t)0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = DT == TG_BF16 ? __uint_as_float((uint32_t)e[k] << 16)
                                 : __half2float(__ushort_as_half(e[k]));
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* base, long long i, int n, const float (&x)[8]) {
    if constexpr (DT == TG_F32) {
        float* d = static_cast<float*>(base) + i;
        if (n == 8 && (reinterpret_cast<uintptr_t>(d) & 15u) == 0) {
            *reinterpret_cast<float4*>(d) = *reinterpret_cast<const float4*>(x);
            *reinterpret_cast<float4*>(d + 4) = *reinterpret_cast<const float4*>(x + 4);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) d[k] = x[k];
        }
    } else {
        uint16_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            e[k] = DT == TG_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x[k]))
                                 : __half_as_ushort(__float2half_rn(x[k]));
        uint16_t* d = static_cast<uint16_t*>(base) + i;
        if (n == 8 && (reinterpret_cast<uintptr_t>(d) & 15u) == 0) {
            *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(e);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) d[k] = e[k];
        }
    }
}

// 8 state bytes of a block times its scale.
__device__ __forceinline__ void load_codes(const void* base, long long i, int n, float scale,
                                           float (&x)[8]) {
    const uint8_t* s = static_cast<const uint8_t*>(base) + i;
    uint32_t e[2] = {0, 0};
    if (n == 8 && (reinterpret_cast<uintptr_t>(s) & 7u) == 0) {
        *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(s);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) e[k >> 2] |= (uint32_t)s[k] << (8 * (k & 3));
    }
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float2 f = from_e4m3x2(e[k >> 2] >> (8 * (k & 3)));
        x[k] = f.x * scale;
        x[k + 1] = f.y * scale;
    }
}
__device__ __forceinline__ void store_codes(void* base, long long i, int n, const float (&x)[8]) {
    uint32_t e[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        e[k] = to_e4m3x2(x[4 * k], x[4 * k + 1]) | (to_e4m3x2(x[4 * k + 2], x[4 * k + 3]) << 16);
    uint8_t* d = static_cast<uint8_t*>(base) + i;
    if (n == 8 && (reinterpret_cast<uintptr_t>(d) & 7u) == 0) {
        *reinterpret_cast<uint2*>(d) = make_uint2(e[0], e[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) d[k] = (uint8_t)(e[k >> 2] >> (8 * (k & 3)));
    }
}

// x over a block's scale.  A scale far from the middle of fp32's range (or no
// number) divides instead: its reciprocal or the remainder might not be exact.
__device__ __forceinline__ void over_scale(const float (&x)[8], float scale, float (&q)[8]) {
    if (scale >= 0x1p-100f && scale <= 0x1p100f) {
        const float inv = __frcp_rn(scale);
        const f2 i2 = pair(inv, inv), s2 = pair(-scale, -scale);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const f2 v = pair(x[k], x[k + 1]), a = mul(v, i2), r = fma(fma(a, s2, v), i2, a);
            q[k] = split(r).x;
            q[k + 1] = split(r).y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = scale == 0.0f ? x[k] : __fdiv_rn(x[k], scale);
    }
}

// One chunk per block of 256 threads, 8 consecutive elements per thread: a
// warp holds exactly one 256-element block of the 8-bit states.
template <int PT, int GT, bool EIGHT, int CAP>
__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ AdamParams<CAP> a) {
    int lo = 0, hi = a.count;  // the tensor whose chunks hold this block
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= (int)blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const AdamTensor& t = a.t[lo];
    const long long i = (long long)((int)blockIdx.x - a.first[lo]) * kChunk + threadIdx.x * 8;
    const int n = (int)max(0LL, min(8LL, t.n - i));
    if (!__any_sync(0xffffffffu, n > 0)) return;
    const long long block = i / kBlock8;
    float g[8], w[8], m[8], v[8];
    if (n > 0) {
        load8<GT>(t.g, i, n, g);
        if (t.master)
            load8<TG_F32>(t.master, i, n, w);
        else
            load8<PT>(t.p, i, n, w);
    }
    if (n <= 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = w[k] = m[k] = v[k] = 0.0f;
    } else if constexpr (EIGHT) {
        load_codes(t.m, i, n, t.m_scale[block], m);
        load_codes(t.v, i, n, t.v_scale[block], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * v[k];
    } else {
        load8<TG_F32>(t.m, i, n, m);
        load8<TG_F32>(t.v, i, n, v);
    }
    const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.0f;
    float r[8];  // sqrt(v)
    const f2 b1 = pair(a.beta1, a.beta1), b2 = pair(a.beta2, a.beta2), c1 = pair(a.rest1, a.rest1),
             c2 = pair(a.rest2, a.rest2), gs2 = pair(gs, gs);
    float low = INFINITY, high = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        // the sums are not packed: the compiler contracts packed products and
        // sums, and a fused one differs from the formula's in a quarter of the
        // cases by a last bit
        const f2 gg = mul(pair(g[k], g[k + 1]), gs2);
        const float2 m1 = split(mul(pair(m[k], m[k + 1]), b1)), m2 = split(mul(gg, c1));
        const float2 v1 = split(mul(pair(v[k], v[k + 1]), b2)), v2 = split(mul(mul(gg, gg), c2));
        m[k] = __fadd_rn(m1.x, m2.x);
        m[k + 1] = __fadd_rn(m1.y, m2.y);
        v[k] = __fadd_rn(v1.x, v2.x);
        v[k + 1] = __fadd_rn(v1.y, v2.y);
        low = fminf(low, fminf(v[k], v[k + 1]));
        high = max_nan(high, max_nan(v[k], v[k + 1]));
    }
    roots(v, low, high, r);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        w[k] = fmaf(w[k], a.keep, -(m[k] * reciprocal(fmaf(r[k], a.root, a.eps))) * a.step_size);
    if (n > 0) {
        if (t.master) store8<TG_F32>(t.master, i, n, w);
        store8<PT>(t.p, i, n, w);
    }
    if constexpr (!EIGHT) {
        if (n > 0) {
            store8<TG_F32>(t.m, i, n, m);
            store8<TG_F32>(t.v, i, n, v);
        }
    } else {
        float mt = 0.0f, vt = 0.0f;  // the block's largest magnitudes
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // zeros past the tensor's end
            mt = max_nan(mt, fabsf(m[k]));
            vt = max_nan(vt, r[k]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            mt = max_nan(mt, __shfl_xor_sync(0xffffffffu, mt, o));
            vt = max_nan(vt, __shfl_xor_sync(0xffffffffu, vt, o));
        }
        const float ms = mt * (float)(1.0 / 448.0), vs = vt * (float)(1.0 / 448.0);
        if (n > 0) {
            over_scale(m, ms, m);  // the conversion saturates at 448
            store_codes(t.m, i, n, m);
            over_scale(r, vs, r);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                r[k] = stochastic(r[k], mixed_bits((uint32_t)(i + k), a.seed));
            store_codes(t.v, i, n, r);
            if ((threadIdx.x & 31) == 0) {
                t.m_scale[block] = ms;
                t.v_scale[block] = vs;
            }
        }
    }
}

template <int PT, int GT, int CAP>
cudaError_t launch(const AdamParams<CAP>& a, bool eight, cudaStream_t stream) {
    const unsigned grid = (unsigned)a.first[a.count];
    if (eight)
        adamw_kernel<PT, GT, true, CAP><<<grid, 256, 0, stream>>>(a);
    else
        adamw_kernel<PT, GT, false, CAP><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

// The tensors [0, count) without the empty ones, CAP per launch.
template <int CAP>
cudaError_t step(int64_t count, const tg_adamw_tensor* tensors, const tg_adamw_options* o,
                 cudaStream_t stream) {
    const bool eight = o->state_bits == 8, wide = o->grad_dtype == TG_F32;
    AdamParams<CAP> a;
    a.beta1 = (float)o->beta1;
    a.rest1 = (float)(1.0 - o->beta1);
    a.beta2 = (float)o->beta2;
    a.rest2 = (float)(1.0 - o->beta2);
    a.keep = (float)(1.0 - o->lr * o->weight_decay);
    a.step_size = (float)(o->lr / (1.0 - std::pow(o->beta1, (double)o->step)));
    a.root = (float)(1.0 / std::sqrt(1.0 - std::pow(o->beta2, (double)o->step)));
    a.eps = (float)o->eps;
    a.grad_scale = o->grad_scale;
    a.seed = o->seed;
    a.count = 0;
    a.first[0] = 0;
    cudaError_t e = cudaSuccess;
    for (int64_t k = 0; k < count && e == cudaSuccess; ++k) {
        const tg_adamw_tensor& t = tensors[k];
        if (t.numel > 0) {
            a.t[a.count] = AdamTensor{t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.numel};
            a.first[a.count + 1] = a.first[a.count] + (int)((t.numel + kChunk - 1) / kChunk);
            ++a.count;
        }
        if (a.count == 0 || (a.count < CAP && k + 1 < count)) continue;
        if (o->dtype == TG_F32)
            e = launch<TG_F32, TG_F32>(a, eight, stream);
        else if (o->dtype == TG_BF16)
            e = wide ? launch<TG_BF16, TG_F32>(a, eight, stream)
                     : launch<TG_BF16, TG_BF16>(a, eight, stream);
        else
            e = wide ? launch<TG_F16, TG_F32>(a, eight, stream)
                     : launch<TG_F16, TG_F16>(a, eight, stream);
        a.count = 0;
    }
    return e;
}

int size_of(int dtype) { return dtype == TG_F32 ? 4 : 2; }

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_adamw(int64_t count, const tg_adamw_tensor* tensors, const tg_adamw_options* o,
                        cudaStream_t stream) {
    if (count < 0 || count > kMaxDim || (count > 0 && !tensors) || !o) return TG_ERR_INVALID_ARG;
    auto type_ok = [](int d) { return d == TG_F16 || d == TG_BF16 || d == TG_F32; };
    if (!type_ok((int)o->dtype) || !type_ok((int)o->grad_dtype)) return TG_ERR_DTYPE;
    // a gradient comes in its parameter's type, or wider
    if (o->grad_dtype != o->dtype && o->grad_dtype != TG_F32) return TG_ERR_DTYPE;
    if (o->state_bits != 8 && o->state_bits != 32) return TG_ERR_INVALID_ARG;
    if (o->step < 1 || !(o->beta1 >= 0.0 && o->beta1 < 1.0) || !(o->beta2 >= 0.0 && o->beta2 < 1.0) ||
        !(o->eps >= 0.0) || !std::isfinite(o->lr) || !std::isfinite(o->weight_decay))
        return TG_ERR_INVALID_ARG;
    const bool eight = o->state_bits == 8;
    const int es = size_of((int)o->dtype), gs = size_of((int)o->grad_dtype);
    auto off = [](const void* p, unsigned b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) != 0; };
    if (off(o->grad_scale, 4)) return TG_ERR_ALIGN;
    // the spans of one tensor: the six that are written, then the gradient
    struct Operands {
        const void* ptr[7];
        Span span[7];
    };
    auto operands = [&](const tg_adamw_tensor& t) {
        const u128 n = (u128)t.numel, b = (n + kBlock8 - 1) / kBlock8 * 4;
        Operands r;
        const void* ptr[7] = {t.param, t.master, t.m, t.v, t.m_scale, t.v_scale, t.grad};
        const u128 bytes[7] = {n * es, n * 4, n * (eight ? 1 : 4), n * (eight ? 1 : 4), b, b, n * gs};
        for (int k = 0; k < 7; ++k) {
            r.ptr[k] = (!eight && (k == 4 || k == 5)) ? nullptr : ptr[k];
            r.span[k] = span_bytes(r.ptr[k], bytes[k]);
        }
        return r;
    };
    int64_t chunks = 0;
    for (int64_t k = 0; k < count; ++k) {
        const tg_adamw_tensor& t = tensors[k];
        if (t.numel < 0) return TG_ERR_INVALID_ARG;
        if (t.numel == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale)) ||
            (o->dtype == TG_F32 && t.master))
            return TG_ERR_INVALID_ARG;
        if (off(t.param, es) || off(t.grad, gs) || off(t.master, 4) || off(t.m_scale, 4) ||
            off(t.v_scale, 4) || (!eight && (off(t.m, 4) || off(t.v, 4))))
            return TG_ERR_ALIGN;
        chunks += (t.numel + kChunk - 1) / kChunk;
        if (chunks > kMaxDim) return TG_ERR_INVALID_ARG;
    }
    if (chunks == 0) return TG_OK;
    // no byte that is written may be another operand's: sweep all spans in order
    struct Mark {
        uintptr_t lo;
        u128 hi;
        bool written;
    };
    const std::unique_ptr<Mark[]> marks(new (std::nothrow) Mark[(size_t)count * 7 + 1]);
    if (!marks) return TG_ERR_CUDA;
    size_t used = 0;
    const Span factor = span_bytes(o->grad_scale, 4);  // read by every block
    if (factor.present) marks[used++] = Mark{factor.lo, factor.hi, false};
    for (int64_t k = 0; k < count; ++k) {
        if (tensors[k].numel == 0) continue;
        const Operands r = operands(tensors[k]);
        for (int i = 0; i < 7; ++i)
            if (r.span[i].present) marks[used++] = Mark{r.span[i].lo, r.span[i].hi, i < 6};
    }
    std::sort(marks.get(), marks.get() + used, [](const Mark& x, const Mark& y) { return x.lo < y.lo; });
    u128 any = 0, written = 0;  // furthest end so far
    for (size_t k = 0; k < used; ++k) {
        const Mark& x = marks[k];
        if ((u128)x.lo < written || (x.written && (u128)x.lo < any)) return TG_ERR_OVERLAP;
        if (x.hi > any) any = x.hi;
        if (x.written && x.hi > written) written = x.hi;
    }
    int rc, dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();
    PointerChecks check{dev};
    if ((rc = check(o->grad_scale, factor))) return rc;
    // operand by operand: the tensors of one list often lie side by side
    for (int i = 0; i < 7; ++i)
        for (int64_t k = 0; k < count; ++k) {
            if (tensors[k].numel == 0) continue;
            const Operands r = operands(tensors[k]);
            if ((rc = check(r.ptr[i], r.span[i]))) return rc;
        }
    if ((count <= kFewTensors ? step<kFewTensors>(count, tensors, o, stream)
                              : step<kMaxTensors>(count, tensors, o, stream)) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
