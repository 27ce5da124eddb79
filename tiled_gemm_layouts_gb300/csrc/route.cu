// route.cu -- routing of tokens to experts (tg_route) and its gradient
// (tg_route_grad).
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));   key_e = s_e + b_e, or l_e without a bias
//   the k largest keys among the experts of the best groups;   w_j = c s_j (/ their sum)
//
// A warp per token: lane i holds experts i, i + 32, ...  Each of the k rounds
// finds the largest key left: of a lane's own by comparisons, of the warp's by
// one integer reduction (redux.sync) over keys mapped to integers that order
// alike, and its lowest expert by a second one.
//
// Which expert wins must not depend on how an exponential was rounded, so
// the ranking is that of 64-bit arithmetic.  Doing it in 64 bits throughout would
// take the time of E double exponentials per token; instead keys are fp32 with
// a bound on their error, and a token where two keys that decide something are
// nearer than their errors (about one in a thousand with random logits) is
// ranked again by its warp in 64 bits.  Equal logits with equal biases are
// equal in any arithmetic and need none of it; neither do logits that are keys
// themselves.
//
// Weights come from the logits of the chosen, in fp32.  Renormalised sigmoid
// weights are s_j / sum s with s_j = exp(l_j - m) / (1 + exp(l_j)), m = min(0,
// the largest l_j): the factor exp(-m) cancels, and nothing underflows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "../../include/tilegemm.h"
#include "host_common.h"

namespace tg {
namespace {

constexpr int kWarps = 4;          // tokens at a time per block
constexpr int kMaxExperts = 1024;  // 32 per lane

struct RouteParams {
    long long T;
    int E, k, groups, kept, top, size;  // size: experts per group
    int sigmoid, renorm;
    float scale;
    const void* logits;
    long long ld;
    const float* bias;
    int* index;
    float* weight;
    // gradient
    const int* chosen;
    const float* dweight;
    void* dlogits;
    long long lddl;
};

__device__ __forceinline__ float load_one(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ void store_one(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }

__device__ __forceinline__ unsigned warp_max(unsigned x) {
    unsigned r;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ unsigned warp_min(unsigned x) {
    unsigned r;
    asm volatile("redux.sync.min.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(x));
    return r;
}
// fp32 -> an integer that orders alike, above 0 for everything but NaN; +0 and
// -0 are one value.
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
template <class T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
__device__ __forceinline__ float warp_fmax(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Whether groups g of this lane is among the best: fewer than `kept` come before
// it.  `near`: a value that decides it is closer to this one than their errors.
template <class F>
__device__ __forceinline__ bool group_kept(const RouteParams& p, F value, F error, int g, bool& near) {
    int ahead = 0;
    bool close_below = false, close_above = false;
    for (int o = 0; o < p.groups; ++o) {
        const F v = __shfl_sync(0xffffffffu, value, o), err = __shfl_sync(0xffffffffu, error, o);
        const bool first = v > value || (v == value && o < g);
        ahead += first;
        const F gap = v > value ? v - value : value - v;
        if (o != g && err + error > F(0) && gap <= err + error) (first ? close_above : close_below) = true;
    }
    const bool kept = ahead < p.kept;
    // (a close neighbour on the same side of the border is found closer still
    // by the groups at the border: it is enough that any pair there is close)
    near = (g < p.groups) && (close_above || close_below);
    return kept && g < p.groups;
}

// One token ranked in 64 bits by its warp; keys: E doubles of shared memory.
// Returns, in lane j < k, its j-th expert or -1.
template <class IN>
__device__ __noinline__ int rank_in_64_bits(const RouteParams& p, const IN* row, double* keys, int lane) {
    double top = -INFINITY, sum = 0.0;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 32) top = fmax(top, (double)load_one(row + e));
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    // (of a row with +inf: the limit; a NaN takes no part)
    auto mass = [&](double l) { return l == top ? 1.0 : exp(l - top); };
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 32) {
            const double l = load_one(row + e);
            if (l > -INFINITY) sum += mass(l);
        }
        sum = warp_sum(sum);
    }
    auto score = [&](double l) { return p.sigmoid ? 1.0 / (1.0 + exp(-l)) : mass(l) / sum; };
    const bool by_score = p.bias || p.top == 2;  // a group's key
    unsigned kept = 0xffffffffu;
    if (p.groups > 1) {
        for (int e = lane; e < p.E; e += 32) {
            const double l = load_one(row + e);
            const bool may = l > -INFINITY;
            keys[e] = !may ? -INFINITY : by_score ? score(l) + (p.bias ? (double)p.bias[e] : 0.0) : l;
        }
        __syncwarp();
        double a = -INFINITY, b = -INFINITY;
        if (lane < p.groups)
            for (int i = 0; i < p.size; ++i) {
                const double x = keys[lane * p.size + i];
                if (x > a) {
                    b = a;
                    a = x;
                } else if (x > b) {
                    b = x;
                }
            }
        const double value = a + (p.top == 2 && b > -INFINITY ? b : 0.0);
        bool near;
        kept = __ballot_sync(0xffffffffu, group_kept<double>(p, value, 0.0, lane, near));
        __syncwarp();
    }
    for (int e = lane; e < p.E; e += 32) {
        const double l = load_one(row + e);
        const bool may = l > -INFINITY && (p.groups == 1 || (kept >> (e / p.size) & 1u));
        keys[e] = !may ? -INFINITY : p.bias ? score(l) + (double)p.bias[e] : l;
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        double best = -INFINITY;
        int at = p.E;
        for (int e = lane; e < p.E; e += 32)
            if (keys[e] > best) {
                best = keys[e];
                at = e;
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double other = __shfl_xor_sync(0xffffffffu, best, d);
            const int where = __shfl_xor_sync(0xffffffffu, at, d);
            if (other > best || (other == best && where < at)) {
                best = other;
                at = where;
            }
        }
        if (at == p.E) break;
        if (lane == j) mine = at;
        if (lane == at % 32) keys[at] = -INFINITY;  // this lane's own
        __syncwarp();
    }
    return mine;
}

template <class IN, int V>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteParams p) {
    extern __shared__ double shared_keys[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double* wide = shared_keys + (size_t)warp * p.E;
    float* narrow = reinterpret_cast<float*>(wide);
    float b[V];
    int group[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 32 + lane;
        b[v] = p.bias && e < p.E ? p.bias[e] : 0.0f;
        group[v] = e / p.size;
    }
    // Largest relative errors of a score and of a rounded sum.  A score's: 2^-18
    // from the exponential's argument l - top below 128 (beyond, scores are
    // below 1e-55), 2^-18.8 from a sum of 37 steps, 2^-21 from functions and quotient.
    constexpr float kScoreError = 0x1p-17f, kSumError = 0x1p-23f;
    const bool need_scores = p.bias || (p.groups > 1 && p.top == 2) || (!p.sigmoid && !p.renorm);
    for (long long t = (long long)blockIdx.x * kWarps + warp; t < p.T; t += (long long)gridDim.x * kWarps) {
        const IN* row = static_cast<const IN*>(p.logits) + t * p.ld;
        float l[V], s[V];
        bool may[V];
        bool spoilt = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 32 + lane;
            l[v] = e < p.E ? load_one(row + e) : -INFINITY;
            may[v] = l[v] > -INFINITY;
            spoilt |= !(l[v] < INFINITY);  // NaN or +inf
        }
        spoilt = __any_sync(0xffffffffu, spoilt);
        float top = -INFINITY, sum = 1.0f;
        if (need_scores && !p.sigmoid) {
            sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
            top = warp_fmax(top);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = !may[v] ? 0.0f : l[v] == top ? 1.0f : expf(l[v] - top);  // (of +inf: the limit)
                sum += s[v];
            }
            sum = warp_sum(sum);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = __fdividef(s[v], sum);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = need_scores ? sigmoid(l[v]) : 0.0f;
        }
        bool near = false;
        if (p.groups > 1) {
            const bool by_score = p.bias || p.top == 2;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = v * 32 + lane;
                if (e < p.E) narrow[e] = !may[v] ? -INFINITY : by_score ? s[v] + b[v] : l[v];
            }
            __syncwarp();
            // 32 / groups lanes (a power of two) per group, each with every so many of its keys
            int lanes = 1;
            while (lanes * 2 * p.groups <= 32) lanes *= 2;
            const int g = lane / lanes, part = lane % lanes, steps = (p.size + lanes - 1) / lanes;
            float first = -INFINITY, second = -INFINITY;
            if (g < p.groups) {
                int i = g % steps;  // groups start at different steps, in different banks
                for (int n = 0; n < steps; ++n) {
                    const int at = i * lanes + part;
                    if (at < p.size) {
                        const float x = narrow[g * p.size + at];
                        second = fmaxf(second, fminf(first, x));
                        first = fmaxf(first, x);
                    }
                    i = i + 1 == steps ? 0 : i + 1;
                }
            }
            for (int d = 1; d < lanes; d *= 2) {
                const float of = __shfl_xor_sync(0xffffffffu, first, d), os = __shfl_xor_sync(0xffffffffu, second, d);
                second = fmaxf(fmaxf(second, os), fminf(first, of));
                first = fmaxf(first, of);
            }
            const float mine = first + (p.top == 2 && second > -INFINITY ? second : 0.0f);
            // lane g's own: the value of group g
            const float value = __shfl_sync(0xffffffffu, mine, (lane * lanes) & 31);
            const float error = !by_score ? 0.0f : 2.0f * kScoreError + 4.0f * kSumError * fabsf(value) + 8.0f * kSumError;
            bool close;
            const bool kept = group_kept<float>(p, lane < p.groups ? value : -INFINITY,
                                                lane < p.groups && value > -INFINITY ? error : 0.0f, lane, close);
            near = __any_sync(0xffffffffu, close);
            const unsigned mask = __ballot_sync(0xffffffffu, kept);
#pragma unroll
            for (int v = 0; v < V; ++v) may[v] = may[v] && (mask >> (group[v] & 31) & 1u);
            __syncwarp();
        }
        // the keys, as integers that order alike; 0: not to be chosen (any more)
        unsigned key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = may[v] ? ordered(p.bias ? s[v] + b[v] : l[v]) : 0u;
        int mine = -1;
        unsigned my_key = 0, last = 0;
        unsigned best = 0;
        int at = 0;
        auto find = [&]() {
            best = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] > best) {
                    best = key[v];
                    at = v;
                }
        };
        find();
        for (int j = 0; j < p.k; ++j) {
            const unsigned winner = warp_max(best);
            if (winner == 0) {
                last = 0;
                break;
            }
            const unsigned e = warp_min(best == winner ? (unsigned)(at * 32 + lane) : 0xffffffffu);
            if (lane == j) {
                mine = (int)e;
                my_key = winner;
            }
            last = winner;
            if (e % 32 == lane) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v == at) key[v] = 0;
                find();
            }
        }
        if (p.bias && !near) {
            // neighbours in the order, and the last one and those left out
            const float value = unordered(my_key);
            float logit = 0.0f, bias = 0.0f, error = 0.0f;
            if (mine >= 0) {
                logit = load_one(row + mine);
                bias = p.bias[mine];
                error = kScoreError * (fabsf(value) + fabsf(bias)) + 4.0f * kSumError * (fabsf(value) + fabsf(bias)) + 1e-30f;
            }
            const float next = __shfl_down_sync(0xffffffffu, value, 1), next_error = __shfl_down_sync(0xffffffffu, error, 1);
            const float next_logit = __shfl_down_sync(0xffffffffu, logit, 1);
            const float next_bias = __shfl_down_sync(0xffffffffu, bias, 1);
            const int next_mine = __shfl_down_sync(0xffffffffu, mine, 1);
            bool close = lane + 1 < p.k && next_mine >= 0 && value - next <= error + next_error &&
                         !(logit == next_logit && bias == next_bias);
            if (last) {
                const float edge = unordered(last) - __shfl_sync(0xffffffffu, error, p.k - 1);
                const float edge_logit = __shfl_sync(0xffffffffu, logit, p.k - 1);
                const float edge_bias = __shfl_sync(0xffffffffu, bias, p.k - 1);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (key[v] == 0) continue;
                    const float x = unordered(key[v]), size = fabsf(x) + fabsf(b[v]);
                    close |= x + (kScoreError + 4.0f * kSumError) * size + 1e-30f >= edge &&
                             !(l[v] == edge_logit && b[v] == edge_bias);
                }
            }
            near = __any_sync(0xffffffffu, close);
        }
        if (near) mine = rank_in_64_bits<IN>(p, row, wide, lane);
        // weights
        const float logit = mine >= 0 ? load_one(row + mine) : -INFINITY;
        float w = 0.0f;
        if (p.renorm) {
            float m = warp_fmax(logit);
            if (p.sigmoid) m = fminf(m, 0.0f);
            w = mine < 0 ? 0.0f : !p.sigmoid ? expf(logit - m) : logit > 0.0f ? sigmoid(logit)
                                : expf(logit - m) / (1.0f + expf(logit));
            // (m = 0 where a logit is above it, so both forms have the same factor)
            const float total = warp_sum(w);
            w = mine < 0 ? 0.0f : w / total;
        } else if (mine >= 0) {
            w = p.sigmoid ? sigmoid(logit) : expf(logit - top) / sum;
        }
        if (!p.sigmoid && spoilt && mine >= 0) w = NAN;
        if (lane < p.k) {
            p.index[t * p.k + lane] = mine;
            p.weight[t * p.k + lane] = w * p.scale;
        }
        __syncwarp();
    }
}

// dlogits.  With p_e the softmax, g_j = c dweight_j and w_j the weights over c:
//   softmax                p_e ([e chosen] g_e - sum g_j p_j)
//   softmax, renormalised  [e chosen] w_e (g_e - sum g_j w_j)
//   sigmoid                [e chosen] g_e s_e (1 - s_e)
//   sigmoid, renormalised  [e chosen] w_e (1 - s_e) (g_e - sum g_j w_j)
// so all but the first need only the chosen logits.
template <class IN, int V>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const RouteParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool dense = !p.sigmoid && !p.renorm;
    for (long long t = (long long)blockIdx.x * kWarps + warp; t < p.T; t += (long long)gridDim.x * kWarps) {
        const IN* row = static_cast<const IN*>(p.logits) + t * p.ld;
        IN* out = static_cast<IN*>(p.dlogits) + t * p.lddl;
        int e = lane < p.k ? p.chosen[t * p.k + lane] : -1;
        if (e < 0 || e >= p.E) e = -1;
        const float g = e >= 0 ? p.dweight[t * p.k + lane] * p.scale : 0.0f;
        const float logit = e >= 0 ? load_one(row + e) : -INFINITY;
        float prob[V];
        float d, dot = 0.0f;
        if (dense) {
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int x = v * 32 + lane;
                prob[v] = x < p.E ? load_one(row + x) : -INFINITY;
                top = fmaxf(top, prob[v]);
            }
            top = warp_fmax(top);
            const float base = top == -INFINITY ? 0.0f : top;  // a row of -inf: no mass anywhere
#pragma unroll
            for (int v = 0; v < V; ++v) {
                prob[v] = expf(prob[v] - base);
                sum += prob[v];
            }
            sum = warp_sum(sum);
            const float inverse = top == -INFINITY ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int v = 0; v < V; ++v) prob[v] *= inverse;
            const float part = e >= 0 ? g * (expf(logit - base) * inverse) : 0.0f;
            dot = warp_sum(part);
            d = g;
        } else if (p.renorm) {
            float m = warp_fmax(logit);
            if (p.sigmoid) m = fminf(m, 0.0f);
            float w = e < 0 ? 0.0f : !p.sigmoid ? expf(logit - m) : logit > 0.0f ? sigmoid(logit)
                             : expf(logit - m) / (1.0f + expf(logit));
            const float total = warp_sum(w);
            w = e < 0 ? 0.0f : w / total;
            const float mean = warp_sum(g * w);
            d = w * (g - mean);
            if (p.sigmoid) d *= 1.0f / (1.0f + expf(logit));
        } else {
            d = e < 0 ? 0.0f : g * sigmoid(logit) * (1.0f / (1.0f + expf(logit)));
        }
        if (e < 0) d = 0.0f;
        float full[V];
#pragma unroll
        for (int v = 0; v < V; ++v) full[v] = 0.0f;
        for (int j = 0; j < p.k; ++j) {
            const int at = __shfl_sync(0xffffffffu, e, j);
            const float x = __shfl_sync(0xffffffffu, d, j);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at == v * 32 + lane) full[v] += x;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int x = v * 32 + lane;
            if (x < p.E) store_one(out + x, dense ? prob[v] * (full[v] - dot) : full[v]);
        }
    }
}

template <class IN, int V>
cudaError_t launch_one(const RouteParams& p, bool grad, int sms, cudaStream_t stream) {
    const long long blocks = (p.T + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(blocks < 16LL * sms ? blocks : 16LL * sms);
    if (grad)
        route_grad_kernel<IN, V><<<grid, 32 * kWarps, 0, stream>>>(p);
    else
        route_kernel<IN, V><<<grid, 32 * kWarps, (size_t)kWarps * p.E * sizeof(double), stream>>>(p);
    return cudaGetLastError();
}

template <class IN>
cudaError_t launch_typed(const RouteParams& p, bool grad, int sms, cudaStream_t stream) {
    if (p.E <= 32) return launch_one<IN, 1>(p, grad, sms, stream);
    if (p.E <= 64) return launch_one<IN, 2>(p, grad, sms, stream);
    if (p.E <= 128) return launch_one<IN, 4>(p, grad, sms, stream);
    if (p.E <= 256) return launch_one<IN, 8>(p, grad, sms, stream);
    if (p.E <= 512) return launch_one<IN, 16>(p, grad, sms, stream);
    return launch_one<IN, 32>(p, grad, sms, stream);
}

int launch(const RouteParams& p, bool grad, int dtype, int sms, cudaStream_t stream) {
    const cudaError_t e = dtype == TG_F32    ? launch_typed<float>(p, grad, sms, stream)
                          : dtype == TG_BF16 ? launch_typed<__nv_bfloat16>(p, grad, sms, stream)
                                             : launch_typed<__half>(p, grad, sms, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}

int check_options(int64_t T, int64_t E, const tg_route_options* o, int dtype) {
    if (T <= 0 || E <= 0 || T > kMaxDim || E > kMaxExperts || !o) return TG_ERR_INVALID_ARG;
    if ((o->score != TG_ROUTE_SOFTMAX && o->score != TG_ROUTE_SIGMOID) || o->groups < 1 || o->groups > 32 ||
        E % o->groups != 0 || o->groups_kept < 1 || o->groups_kept > o->groups ||
        (o->group_top != 1 && o->group_top != 2) || (o->renormalise != 0 && o->renormalise != 1) ||
        o->k < 1 || o->k > 32 || o->k > E / o->groups * o->groups_kept || !std::isfinite(o->scale))
        return TG_ERR_INVALID_ARG;
    if (dtype != TG_F16 && dtype != TG_BF16 && dtype != TG_F32) return TG_ERR_DTYPE;
    return TG_OK;
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

Span rows_span(const void* p, int64_t rows, int64_t width, int64_t ld, int size) {
    return span_bytes(p, ((u128)(rows - 1) * (u128)ld + (u128)width) * (u128)size);
}

RouteParams params_of(int64_t T, int64_t E, const tg_route_options& o) {
    RouteParams p = {};
    p.T = T;
    p.E = (int)E;
    p.k = o.k;
    p.groups = o.groups;
    p.kept = o.groups_kept;
    p.top = o.group_top;
    p.size = (int)(E / o.groups);
    p.sigmoid = o.score == TG_ROUTE_SIGMOID;
    p.renorm = o.renormalise;
    p.scale = o.scale;
    return p;
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_route(int64_t T, int64_t E, const void* logits, int64_t ld, const float* bias,
                        int32_t* index, float* weight, tg_dtype dtype, const tg_route_options* options,
                        cudaStream_t stream) {
    int rc = check_options(T, E, options, (int)dtype);
    if (rc) return rc;
    if (!logits || !index || !weight) return TG_ERR_INVALID_ARG;
    if (ld < E || ld > kMaxLd) return TG_ERR_STRIDE;
    const int size = dtype == TG_F32 ? 4 : 2;
    if (off(logits, size) || off(bias, 4) || off(index, 4) || off(weight, 4)) return TG_ERR_ALIGN;
    const Span spans[4] = {span_bytes(index, (u128)T * options->k * 4), span_bytes(weight, (u128)T * options->k * 4),
                           rows_span(logits, T, E, ld, size), span_bytes(bias, (u128)E * 4)};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (intersects(spans[i], spans[j])) return TG_ERR_OVERLAP;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();  // the allocation-range query of check_pointer
    const void* ptrs[4] = {index, weight, logits, bias};
    PointerChecks check{dev};
    for (int i = 0; i < 4; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    RouteParams p = params_of(T, E, *options);
    p.logits = logits;
    p.ld = ld;
    p.bias = bias;
    p.index = index;
    p.weight = weight;
    return launch(p, false, (int)dtype, info->sms, stream);
}

extern "C" int tg_route_grad(int64_t T, int64_t E, const void* logits, int64_t ld, const int32_t* index,
                             const float* dweight, void* dlogits, int64_t lddl, tg_dtype dtype,
                             const tg_route_options* options, cudaStream_t stream) {
    int rc = check_options(T, E, options, (int)dtype);
    if (rc) return rc;
    if (!logits || !index || !dweight || !dlogits) return TG_ERR_INVALID_ARG;
    if (ld < E || ld > kMaxLd || lddl < E || lddl > kMaxLd) return TG_ERR_STRIDE;
    const int size = dtype == TG_F32 ? 4 : 2;
    if (off(logits, size) || off(dlogits, size) || off(index, 4) || off(dweight, 4)) return TG_ERR_ALIGN;
    const Span spans[4] = {rows_span(dlogits, T, E, lddl, size), rows_span(logits, T, E, ld, size),
                           span_bytes(index, (u128)T * options->k * 4), span_bytes(dweight, (u128)T * options->k * 4)};
    for (int j = 1; j < 4; ++j)
        if (intersects(spans[0], spans[j])) return TG_ERR_OVERLAP;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    load_driver_entry_points();
    const void* ptrs[4] = {dlogits, logits, index, dweight};
    PointerChecks check{dev};
    for (int i = 0; i < 4; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    RouteParams p = params_of(T, E, *options);
    p.logits = logits;
    p.ld = ld;
    p.chosen = index;
    p.dweight = dweight;
    p.dlogits = dlogits;
    p.lddl = lddl;
    return launch(p, true, (int)dtype, info->sms, stream);
}
