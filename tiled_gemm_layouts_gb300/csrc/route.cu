// route.cu -- routing of tokens to experts (tg_route) and its gradient
// (tg_route_grad).
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));   key_e = s_e + b_e, or l_e without a bias
//   the k largest keys among the experts of the best groups;   w_j = c s_j (/ their sum)
//
// Bound by the latency of its chains of instructions: 16384 tokens of 256 experts are
// 8 MB, 1.2 us, and take 18 to 22, with half of the issue slots used and 1.12 rounds of
// blocks (14592 tokens, one round: 17).  So as little as possible is done across lanes.  A token has as many lanes as its
// experts, in runs of at most 32 (64 where that makes too many) of one group each,
// need, rounded up to a power of two, and a warp 32 / lanes tokens.  A lane's keys lie
// in shared memory, four by four; registers hold a maximum per four.  A group's
// two largest are then a lane's or a few lanes' affair, and each of the k rounds
// that find the largest key left costs a lane a maximum over its registers, a few
// shuffles, and, if it was its own, one read and one write of four.  (A warp per
// token with its keys 32 experts apart and integer reductions over the warp: about
// 1100 instructions a token, 45 us; runs in registers instead of shared memory: as
// long, for the branches that taking a key out of one of 32 registers needs.)
//
// Which expert wins must not depend on how an exponential was rounded, so
// the ranking is that of 64-bit arithmetic.  Doing it in 64 bits throughout would
// take the time of E double exponentials per token; instead keys are fp32 with
// a bound on their error.  Where groups at the border of those kept are nearer
// than their errors, their largest experts' keys are computed in 64 bits; where
// chosen keys are near one another or one left out, those are, one per lane; and
// only where too many are, all of them (about one token in two thousand needs any
// of it with random logits).  Equal logits with equal biases are equal in any
// arithmetic and need none of it; neither do logits that are keys themselves.
//
// Weights come from the logits of the chosen, in fp32.  Renormalised sigmoid
// weights are s_j / sum s with s_j = exp(l_j - m) / (1 + exp(l_j)), m = min(0,
// the largest l_j): the factor exp(-m) cancels, and nothing underflows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "../../include/tilegemm.h"
#include "host_common.h"

namespace tg {
namespace {

constexpr int kWarps = 4;          // per block
constexpr int kMaxExperts = 1024;

struct RouteParams {
    long long T;
    int E, k, groups, kept, top, size;  // size: experts per group
    int lanes, parts, run;              // of a token, of a group; experts of a lane
    int whole;                          // runs are whole, aligned 16-byte units
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
// e^x and 1 / x to within 2^-22 (and 2^-24 |x|) of themselves, for keys.
__device__ __forceinline__ float power(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// A double as an integer that orders alike, above 0 for everything but NaN, and back.
__device__ __forceinline__ unsigned long long ordered(double x) {
    const unsigned long long u = __double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double unordered(unsigned long long u) {
    return __longlong_as_double(u >> 63 ? u & ~(1ull << 63) : ~u);
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long x) {
    const unsigned high = warp_max((unsigned)(x >> 32));
    const unsigned low = warp_max((unsigned)(x >> 32) == high ? (unsigned)x : 0u);
    return (unsigned long long)high << 32 | low;
}

// What a token's keys in 64 bits need of its whole row, by its warp: a softmax's
// largest logit and sum of exponentials.
struct RowMass {
    float top;
    double sum;
};
template <class IN>
__device__ __noinline__ RowMass row_mass(const RouteParams& p, const IN* row, int lane) {
    RowMass r{-INFINITY, 0.0};
    if (p.sigmoid) return r;
    for (int e = lane; e < p.E; e += 32) r.top = fmaxf(r.top, load_one(row + e));
    r.top = warp_fmax(r.top);
    // (four at a time: a double operation's latency is far above its rate)
#pragma unroll 1
    for (int e0 = lane; e0 < p.E; e0 += 128) {
        double m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float l = e0 + 32 * j < p.E ? load_one(row + e0 + 32 * j) : -INFINITY;
            m[j] = !(l > -INFINITY) ? 0.0 : l == r.top ? 1.0 : exp((double)l - r.top);  // (of +inf: the limit)
        }
        r.sum += (m[0] + m[1]) + (m[2] + m[3]);
    }
    r.sum = warp_sum(r.sum);
    return r;
}
// An expert's score + bias in 64 bits.
__device__ __noinline__ double wide_key(const RouteParams& p, float l, float bias, RowMass r) {
    const double m = !p.sigmoid && l == r.top ? 1.0 : exp(p.sigmoid ? -(double)l : (double)l - r.top);
    return (p.sigmoid ? 1.0 / (1.0 + m) : m / r.sum) + (double)bias;
}

// One token ranked in 64 bits by its warp; keys: E words of shared memory.
// Returns, in lane j < k, its j-th expert or -1.  A double operation takes a warp
// 16 cycles of its SM's only unit, so every score is computed once and all
// comparisons are of integers.
template <class IN>
__device__ __noinline__ int rank_in_64_bits(const RouteParams& p, const IN* row, unsigned long long* keys, int lane) {
    const unsigned long long none = ordered(-(double)INFINITY);
    const bool by_score = p.bias || p.top == 2;  // a group's key
    const RowMass r = row_mass<IN>(p, row, lane);
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
        const float l = load_one(row + e);
        keys[e] = !(l > -INFINITY) ? none : ordered(by_score ? wide_key(p, l, p.bias ? p.bias[e] : 0.0f, r) : (double)l);
    }
    __syncwarp();
    unsigned kept = 0xffffffffu;
    if (p.groups > 1) {
        unsigned long long a = none, b = none;
        if (lane < p.groups)
            for (int i = 0; i < p.size; ++i) {
                const unsigned long long x = keys[lane * p.size + i];
                b = max(b, min(a, x));
                a = max(a, x);
            }
        const double value = p.top == 2 && b > none ? unordered(a) + unordered(b) : unordered(a);
        int ahead = 0;  // groups that come before this lane's
        for (int o = 0; o < p.groups; ++o) {
            const double v = __shfl_sync(0xffffffffu, value, o);
            ahead += v > value || (v == value && o < lane);
        }
        kept = __ballot_sync(0xffffffffu, ahead < p.kept && lane < p.groups);
        __syncwarp();
    }
    for (int e = lane; e < p.E; e += 32) {
        const float l = load_one(row + e);
        if (!(l > -INFINITY) || (p.groups > 1 && !(kept >> (e / p.size) & 1u)))
            keys[e] = 0;
        else if (!p.bias)
            keys[e] = ordered((double)l);
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        int at = 0;
        for (int e = lane; e < p.E; e += 32)
            if (keys[e] > best) {
                best = keys[e];
                at = e;
            }
        const unsigned long long winner = warp_max(best);
        if (winner == 0) break;
        const int e = (int)warp_min(best == winner ? (unsigned)at : 0xffffffffu);
        if (lane == j) mine = e;
        if (e % 32 == lane) keys[e] = 0;  // this lane's own
    }
    __syncwarp();
    return mine;
}

// Shared memory: the biases by lane and where each expert belongs, for the block;
// then per warp the keys (or one token's 64-bit keys), what is chosen (expert and
// key of each of the warp's 32 / lanes x k), and 33 words of candidates.
__host__ __device__ inline int block_words(int E, int C) { return 32 * C + (E + 1) / 2; }
__host__ __device__ inline int warp_words(int E, int C, int lanes, int k) {
    const int wide = 2 * E;
    return ((32 * C > wide ? 32 * C : wide) + 2 * (32 / lanes) * k + 33 + 3) & ~3;
}

inline int route_bytes(int E, int C, int lanes, int k) {
    return 4 * (((block_words(E, C) + 3) & ~3) + kWarps * warp_words(E, C, lanes, k));
}

// C: most experts of a lane.
template <class IN, int C, bool SIGMOID>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int Q = C / 4;
    extern __shared__ float4 shared_words[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = p.lanes, tokens = 32 / L;
    const int token = lane / (unsigned)L, in_token = lane & (L - 1);
    const unsigned of_token = (L == 32 ? 0xffffffffu : (1u << L) - 1u) << (token * L);
    // this lane's run of experts e0 .. e0 + n - 1, of group g
    const int g = in_token / (unsigned)p.parts, part = in_token - g * p.parts;
    const int e0 = g * p.size + part * p.run;
    const int n = g < p.groups ? min(p.run, p.size - part * p.run) : 0;
    // four keys q of a lane: neighbouring fours of a run lie in different banks
    auto four = [&](int q, int of_lane) { return q * 32 + ((of_lane + q) & 31); };
    float4* bias = shared_words;
    uint16_t* home = reinterpret_cast<uint16_t*>(bias + 32 * Q);  // of an expert: its lane and place in the run
    float* own_words = reinterpret_cast<float*>(shared_words) + ((block_words(p.E, C) + 3) & ~3) +
                       (size_t)warp * warp_words(p.E, C, L, p.k);
    float4* keys = reinterpret_cast<float4*>(own_words);
    int* candidates = reinterpret_cast<int*>(own_words) + warp_words(p.E, C, L, p.k) - 33;  // their number, and they
    int* chosen = candidates - 2 * tokens * p.k;
    float* chosen_key = reinterpret_cast<float*>(chosen + tokens * p.k);
    const bool by_score = p.bias || p.top == 2;  // a group's key
    const bool scores = p.bias || (p.groups > 1 && p.top == 2) || (!SIGMOID && !p.renorm);
    float largest_bias = 0.0f;
    if (p.bias || !p.whole) {
        for (int e = threadIdx.x; e < p.E; e += 32 * kWarps) {
            const float of_e = p.bias ? p.bias[e] : 0.0f;
            const int in = e / p.size, i = (e - in * p.size) / p.run, to = in * p.parts + i;
            const int at = e - in * p.size - i * p.run;
            home[e] = (uint16_t)(to << 8 | at);
            reinterpret_cast<float*>(&bias[four(at >> 2, to)])[at & 3] = of_e;
            largest_bias = fmaxf(largest_bias, fabsf(of_e));
        }
        // (of all warps' experts)
        largest_bias = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(largest_bias)));
        if (lane == 0) reinterpret_cast<float*>(keys)[0] = largest_bias;
        __syncthreads();
#pragma unroll
        for (int other = 0; other < kWarps; ++other)
            largest_bias = fmaxf(largest_bias, own_words[(other - warp) * warp_words(p.E, C, L, p.k)]);
        __syncthreads();
    }
    // Largest errors, absolute, over the row's largest score: of a sigmoid (its
    // exponential's argument x is off by 2^-24 |x| and its value by 2^-22, times
    // a slope s (1 - s); sum and quotient 2^-23), of a softmax's share (the same
    // where it is large, and a sum of up to 23 steps); and of a rounded sum of score and bias.
    const float kScoreError = SIGMOID ? 0x1p-21f : 0x1p-19f;
    constexpr float kSumError = 0x1p-23f;
    auto token_max = [&](float x) {
#pragma unroll
        for (int d = 1; d < 32; d *= 2)
            if (d < L) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        return x;
    };
    auto token_sum = [&](float x) {
#pragma unroll
        for (int d = 1; d < 32; d *= 2)
            if (d < L) x += __shfl_xor_sync(0xffffffffu, x, d);
        return x;
    };
    // a lane's run, four experts at a time
    const int fours = (p.run + 3) >> 2;
    auto each = [&](auto f) {
#pragma unroll 4
        for (int q = 0; q < fours; ++q) f(q, keys[four(q, lane)]);
    };
    const float4 nothing = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    for (long long first = ((long long)blockIdx.x * kWarps + warp) * tokens; first < p.T;
         first += (long long)gridDim.x * kWarps * tokens) {
        const long long t = first + token;  // may lie behind the last one
        const IN* row = static_cast<const IN*>(p.logits) + (t < p.T ? t : first) * p.ld;
        // logits; -inf where nothing is to be chosen
        float top = -INFINITY, sum = 1.0f;
        bool spoilt = false;
        auto checked = [&](float x) {
            spoilt |= !(x < INFINITY);  // NaN or +inf
            x = x == x ? x : -INFINITY;
            top = fmaxf(top, x);
            return x;
        };
        if (p.whole) {
            constexpr int kUnit = 16 / sizeof(IN);
#pragma unroll 4
            for (int i = 0; i < p.run; i += kUnit) {
                if (n == 0) {
                    for (int j = 0; j < kUnit; j += 4) keys[four((i + j) >> 2, lane)] = nothing;
                    continue;
                }
                const uint4 u = *reinterpret_cast<const uint4*>(row + e0 + i);
                const IN* v = reinterpret_cast<const IN*>(&u);
#pragma unroll
                for (int j = 0; j < kUnit; j += 4)
                    keys[four((i + j) >> 2, lane)] = make_float4(checked(load_one(v + j)), checked(load_one(v + j + 1)),
                                                                 checked(load_one(v + j + 2)), checked(load_one(v + j + 3)));
            }
        } else {
            for (int of = 0; of < tokens && first + of < p.T; ++of) {
                const IN* from = static_cast<const IN*>(p.logits) + (first + of) * p.ld;
#pragma unroll 4
                for (int e = lane; e < p.E; e += 32) {
                    const int h = home[e], i = h & 255;
                    reinterpret_cast<float*>(&keys[four(i >> 2, of * L + (h >> 8))])[i & 3] = load_one(from + e);
                }
            }
            __syncwarp();
            each([&](int q, float4 v) {
                v.x = 4 * q < n ? checked(v.x) : -INFINITY;
                v.y = 4 * q + 1 < n ? checked(v.y) : -INFINITY;
                v.z = 4 * q + 2 < n ? checked(v.z) : -INFINITY;
                v.w = 4 * q + 3 < n ? checked(v.w) : -INFINITY;
                keys[four(q, lane)] = v;
            });
        }
        spoilt = (__ballot_sync(0xffffffffu, spoilt) & of_token) != 0;
        if (scores && !SIGMOID) {
            top = token_max(top);
            sum = 0.0f;
            // (of +inf: the limit)
            auto mass = [&](float x) { return x == -INFINITY ? 0.0f : x == top ? 1.0f : expf(x - top); };
            each([&](int, float4 v) { sum += (mass(v.x) + mass(v.y)) + (mass(v.z) + mass(v.w)); });
            sum = token_sum(sum);
        }
        const float inverse = 1.0f / sum;
        auto score = [&](float x) {
            return SIGMOID ? reciprocal(1.0f + power(-x)) : x == top ? inverse : expf(x - top) * inverse;
        };
        // of one key
        const float error = (kScoreError + kSumError) * (SIGMOID ? 1.0f : inverse) + kSumError * largest_bias + 1e-30f;
        // the largest two of the lane's keys (without a bias: logits, which order as scores do)
        float one = -INFINITY, two = -INFINITY;
        auto rank = [&](float v) {
            two = fmaxf(two, fminf(one, v));
            one = fmaxf(one, v);
        };
        if (p.bias) {
            each([&](int q, float4 v) {
                const float4 c = bias[four(q, in_token)];
                v.x = v.x == -INFINITY ? v.x : score(v.x) + c.x;
                v.y = v.y == -INFINITY ? v.y : score(v.y) + c.y;
                v.z = v.z == -INFINITY ? v.z : score(v.z) + c.z;
                v.w = v.w == -INFINITY ? v.w : score(v.w) + c.w;
                keys[four(q, lane)] = v;
                rank(v.x), rank(v.y), rank(v.z), rank(v.w);
            });
        } else if (p.groups > 1) {
            each([&](int, float4 v) { rank(v.x), rank(v.y), rank(v.z), rank(v.w); });
        }
        bool wide = false;  // only 64 bits throughout can tell
        bool kept = true;
        if (p.groups > 1) {
            // a group's lanes one after another: every lane gets its group's two largest
            auto of_group = [&](auto& a, auto& b) {
                auto x = a, y = a;
                x = y = -INFINITY;
                for (int o = 0; o < p.parts; ++o) {
                    const int from = (token * L + g * p.parts + o) & 31;
                    const auto v1 = __shfl_sync(0xffffffffu, a, from), v2 = __shfl_sync(0xffffffffu, b, from);
                    const auto low = x < v1 ? x : v1, high = y > v2 ? y : v2;
                    y = high > low ? high : low;
                    x = x > v1 ? x : v1;
                }
                a = g < p.groups ? x : -INFINITY;
                b = g < p.groups ? y : -INFINITY;
            };
            of_group(one, two);
            auto value_of = [&](auto a, auto b) { return p.top == 2 && b > -INFINITY ? a + b : a; };
            const bool by_two_scores = !p.bias && p.top == 2;
            float value = !by_two_scores || one == -INFINITY ? value_of(one, two)
                                                             : value_of(score(one), two == -INFINITY ? two : score(two));
            // (the sum of two finite keys may lie outside fp32's range; a group without any keeps -inf)
            if (fabsf(one) < INFINITY) value = fmaxf(fminf(value, FLT_MAX), -FLT_MAX);
            auto is_kept = [&](auto value) {
                int ahead = 0;  // groups that come before this lane's
                for (int o = 0; o < p.groups; ++o) {
                    const auto v = __shfl_sync(0xffffffffu, value, token * L + o * p.parts);
                    ahead += v > value || (v == value && o < g);
                }
                return ahead < p.kept;
            };
            kept = is_kept(value);
            // the least of those kept and the best of those not are what decides
            const float least = -token_max(kept && n > 0 ? -value : -INFINITY), best = token_max(kept || n == 0 ? -INFINITY : value);
            bool near = by_score && least - best <= 4.0f * error;  // (no number if nothing is left in them)
            if (by_two_scores && __any_sync(0xffffffffu, near)) {
                // groups with the same two logits are equal in any arithmetic
                bool different = false;
                for (int o = 0; o < p.groups; ++o) {
                    const int from = token * L + o * p.parts;
                    const float v = __shfl_sync(0xffffffffu, value, from), v1 = __shfl_sync(0xffffffffu, one, from);
                    const float v2 = __shfl_sync(0xffffffffu, two, from);
                    const bool other = __shfl_sync(0xffffffffu, (int)kept, from) == 0;
                    different |= kept && other && value - v <= 4.0f * error && !(v1 == one && v2 == two);
                }
                const unsigned unlike = __ballot_sync(0xffffffffu, different);
                near = near && (unlike & of_token) != 0;
            }
            for (unsigned left = __ballot_sync(0xffffffffu, near); left;) {
                const int of = (__ffs(left) - 1) / (unsigned)L;
                left &= ~((L == 32 ? 0xffffffffu : (1u << L) - 1u) << (of * L));
                const RowMass r = row_mass<IN>(p, static_cast<const IN*>(p.logits) + (first + of < p.T ? first + of : first) * p.ld, lane);
                // the experts that may be among their groups' largest, one per lane, in 64 bits
                if (lane == 0) candidates[0] = 0;
                __syncwarp();
                if (token == of && one > -INFINITY) {
                    const float limit = (p.top == 2 ? two : one) - (p.bias ? 2.0f * error : 0.0f);
                    each([&](int q, float4 v) {
                        const float x[4] = {v.x, v.y, v.z, v.w};
                        for (int i = 0; i < 4; ++i)
                            if (4 * q + i < n && x[i] > -INFINITY && x[i] >= limit) {
                                const int at = atomicAdd(candidates, 1);
                                if (at < 32) candidates[1 + at] = e0 + 4 * q + i;
                            }
                    });
                }
                __syncwarp();
                const int number = candidates[0];
                if (number > 32) {
                    wide |= token == of;
                    __syncwarp();
                    continue;
                }
                const int e = lane < number ? candidates[1 + lane] : 0;
                const IN* its_row = static_cast<const IN*>(p.logits) + (first + of < p.T ? first + of : first) * p.ld;
                const double key = lane < number ? wide_key(p, load_one(its_row + e), p.bias ? p.bias[e] : 0.0f, r) : -INFINITY;
                double a = -INFINITY, b = -INFINITY;
                for (int o = 0; o < number; ++o) {
                    const double v = __shfl_sync(0xffffffffu, key, o);
                    const int its_e = __shfl_sync(0xffffffffu, e, o);
                    if (n == 0 || its_e < e0 || its_e >= e0 + n) continue;  // another lane's
                    b = v > a ? a : v > b ? v : b;
                    a = v > a ? v : a;
                }
                __syncwarp();
                of_group(a, b);
                const bool now = is_kept(value_of(a, b));
                if (token == of) kept = now;
            }
            wide = (__ballot_sync(0xffffffffu, wide) & of_token) != 0;
        }
        // k times the largest left; of equal ones the lane's first, and the first lane's
        float most[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            most[q] = -INFINITY;
            if (kept && 4 * q < n && t < p.T) {
                const float4 v = keys[four(q, lane)];
                most[q] = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
            }
        }
        float last = -INFINITY;
        int found = 0;
        auto largest = [&]() {
            float m = most[0];
#pragma unroll
            for (int q = 1; q < Q; ++q) m = fmaxf(m, most[q]);
            return m;
        };
#pragma unroll 1
        for (int j = 0; j < p.k; ++j) {
            const float own = largest();
            const float winner = token_max(own);
            const unsigned equal = __ballot_sync(0xffffffffu, own == winner) & of_token;
            last = winner;
            if (winner == -INFINITY) continue;
            ++found;
            if (lane != __ffs(equal) - 1) continue;
            int q = Q - 1;
#pragma unroll
            for (int c = Q - 2; c >= 0; --c) q = most[c] == winner ? c : q;
            float4 v = keys[four(q, lane)];
            const int i = v.x == winner ? 0 : v.y == winner ? 1 : v.z == winner ? 2 : 3;
            v.x = i == 0 ? -INFINITY : v.x;
            v.y = i == 1 ? -INFINITY : v.y;
            v.z = i == 2 ? -INFINITY : v.z;
            v.w = i == 3 ? -INFINITY : v.w;
            keys[four(q, lane)] = v;
            const float rest = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
#pragma unroll
            for (int c = 0; c < Q; ++c) most[c] = c == q ? rest : most[c];
            chosen[token * p.k + j] = e0 + 4 * q + i;
            chosen_key[token * p.k + j] = winner;
        }
        __syncwarp();
        const int* mine = chosen + token * p.k;
        if (p.bias) {
            // whether neighbours in the order, or a key left out and the last, are nearer
            // than the errors and not the same logit and bias
            auto same = [&](int c, int d) { return load_one(row + c) == load_one(row + d) && p.bias[c] == p.bias[d]; };
            bool near = false;
            const float* value = chosen_key + token * p.k;
            for (int j = in_token; j + 1 < found; j += L)
                if (value[j] - value[j + 1] <= 2.0f * error) near |= !same(mine[j], mine[j + 1]);
            const bool reached = found == p.k && largest() + 2.0f * error >= last;  // by a key left out
            auto left_out = [&](auto f) {
                if (!reached) return;
                each([&](int q, float4 v) {
                    const float x[4] = {v.x, v.y, v.z, v.w};
                    for (int i = 0; i < 4; ++i)
                        if (4 * q + i < n && x[i] > -INFINITY && x[i] + 2.0f * error >= last) f(e0 + 4 * q + i);
                });
            };
            if (kept) left_out([&](int e) { near |= !same(e, mine[p.k - 1]); });
            for (unsigned left = __ballot_sync(0xffffffffu, near && t < p.T); left;) {
                const int of = (__ffs(left) - 1) / (unsigned)L;
                left &= ~((L == 32 ? 0xffffffffu : (1u << L) - 1u) << (of * L));
                const IN* its_row = static_cast<const IN*>(p.logits) + (first + of) * p.ld;
                // what is chosen and what is near the last of it, one per lane, in 64 bits
                const int its_found = __shfl_sync(0xffffffffu, found, of * L);
                int* its_chosen = chosen + of * p.k;
                if (lane < its_found) candidates[1 + lane] = its_chosen[lane];
                if (lane == 0) candidates[0] = its_found;
                __syncwarp();
                if (token == of && kept) left_out([&](int e) {
                    const int at = atomicAdd(candidates, 1);
                    if (at < 32) candidates[1 + at] = e;
                });
                __syncwarp();
                const int number = candidates[0];
                if (number > 32) {
                    wide |= token == of;
                    __syncwarp();
                    continue;
                }
                const RowMass r = row_mass<IN>(p, its_row, lane);
                const int e = lane < number ? candidates[1 + lane] : p.E;
                const unsigned long long key = lane < number ? ordered(wide_key(p, load_one(its_row + e), p.bias[e], r)) : 0ull;
                int ahead = 0;
                for (int o = 0; o < number; ++o) {
                    const unsigned long long other = __shfl_sync(0xffffffffu, key, o);
                    const int other_e = __shfl_sync(0xffffffffu, e, o);
                    ahead += other > key || (other == key && other_e < e);
                }
                if (lane < number && ahead < its_found) its_chosen[ahead] = e;
                __syncwarp();
            }
        }
        for (unsigned left = __ballot_sync(0xffffffffu, wide && t < p.T); left;) {
            const int of = (__ffs(left) - 1) / (unsigned)L;
            left &= ~((L == 32 ? 0xffffffffu : (1u << L) - 1u) << (of * L));
            const int e = rank_in_64_bits<IN>(p, static_cast<const IN*>(p.logits) + (first + of) * p.ld,
                                              reinterpret_cast<unsigned long long*>(keys), lane);
            if (lane < p.k) chosen[of * p.k + lane] = e;
            const int all = __popc(__ballot_sync(0xffffffffu, lane < p.k && e >= 0));
            if (token == of) found = all;  // (other groups may hold fewer experts that can be chosen)
            __syncwarp();
        }
        // weights: a lane takes every L-th of its token's
        float m = -INFINITY, total = 0.0f;
        auto form = [&](float logit) {  // a sigmoid's are exp(-m) too large, with one m for all
            return !SIGMOID ? expf(logit - m) : logit > 0.0f ? sigmoid(logit) : expf(logit - m) / (1.0f + expf(logit));
        };
        if (p.renorm) {
            for (int j = in_token; j < found; j += L) m = fmaxf(m, load_one(row + mine[j]));
            m = token_max(m);
            if (SIGMOID) m = fminf(m, 0.0f);
            for (int j = in_token; j < found; j += L) total += form(load_one(row + mine[j]));
            total = token_sum(total);
        }
        if (t < p.T) {
            for (int j = in_token; j < p.k; j += L) {
                int e = -1;
                float w = 0.0f;
                if (j < found) {
                    e = mine[j];
                    const float logit = load_one(row + e);
                    w = p.renorm ? form(logit) / total : SIGMOID ? sigmoid(logit) : expf(logit - top) / sum;
                    if (!SIGMOID && spoilt) w = NAN;
                }
                p.index[t * p.k + j] = e;
                p.weight[t * p.k + j] = w * p.scale;
            }
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
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const __grid_constant__ RouteParams p) {
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
        float d, dot = 0.0f, own = 0.0f;  // own: the softmax's share of this lane's expert
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
            own = e >= 0 ? expf(logit - base) * inverse : 0.0f;
            dot = warp_sum(e >= 0 ? g * own : 0.0f);
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
        // what is not chosen, and then what is: an expert's first lane stores its sum
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int x = v * 32 + lane;
            if (x < p.E) store_one(out + x, dense ? prob[v] * -dot : 0.0f);
        }
        float sum = 0.0f;
        bool first = e >= 0;
        for (int j = 0; j < p.k; ++j) {
            const int other = __shfl_sync(0xffffffffu, e, j);
            const float x = __shfl_sync(0xffffffffu, d, j);
            if (other == e) sum += x;
            if (other == e && j < lane) first = false;
        }
        __syncwarp();  // (the stores above come before)
        if (first) store_one(out + e, dense ? own * (sum - dot) : sum);
    }
}

template <class IN, int V>
cudaError_t launch_grad(const RouteParams& p, int sms, cudaStream_t stream) {
    const long long blocks = (p.T + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(blocks < 16LL * sms ? blocks : 16LL * sms);
    route_grad_kernel<IN, V><<<grid, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

template <class IN, int C>
cudaError_t launch_route(const RouteParams& p, int sms, cudaStream_t stream) {
    const long long per_block = (long long)kWarps * (32 / p.lanes), blocks = (p.T + per_block - 1) / per_block;
    // about as many as are resident: what a warp sets up is shared by its tokens
    const unsigned grid = (unsigned)(blocks < 6LL * sms ? blocks : 6LL * sms);
    const int bytes = route_bytes(p.E, C, p.lanes, p.k);
    auto kern = p.sigmoid ? route_kernel<IN, C, true> : route_kernel<IN, C, false>;
    if (bytes > 48 * 1024) {
        // (what any call may want: another thread's may be on its way)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   route_bytes(kMaxExperts, C, 1, 32));
        if (e != cudaSuccess) return e;
    }
    kern<<<grid, 32 * kWarps, bytes, stream>>>(p);
    return cudaGetLastError();
}

template <class IN>
cudaError_t launch_typed(const RouteParams& p, bool grad, int sms, cudaStream_t stream) {
    if (!grad) {
        if (p.run <= 8) return launch_route<IN, 8>(p, sms, stream);
        if (p.run <= 16) return launch_route<IN, 16>(p, sms, stream);
        if (p.run <= 32) return launch_route<IN, 32>(p, sms, stream);
        return launch_route<IN, 64>(p, sms, stream);
    }
    if (p.E <= 32) return launch_grad<IN, 1>(p, sms, stream);
    if (p.E <= 64) return launch_grad<IN, 2>(p, sms, stream);
    if (p.E <= 128) return launch_grad<IN, 4>(p, sms, stream);
    if (p.E <= 256) return launch_grad<IN, 8>(p, sms, stream);
    if (p.E <= 512) return launch_grad<IN, 16>(p, sms, stream);
    return launch_grad<IN, 32>(p, sms, stream);
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
    // Short runs while every token finds a warp of its own at once (one token of 256
    // experts: 6.8 us in runs of 8, 9.7 of 32), then of at most 32 experts, or of 64: with
    // that 32 lanes hold any 1024 experts in 32 groups.
    for (int most = T <= 2048 ? 8 : 32; most <= 64; most *= 2) {
        p.parts = (p.size + most - 1) / most;
        if (p.groups * p.parts <= 32) break;
    }
    p.run = (p.size + p.parts - 1) / p.parts;
    p.lanes = 1;
    while (p.lanes < p.groups * p.parts) p.lanes *= 2;
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
    p.whole = aligned16(logits) && ld * size % 16 == 0 && p.size * size % 16 == 0 && p.run * size % 16 == 0 && p.size % p.run == 0;
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
