// layernorm.cu -- layer norm and its gradient (tg_layernorm,
// tg_layernorm_grad).
//
//   xh = (x - mean) rstd      y = xh w + b
//   g = dy w;  dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh;  db = sum over rows of dy
//
// Both are bound by memory: every element is read once and written once.  A
// row stays in registers between its two reductions (mean, then squared
// differences from it: no cancellation), held by one warp up to 512 columns
// and by a team of up to 16 warps beyond.  Statistics and sums are fp32.
//
// Rows of whole 16-byte units come through a ring in shared memory: a team
// walks over rows while bulk copies bring the next ones, so that loads never
// wait for a reduction's barrier (16384 x 4096 in bf16: forward 47.3 us, 5.7
// TB/s, backward 62.5 us, 6.4 TB/s, and 7 of reduction).  So do long rows of
// other widths or alignments (16384 x 4095: forward 57.6 us, backward 89).
// Short ones are loaded by element or by pair into registers, and rows too long
// for registers are read again from L2 in chunks (wide kernels; 2000 x 32768:
// forward 74 us, 3.6 TB/s, backward 237 us, whose accesses are single elements).
//
// The gradient's blocks walk over rows and keep their columns' dw and db in
// fp32 registers; one partial row per block goes to the workspace and a second
// kernel adds them in a fixed order, so results repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstring>
#include <initializer_list>

#include "../../include/tilegemm.h"
#include "chained.cuh"
#include "gemm_params.h"
#include "host_common.h"
#include "packed.cuh"
#include "ptx.cuh"
#include "ring.cuh"
#include "stage.cuh"

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

// A pack from p; `left` elements of the row start there.  Packs of rows that
// are not aligned to them (WHOLE = false) are read element by element, zeros
// past the end; whole packs lie inside the row or outside.
template <int VEC, bool WHOLE>
__device__ __forceinline__ Pack<VEC> load(const uint16_t* p, int left) {
    Pack<VEC> v{};
    if constexpr (!WHOLE) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (k < left) v.e[k] = __ldg(p + k);
    } else if (left > 0) {
        if constexpr (VEC == 8)
            *reinterpret_cast<uint4*>(&v) = __ldg(reinterpret_cast<const uint4*>(p));
        else
            *reinterpret_cast<uint32_t*>(&v) = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
    return v;
}
template <int VEC, bool WHOLE>
__device__ __forceinline__ void store(uint16_t* p, int left, const Pack<VEC>& v) {
    if constexpr (!WHOLE) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (k < left) p[k] = v.e[k];
    } else if (left > 0) {
        *reinterpret_cast<Pack<VEC>*>(p) = v;
    }
}

// Sums of N values over the WARPS warps that share a row (0: the block's, up to
// 16); every thread gets them.  `buf` has room for N * row_slots(WARPS) floats and
// alternates between calls, so one barrier per call is enough.
__host__ __device__ constexpr int row_slots(int warps) { return warps ? warps : 16; }
template <int N, int WARPS>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (WARPS != 1) {
        constexpr int SLOTS = row_slots(WARPS);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int warps = WARPS ? WARPS : (int)blockDim.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) buf[k * SLOTS + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float x = lane < warps ? buf[k * SLOTS + lane] : 0.0f;
#pragma unroll
            for (int o = SLOTS / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
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
    float* part;  // gradient: [blocks][2][pitch]
    int pitch;
    int stages;   // ring: rows in flight per team
    const uint16_t *x_end, *dy_end;  // ring: ends of x and dy
    long long timeout_cycles;
    int* status;
};

template <bool BF>
__device__ __forceinline__ f2 widen2(const uint16_t* e) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(e);
    if constexpr (BF) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pair(f.x, f.y);
}
template <bool BF>
__device__ __forceinline__ uint32_t narrow2(f2 a) {
    const float2 f = split(a);
    uint32_t w;
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        w = *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        w = *reinterpret_cast<const uint32_t*>(&h);
    }
    return w;
}

// ------------------------------------------------------------- row ring
//
// Rows of whole 16-byte packs travel through shared memory: each team of
// warps (one row at a time) keeps `stages` rows in flight as bulk copies,
// counted on one mbarrier per stage.  Loads into registers keep at most 32 KB
// per SM in flight here, since a thread's columns also hold its weights and
// sums, and memory's latency times its rate is about 50 KB per SM.
constexpr int kMaxStages = 8;

// Rows of other widths or alignments (SHIFT).  A team walks over rows by a
// multiple of 8, so where its rows start within 16 bytes is the same for all of
// them, whatever the stride.  Its threads take windows of 8 columns that are
// aligned in the *output*, whose stores are then whole; the weights are loaded
// once, at that shift.  A stage holds the aligned 16-byte units around a row,
// and a window is funnelled out of two of them (by 15 selects and shifts; none
// where input and output are shifted alike).  The columns before the first
// window and after the last, 14 at most, are taken one each by the team's last
// threads.  (Windows over the row's ends instead, with what lies outside masked:
// 64 us for 16384 x 4089 where whole rows of 4096 took 53; the masks and element
// stores of two warps held up the row's barriers.)
__host__ __device__ constexpr uint32_t stage_bytes(bool shift, int cols) {
    return shift ? (((uint32_t)cols + 14) / 8 + 1) * 16 : (uint32_t)cols * 2;
}

// Where a thread's columns are.
struct Columns {
    int front;    // columns before the first window
    int end;      // end of the last window
    int extra;    // the thread's single column, or -1
};
template <bool SHIFT>
__device__ __forceinline__ Columns columns_of(const uint16_t* out, int cols, int tid, int width) {
    if constexpr (!SHIFT) return {0, cols, -1};
    Columns c;
    c.front = min(-shift_of(out) & 7, cols);
    c.end = c.front + ((cols - c.front) & ~7);
    const int k = width - 1 - tid, e = k < c.front ? k : c.end + k - c.front;
    c.extra = e < cols ? e : -1;
    return c;
}

// 8 columns of the weights or the bias from `c`.
template <bool SHIFT>
__device__ __forceinline__ Pack<8> load_columns(const uint16_t* p, int c, int end) {
    if constexpr (!SHIFT) return load<8, true>(p + c, end - c);
    Pack<8> v{};
    if (c >= end) return v;
    const uintptr_t unit = reinterpret_cast<uintptr_t>(p + c) & ~uintptr_t(15);
    if (unit + 32 <= reinterpret_cast<uintptr_t>(p + end)) {
        *reinterpret_cast<uint4*>(&v) = load_shifted(p + c);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.e[j] = __ldg(p + c + j);
    }
    return v;
}

// WARPS warps per row, NV packs of VEC elements per thread.
constexpr int kRowsPerBlock = 4;  // rows of a block whose rows take one warp each
constexpr int row_threads(int warps) { return 32 * (warps == 1 ? kRowsPerBlock : warps); }

// A row in registers, or (WIDE) read again from memory for each pass, which
// finds most of it in L2.
template <bool BF, int VEC, bool WHOLE, int WARPS, int NV, bool WIDE>
__global__ void __launch_bounds__(row_threads(WARPS))
ln_forward_kernel(const LnParams p) {
    __shared__ float buf[2][WARPS == 1 ? 1 : WARPS];
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    constexpr int kThreads = 32 * WARPS, kStep = kThreads * VEC, PAIRS = VEC / 2;
    const long long row = WARPS == 1 ? (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5)
                                     : (long long)blockIdx.x;
    if (row >= p.rows) return;
    const uint16_t* x = p.x + row * p.ldx;
    uint16_t* y = p.out + row * p.ldo;
    const int chunks = WIDE ? (p.cols + kStep * NV - 1) / (kStep * NV) : 1;
    auto column = [&](int chunk, int i) { return (chunk * NV + i) * kStep + tid * VEC; };
    Pack<VEC> v[NV];
    auto fetch = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(chunk, i);
            v[i] = load<VEC, WHOLE>(x + c, p.cols - c);
        }
    };
    f2 acc = pair(0.0f, 0.0f);
    for (int k = 0; k < chunks; ++k) {
        fetch(k);
#pragma unroll
        for (int i = 0; i < NV; ++i)  // zeros past the row's end
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) acc = add(acc, widen2<BF>(v[i].e + 2 * j));
    }
    float2 a = split(acc);
    float sum[1] = {a.x + a.y};
    row_sum<1, WARPS>(sum, buf[0]);
    const float mean = sum[0] / (float)p.cols;
    const f2 minus = pair(-mean, -mean);
    acc = pair(0.0f, 0.0f);
    for (int k = 0; k < chunks; ++k) {
        if (WIDE) fetch(k);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int left = p.cols - column(k, i);
            if (WHOLE && left <= 0) continue;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                f2 d = add(widen2<BF>(v[i].e + 2 * j), minus);
                if (!WHOLE && 2 * j + 1 >= left)
                    d = pair(2 * j < left ? split(d).x : 0.0f, 0.0f);
                acc = fma(d, d, acc);
            }
        }
    }
    a = split(acc);
    float sq[1] = {a.x + a.y};
    row_sum<1, WARPS>(sq, buf[1]);
    const float rstd = 1.0f / sqrtf(sq[0] / (float)p.cols + p.eps);
    if (tid == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
    }
    const f2 scale = pair(rstd, rstd);
    for (int k = 0; k < chunks; ++k) {
        if (WIDE) fetch(k);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(k, i), left = p.cols - c;
            if (left <= 0) continue;
            const Pack<VEC> w = load<VEC, WHOLE>(p.weight + c, left);
            Pack<VEC> b{};
            if (p.bias) b = load<VEC, WHOLE>(p.bias + c, left);
            Pack<VEC> o;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const f2 xh = mul(add(widen2<BF>(v[i].e + 2 * j), minus), scale);
                const uint32_t word =
                    narrow2<BF>(fma(xh, widen2<BF>(w.e + 2 * j), widen2<BF>(b.e + 2 * j)));
                *reinterpret_cast<uint32_t*>(o.e + 2 * j) = word;
            }
            store<VEC, WHOLE>(y + c, left, o);
        }
    }
}

// The forward pass through the ring: teams walk over rows.
// (1024 threads per SM with 64 registers each: 49.5 us against 47.6.)
constexpr int forward_threads(int nv) { return nv == 4 ? 512 : 768; }  // per SM
constexpr int most_threads(int warps) { return warps ? row_threads(warps) : 512; }
template <bool BF, int WARPS, int NV, bool SHIFT>
__global__ void __launch_bounds__(most_threads(WARPS), forward_threads(NV) / most_threads(WARPS))
ln_forward_ring_kernel(const LnParams p) {
    constexpr int VEC = 8, PAIRS = VEC / 2, kTeams = WARPS == 1 ? kRowsPerBlock : 1;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float buf[2][row_slots(WARPS)];
    __shared__ uint64_t full[kTeams][kMaxStages];
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int width = WARPS ? 32 * WARPS : (int)blockDim.x;  // threads of a team
    const int team = WARPS == 1 ? threadIdx.x >> 5 : 0;
    const uint32_t bytes = stage_bytes(SHIFT, p.cols);
    uint8_t* stages = ring + (size_t)team * p.stages * bytes;
    if (threadIdx.x < kTeams * kMaxStages) {
        mbar_init(smem_addr(&full[0][0] + threadIdx.x), 1);
        fence_barrier_init();  // of this thread's barrier
    }
    __syncthreads();
    const long long first = (long long)blockIdx.x * kTeams + team, step = (long long)gridDim.x * kTeams;
    auto issue = [&](long long row, int st) {
        const uint32_t bar = smem_addr(&full[team][st]);
        uint8_t* dst = stages + st * bytes;
        if constexpr (SHIFT) {
            const RowCopy x = row_copy(dst, p.x + row * p.ldx, p.x_end, p.cols);
            mbar_arrive_expect_tx(bar, x.bytes);
            if (x.bytes) bulk_load(smem_addr(dst), x.src, x.bytes, bar);
        } else {
            mbar_arrive_expect_tx(bar, bytes);
            bulk_load(smem_addr(dst), p.x + row * p.ldx, bytes, bar);
        }
    };
    if (tid == 0)
        for (int st = 0; st < p.stages && first + st * step < p.rows; ++st) issue(first + st * step, st);
    const Columns at = columns_of<SHIFT>(p.out + first * p.ldo, p.cols, tid, width);
    const int x_shift = SHIFT ? shift_of(p.x + first * p.ldx) : 0;
    Pack<VEC> w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = at.front + (i * width + tid) * VEC;
        w[i] = load_columns<SHIFT>(p.weight, c, at.end);
        b[i] = Pack<VEC>{};
        if (p.bias) b[i] = load_columns<SHIFT>(p.bias, c, at.end);
    }
    float we = 0.0f, be = 0.0f;  // of the single column
    if (SHIFT && at.extra >= 0) {
        we = widen<BF>(__ldg(p.weight + at.extra));
        if (p.bias) be = widen<BF>(__ldg(p.bias + at.extra));
    }
    int st = 0;
    uint32_t phase = 0;
    for (long long row = first; row < p.rows; row += step) {
        if (!stage_ready(smem_addr(&full[team][st]), phase, p.timeout_cycles, p.status)) return;
        f2 v[NV][PAIRS], acc = pair(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at.front + (i * width + tid) * VEC;
            Pack<VEC> x{};
            if (c < at.end) {
                if constexpr (SHIFT)
                    *reinterpret_cast<uint4*>(&x) =
                        window(stages + st * bytes, i * width + tid, x_shift + at.front);
                else
                    x = *reinterpret_cast<const Pack<VEC>*>(stages + st * bytes + c * 2);
            }
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                v[i][j] = widen2<BF>(x.e + 2 * j);
                acc = add(acc, v[i][j]);
            }
        }
        float2 a = split(acc);
        float sum[1] = {a.x + a.y};
        float ve = 0.0f;
        if (SHIFT && at.extra >= 0) {
            ve = widen<BF>(*reinterpret_cast<const uint16_t*>(stages + st * bytes + (x_shift + at.extra) * 2));
            sum[0] += ve;
        }
        row_sum<1, WARPS>(sum, buf[0]);
        // everyone has read the stage
        if constexpr (WARPS == 1) __syncwarp();
        if (tid == 0 && row + p.stages * step < p.rows) issue(row + p.stages * step, st);
        const float mean = sum[0] / (float)p.cols;
        const f2 minus = pair(-mean, -mean);
        acc = pair(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at.front + (i * width + tid) * VEC;
            if (c < at.end)
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    v[i][j] = add(v[i][j], minus);
                    acc = fma(v[i][j], v[i][j], acc);
                }
        }
        a = split(acc);
        float sq[1] = {a.x + a.y};
        if (SHIFT && at.extra >= 0) {
            ve -= mean;
            sq[0] = fmaf(ve, ve, sq[0]);
        }
        row_sum<1, WARPS>(sq, buf[1]);
        const float rstd = 1.0f / sqrtf(sq[0] / (float)p.cols + p.eps);
        if (tid == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
        const f2 scale = pair(rstd, rstd);
        uint16_t* y = p.out + row * p.ldo;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at.front + (i * width + tid) * VEC;
            if (c >= at.end) continue;
            Pack<VEC> o;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const uint32_t word = narrow2<BF>(fma(mul(v[i][j], scale), widen2<BF>(w[i].e + 2 * j),
                                                      widen2<BF>(b[i].e + 2 * j)));
                *reinterpret_cast<uint32_t*>(o.e + 2 * j) = word;
            }
            *reinterpret_cast<Pack<VEC>*>(y + c) = o;
        }
        if (SHIFT && at.extra >= 0) y[at.extra] = narrow<BF>(fmaf(ve * rstd, we, be));
        if (++st == p.stages) {
            st = 0;
            phase ^= 1;
        }
    }
}

// One partial row per block: [block][2][pitch]; rows that a block's warps took
// side by side are added in the order of the warps.  Column c is at c + lead, so
// that windows are whole 32-byte sectors (float by float at their stride, the
// stores of 304 blocks took 7 of 16384 x 4096's 78 us).  `dwe`, `dbe`:
// of a thread's single column.
__host__ __device__ constexpr int lead_of(int front) { return 8 - front; }
int pitch_of(int64_t cols) { return (int)(cdiv(cols + 8, 32) * 32); }  // whole lines for the sums
template <int VEC, int WARPS, int NV, bool SHIFT>
__device__ __forceinline__ void write_partials(const LnParams& p, const f2 (&dw)[NV][VEC / 2],
                                               const f2 (&db)[NV][VEC / 2], const Columns& at, float dwe,
                                               float dbe) {
    constexpr int PAIRS = VEC / 2;
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int group = WARPS == 1 ? threadIdx.x >> 5 : 0;
    float* part_w = p.part + (long long)blockIdx.x * 2 * p.pitch + (SHIFT ? lead_of(at.front) : 0);
    float* part_b = part_w + p.pitch;
    if constexpr (WARPS == 1) {
        __shared__ float2 part[kRowsPerBlock][32 * NV * PAIRS];
        for (int what = 0; what < 2; ++what) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < PAIRS; ++j)
                    part[group][(i * PAIRS + j) * 32 + tid] = split(what ? db[i][j] : dw[i][j]);
            __syncthreads();
            float* out = what ? part_b : part_w;
            for (int c = 2 * threadIdx.x; c < p.cols; c += 64 * kRowsPerBlock) {
                const int lane = c / VEC % 32, k = (c / (32 * VEC) * PAIRS + c % VEC / 2) * 32 + lane;
                float2 s = part[0][k];
#pragma unroll
                for (int y = 1; y < kRowsPerBlock; ++y) {
                    s.x += part[y][k].x;
                    s.y += part[y][k].y;
                }
                *reinterpret_cast<float2*>(out + c) = s;
            }
            __syncthreads();
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at.front + (i * (int)blockDim.x + tid) * VEC;
            if (c >= at.end) continue;
            if constexpr (VEC == 2) {
                *reinterpret_cast<float2*>(part_w + c) = split(dw[i][0]);
                *reinterpret_cast<float2*>(part_b + c) = split(db[i][0]);
            } else {
#pragma unroll
                for (int j = 0; j < PAIRS; j += 2) {
                    const float2 w0 = split(dw[i][j]), w1 = split(dw[i][j + 1]);
                    const float2 b0 = split(db[i][j]), b1 = split(db[i][j + 1]);
                    *reinterpret_cast<float4*>(part_w + c + 2 * j) = make_float4(w0.x, w0.y, w1.x, w1.y);
                    *reinterpret_cast<float4*>(part_b + c + 2 * j) = make_float4(b0.x, b0.y, b1.x, b1.y);
                }
            }
        }
        if (SHIFT && at.extra >= 0) {
            part_w[at.extra] = dwe;
            part_b[at.extra] = dbe;
        }
    }
}

// dx, and this block's partial sums of dw and db; 16 elements per thread, 512
// threads per SM with 128 registers each.  The next row's loads into registers
// are in flight while this row is reduced and written; xh and g stay in
// registers between the reduction and dx.  (Rows of whole pairs gain nothing
// from loading pairs: 16384 x 1500 in bf16 68 us, by elements 48.)
constexpr int kGradThreadsPerSm = 512;

template <bool BF, int WARPS, int NV>
__global__ void __launch_bounds__(row_threads(WARPS), kGradThreadsPerSm / row_threads(WARPS))
ln_backward_kernel(const LnParams p) {
    constexpr int VEC = 2, kStep = 32 * WARPS * VEC, PAIRS = VEC / 2;
    constexpr int kGroups = WARPS == 1 ? kRowsPerBlock : 1;  // rows in work at once
    __shared__ float buf[2][WARPS == 1 ? 1 : 2 * WARPS];
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int group = WARPS == 1 ? threadIdx.x >> 5 : 0;
    f2 dw[NV][PAIRS], db[NV][PAIRS];
    Pack<VEC> w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kStep + tid * VEC;
        w[i] = load<VEC, false>(p.weight + c, p.cols - c);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) dw[i][j] = db[i][j] = pair(0.0f, 0.0f);
    }
    allow_next_kernel();
    const float inv = 1.0f / (float)p.cols;
    const long long step = (long long)gridDim.x * kGroups;
    Pack<VEC> vx[NV], vd[NV], nx[NV], nd[NV];
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](long long row, Pack<VEC>(&x)[NV], Pack<VEC>(&d)[NV]) {
        const uint16_t* px = p.x + row * p.ldx;
        const uint16_t* pd = p.dy + row * p.lddy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * kStep + tid * VEC;
            x[i] = load<VEC, false>(px + c, p.cols - c);
            d[i] = load<VEC, false>(pd + c, p.cols - c);
        }
        mean = __ldg(p.mean + row);
        rstd = __ldg(p.rstd + row);
    };
    long long row = (long long)blockIdx.x * kGroups + group;
    if (row < p.rows) fetch(row, nx, nd);
    int flip = 0;
    for (; row < p.rows; row += step) {
        const float r = rstd;
        // x - mean first: scaled apart, the two would cancel with their roundings
        const f2 scale = pair(r, r), minus = pair(-mean, -mean);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            vx[i] = nx[i];
            vd[i] = nd[i];
        }
        if (row + step < p.rows) fetch(row + step, nx, nd);
        f2 s0 = pair(0.0f, 0.0f), s1 = s0;  // sums of g and of g xh
        f2 g[NV][PAIRS], xh[NV][PAIRS];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                // columns past the row's end hold zeros in dy and w: they add nothing
                const f2 d = widen2<BF>(vd[i].e + 2 * j);
                const f2 x = mul(add(widen2<BF>(vx[i].e + 2 * j), minus), scale);
                const f2 gg = mul(d, widen2<BF>(w[i].e + 2 * j));
                s0 = add(s0, gg);
                s1 = fma(gg, x, s1);
                dw[i][j] = fma(d, x, dw[i][j]);
                db[i][j] = add(db[i][j], d);
                xh[i][j] = x;
                g[i][j] = gg;
            }
        }
        const float2 a = split(s0), b = split(s1);
        float s[2] = {a.x + a.y, b.x + b.y};
        row_sum<2, WARPS>(s, buf[flip]);
        flip ^= 1;
        const float c1 = -r * s[0] * inv, c2 = -r * s[1] * inv;
        const f2 k1 = pair(c1, c1), k2 = pair(c2, c2);
        uint16_t* dx = p.out + row * p.ldo;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * kStep + tid * VEC;
            if (c >= p.cols) continue;
            Pack<VEC> o;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const uint32_t word = narrow2<BF>(fma(xh[i][j], k2, fma(g[i][j], scale, k1)));
                *reinterpret_cast<uint32_t*>(o.e + 2 * j) = word;
            }
            store<VEC, false>(dx + c, p.cols - c, o);
        }
    }
    write_partials<VEC, WARPS, NV, false>(p, dw, db, {0, p.cols, -1}, 0.0f, 0.0f);
}

// The same through the ring.  With 4 packs per thread, whose sums alone are 64
// registers, a row's stage is read twice, before and after its reduction, and
// filled again after the next row's barrier.
template <bool BF, int WARPS, int NV, bool SHIFT>
__global__ void __launch_bounds__(most_threads(WARPS), kGradThreadsPerSm / most_threads(WARPS))
ln_backward_ring_kernel(const LnParams p) {
    constexpr bool KEEP = NV < 4;
    constexpr int VEC = 8, PAIRS = VEC / 2, kTeams = WARPS == 1 ? kRowsPerBlock : 1;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float buf[2][2 * row_slots(WARPS)];
    __shared__ uint64_t full[kTeams][kMaxStages];
    const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int width = WARPS ? 32 * WARPS : (int)blockDim.x;  // threads of a team
    const int team = WARPS == 1 ? threadIdx.x >> 5 : 0;
    const uint32_t bytes = stage_bytes(SHIFT, p.cols);
    uint8_t* stages = ring + (size_t)team * p.stages * 2 * bytes;
    allow_next_kernel();
    if (threadIdx.x < kTeams * kMaxStages) {
        mbar_init(smem_addr(&full[0][0] + threadIdx.x), 1);
        fence_barrier_init();  // of this thread's barrier
    }
    __syncthreads();
    const long long first = (long long)blockIdx.x * kTeams + team, step = (long long)gridDim.x * kTeams;
    auto issue = [&](long long row, int st) {
        const uint32_t bar = smem_addr(&full[team][st]);
        uint8_t* dst = stages + st * 2 * bytes;
        if constexpr (SHIFT) {
            const RowCopy x = row_copy(dst, p.x + row * p.ldx, p.x_end, p.cols);
            const RowCopy d = row_copy(dst + bytes, p.dy + row * p.lddy, p.dy_end, p.cols);
            mbar_arrive_expect_tx(bar, x.bytes + d.bytes);
            if (x.bytes) bulk_load(smem_addr(dst), x.src, x.bytes, bar);
            if (d.bytes) bulk_load(smem_addr(dst + bytes), d.src, d.bytes, bar);
        } else {
            mbar_arrive_expect_tx(bar, 2 * bytes);
            bulk_load(smem_addr(dst), p.x + row * p.ldx, bytes, bar);
            bulk_load(smem_addr(dst + bytes), p.dy + row * p.lddy, bytes, bar);
        }
    };
    if (tid == 0)
        for (int st = 0; st < p.stages && first + st * step < p.rows; ++st) issue(first + st * step, st);
    const Columns at = columns_of<SHIFT>(p.out + first * p.ldo, p.cols, tid, width);
    const int x_shift = SHIFT ? shift_of(p.x + first * p.ldx) : 0;
    const int d_shift = SHIFT ? shift_of(p.dy + first * p.lddy) : 0;
    // x and dy of window i of a stage
    auto operands = [&](const uint8_t* sx, int i, int c, Pack<VEC>& vx, Pack<VEC>& vd) {
        if constexpr (SHIFT) {
            *reinterpret_cast<uint4*>(&vx) = window(sx, i * width + tid, x_shift + at.front);
            *reinterpret_cast<uint4*>(&vd) =
                window(sx + bytes, i * width + tid, d_shift + at.front);
        } else {
            vx = *reinterpret_cast<const Pack<VEC>*>(sx + c * 2);
            vd = *reinterpret_cast<const Pack<VEC>*>(sx + bytes + c * 2);
        }
    };
    float we = 0.0f, dwe = 0.0f, dbe = 0.0f;  // of the single column
    if (SHIFT && at.extra >= 0) we = widen<BF>(__ldg(p.weight + at.extra));
    f2 dw[NV][PAIRS], db[NV][PAIRS];
    Pack<VEC> w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = at.front + (i * width + tid) * VEC;
        w[i] = load_columns<SHIFT>(p.weight, c, at.end);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) dw[i][j] = db[i][j] = pair(0.0f, 0.0f);
    }
    const float inv = 1.0f / (float)p.cols;
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (first < p.rows) {
        next_mean = __ldg(p.mean + first);
        next_rstd = __ldg(p.rstd + first);
    }
    int st = 0, flip = 0;
    uint32_t phase = 0;
    for (long long row = first; row < p.rows; row += step) {
        const float r = next_rstd, mean = next_mean;
        if (row + step < p.rows) {
            next_mean = __ldg(p.mean + row + step);
            next_rstd = __ldg(p.rstd + row + step);
        }
        // x - mean first: scaled apart, the two would cancel with their roundings
        const f2 scale = pair(r, r), minus = pair(-mean, -mean);
        if (!stage_ready(smem_addr(&full[team][st]), phase, p.timeout_cycles, p.status)) return;
        const uint8_t* sx = stages + st * 2 * bytes;
        f2 s0 = pair(0.0f, 0.0f), s1 = s0;  // sums of g and of g xh
        f2 g[KEEP ? NV : 1][PAIRS], xh[KEEP ? NV : 1][PAIRS];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at.front + (i * width + tid) * VEC;
            Pack<VEC> vx{}, vd{};  // columns past the end add nothing
            if (c < at.end) operands(sx, i, c, vx, vd);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const f2 d = widen2<BF>(vd.e + 2 * j);
                const f2 x = mul(add(widen2<BF>(vx.e + 2 * j), minus), scale);
                const f2 gg = mul(d, widen2<BF>(w[i].e + 2 * j));
                s0 = add(s0, gg);
                s1 = fma(gg, x, s1);
                dw[i][j] = fma(d, x, dw[i][j]);
                db[i][j] = add(db[i][j], d);
                if (KEEP) {
                    xh[i][j] = x;
                    g[i][j] = gg;
                }
            }
        }
        const float2 a = split(s0), b = split(s1);
        float s[2] = {a.x + a.y, b.x + b.y};
        float xe = 0.0f, ge = 0.0f;
        if (SHIFT && at.extra >= 0) {
            const float d = widen<BF>(*reinterpret_cast<const uint16_t*>(sx + bytes + (d_shift + at.extra) * 2));
            xe = (widen<BF>(*reinterpret_cast<const uint16_t*>(sx + (x_shift + at.extra) * 2)) - mean) * r;
            ge = d * we;
            s[0] += ge;
            s[1] = fmaf(ge, xe, s[1]);
            dwe = fmaf(d, xe, dwe);
            dbe += d;
        }
        row_sum<2, WARPS>(s, buf[flip]);
        flip ^= 1;
        if constexpr (WARPS == 1) __syncwarp();
        if (tid == 0) {
            // KEEP: everyone has read this row's stage; else the one before's
            const long long done = KEEP ? row : row - step;
            const int slot = KEEP ? st : (st ? st - 1 : p.stages - 1);
            if (done >= first && done + p.stages * step < p.rows) issue(done + p.stages * step, slot);
        }
        const float c1 = -r * s[0] * inv, c2 = -r * s[1] * inv;
        const f2 k1 = pair(c1, c1), k2 = pair(c2, c2);
        uint16_t* dx = p.out + row * p.ldo;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at.front + (i * width + tid) * VEC;
            if (c >= at.end) continue;
            Pack<VEC> o, vx, vd;
            if (!KEEP) operands(sx, i, c, vx, vd);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const f2 x = KEEP ? xh[i][j] : mul(add(widen2<BF>(vx.e + 2 * j), minus), scale);
                const f2 gg = KEEP ? g[i][j] : mul(widen2<BF>(vd.e + 2 * j), widen2<BF>(w[i].e + 2 * j));
                const uint32_t word = narrow2<BF>(fma(x, k2, fma(gg, scale, k1)));
                *reinterpret_cast<uint32_t*>(o.e + 2 * j) = word;
            }
            *reinterpret_cast<Pack<VEC>*>(dx + c) = o;
        }
        if (SHIFT && at.extra >= 0) dx[at.extra] = narrow<BF>(fmaf(xe, c2, fmaf(ge, r, c1)));
        if (++st == p.stages) {
            st = 0;
            phase ^= 1;
        }
    }
    write_partials<VEC, WARPS, NV, SHIFT>(p, dw, db, at, dwe, dbe);
}

// Rows too wide for registers: dx alone, one block per row.
template <bool BF>
__global__ void __launch_bounds__(1024) ln_backward_wide_kernel(const LnParams p) {
    __shared__ float buf[2 * 32];
    allow_next_kernel();
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
    allow_next_kernel();
    wait_for_previous_kernel();  // so that the end of this kernel is the end of both
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float d = widen<BF>(p.dy[row * p.lddy + c]);
        const float xh = (widen<BF>(p.x[row * p.ldx + c]) - p.mean[row]) * p.rstd[row];
        dw = fmaf(d, xh, dw);
        db += d;
    }
    float* part = p.part + (long long)blockIdx.y * 2 * p.pitch;
    part[c] = dw;
    part[p.pitch + c] = db;
}

// Adds the partial rows in a fixed order: 32 columns per block, Y threads
// along the rows of each, then one over those.  `shifted`: the output whose rows
// set the partial rows' leads (block r's first row is row r), or null.
template <bool BF, int Y>
__global__ void __launch_bounds__(32 * Y)
ln_reduce_kernel(const float* part, int parts, int cols, int pitch, const uint16_t* shifted,
                 long long ldo, uint16_t* __restrict__ dw, uint16_t* __restrict__ db) {
    __shared__ float s[2][Y][32];
    wait_for_previous_kernel();
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.0f, b = 0.0f;
    if (c < cols)
        for (int r = y; r < parts; r += 8 * Y) {  // 16 loads in flight
            float va[8], vb[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool in = r + k * Y < parts;
                const int lead = shifted ? lead_of(-shift_of(shifted + (r + k * Y) * ldo) & 7) : 0;
                const float* row = part + (long long)(r + k * Y) * 2 * pitch + c + lead;
                va[k] = in ? row[0] : 0.0f;
                vb[k] = in ? row[pitch] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a += va[k];
                b += vb[k];
            }
        }
    s[0][y][lane] = a;
    s[1][y][lane] = b;
    __syncthreads();
    if (y > 1 || c >= cols) return;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < Y; ++k) sum += s[y][k][lane];
    uint16_t* out = y == 0 ? dw : db;
    if (out) out[c] = narrow<BF>(sum);
}

// Widest aligned pack that every row, weight and output allows: whole packs
// per row and aligned row starts.  0: none, rows are read by elements.
int pack_of(int64_t cols, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
    for (int vec : {8, 2}) {
        bool ok = cols % vec == 0;
        for (const void* q : ptrs) ok = ok && (reinterpret_cast<uintptr_t>(q) % (2 * vec)) == 0;
        for (int64_t ld : lds) ok = ok && ld % vec == 0;
        if (ok) return vec;
    }
    return 0;
}

// How a row is held.
struct RowShape {
    int warps, packs, vec;  // no warps: too wide for registers
    bool ring;
    int rows() const { return warps == 1 ? kRowsPerBlock : 1; }  // of a block
    int threads() const { return 32 * warps * rows(); }
};
// Warps for `cols` at 512 columns each: 1, 2, 4 or 8.
int even_warps(int64_t cols) { return cols <= 512 ? 1 : cols <= 1024 ? 2 : cols <= 2048 ? 4 : 8; }

// Forward.  Aligned rows go through the ring, others from 768 columns on (3000
// x 777: 7.3 us, in registers 8.3; 12909 x 697: 18.7 and 17.5).  Beyond
// 4096 columns as few warps as hold a row with 4 packs each, so that two or
// three rows are in work on an SM, which hides a row's barriers (8000 x 5120:
// 33 us; 16 warps of 2 packs, one row per SM, 56; 8192: 46 and 60).
RowShape forward_shape(int64_t cols, int vec) {
    if (cols > 16384) return {0, 0, vec, false};
    if (cols > 4096) return {(int)cdiv(cols, 1024), 4, vec, true};
    const int warps = even_warps(cols);
    if (vec == 8 || cols > 768) return {warps, cols <= 256 ? 1 : 2, vec, true};
    return {warps, cols <= 256 ? 4 : 8, vec, false};
}
// Backward.  Aligned rows go through the ring, others from 2048 columns on (16384
// x 4095: 89 us, in registers 107; 10000 x 2047: 41 and 37).  From 8192 on with 4
// packs per thread (4545 x 14557: 109 us; by element, 1024 threads 211).
RowShape backward_shape(int64_t cols, int vec) {
    if (cols > 16384) return {0, 0, vec, false};
    if (cols > 8192) return {(int)cdiv(cols, 1024), 4, vec, true};
    if (cols > 4096) return {(int)cdiv(cols, 512), 2, vec, true};
    const int warps = even_warps(cols);
    if (vec == 8 || cols > 2048) return {warps, cols <= 256 ? 1 : 2, vec, true};
    return {warps, cols <= 256 ? 4 : 8, vec, false};
}
// Blocks that walk over rows by a multiple of 8 (or have one row each).
int64_t walking_blocks(int64_t need, int64_t most) {
    return need <= most ? need : most < 8 ? 8 : most / 8 * 8;
}

// Launches a ring kernel: `operands` rows per stage, `per_sm` blocks on an SM.
template <auto Kern>
cudaError_t launch_ring(LnParams p, const RowShape& s, int operands, int per_sm, int64_t blocks,
                        cudaStream_t stream) {
    constexpr size_t kRoom = 224 * 1024;  // of an SM's shared memory
    // a block's own part: its static shared memory and the 1 KB it reserves
    const size_t fixed = s.warps == 1 ? 10240 : 2048;
    static std::atomic<unsigned long long> attr_set{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(attr_set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kRoom - fixed));
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_release);
    }
    const size_t stage = (size_t)s.rows() * operands * stage_bytes(s.vec != 8, p.cols);
    size_t stages = (kRoom / per_sm - fixed) / stage;
    if (stages > kMaxStages) stages = kMaxStages;
    p.stages = (int)stages;
    Kern<<<(unsigned)blocks, s.threads(), stages * stage, stream>>>(p);
    return cudaGetLastError();
}

template <bool BF>
cudaError_t launch_forward(const LnParams& p, int vec, int sms, cudaStream_t stream) {
    const RowShape s = forward_shape(p.cols, vec);
    if (s.ring) {
        const int per_sm = forward_threads(s.packs) / s.threads();
        const int64_t blocks = walking_blocks(cdiv(p.rows, s.rows()), (int64_t)sms * per_sm);
#define TG_RING(COND, WARPS, NV, SHIFT)                                                             \
    if ((COND) && s.packs == NV && (vec != 8) == SHIFT)                                             \
        return launch_ring<ln_forward_ring_kernel<BF, WARPS, NV, SHIFT>>(p, s, 1, per_sm, blocks, stream);
        TG_RING(s.warps == 1, 1, 1, false)
        TG_RING(s.warps == 1, 1, 2, false)
        TG_RING(s.warps == 2, 2, 2, false)
        TG_RING(s.warps == 4, 4, 2, false)
        TG_RING(s.warps == 8, 8, 2, false)
        TG_RING(true, 0, 4, false)
        TG_RING(s.warps == 2, 2, 2, true)
        TG_RING(s.warps == 4, 4, 2, true)
        TG_RING(s.warps == 8, 8, 2, true)
        TG_RING(true, 0, 4, true)
#undef TG_RING
        return cudaErrorInvalidValue;
    }
    if (!s.warps) {
        const dim3 grid((unsigned)p.rows);
        if (vec == 8)
            ln_forward_kernel<BF, 8, true, 32, 2, true><<<grid, 1024, 0, stream>>>(p);
        else if (vec == 2)
            ln_forward_kernel<BF, 2, true, 32, 8, true><<<grid, 1024, 0, stream>>>(p);
        else
            ln_forward_kernel<BF, 2, false, 32, 8, true><<<grid, 1024, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const unsigned blocks = (unsigned)cdiv(p.rows, s.rows());
#define TG_REGS(WARPS, NV)                                                                            \
    if (s.warps == WARPS && s.packs == NV) {                                                          \
        if (vec == 2)                                                                                 \
            ln_forward_kernel<BF, 2, true, WARPS, NV, false><<<blocks, s.threads(), 0, stream>>>(p);  \
        else                                                                                          \
            ln_forward_kernel<BF, 2, false, WARPS, NV, false><<<blocks, s.threads(), 0, stream>>>(p); \
        return cudaGetLastError();                                                                    \
    }
    TG_REGS(1, 4)
    TG_REGS(1, 8)
    TG_REGS(2, 8)
#undef TG_REGS
    return cudaErrorInvalidValue;
}

// Blocks of the gradient's kernel, each of which leaves one partial row of dw
// and db: what the SMs hold, but at least eight rows each once every SM has a
// block (a partial row is 8 bytes per column against 6 per element; four rows
// each and two blocks: 1000 x 4096 21.5 us instead of 16.4).
struct GradShape {
    RowShape row;
    int per_sm, parts;
};

GradShape grad_shape(int64_t rows, int64_t cols, int vec, int sms) {
    GradShape g{backward_shape(cols, vec), 0, 0};
    if (!g.row.warps) {
        g.parts = (int)(rows < 64 ? rows : 64);
        return g;
    }
    g.per_sm = kGradThreadsPerSm / g.row.threads();
    const int64_t steps = cdiv(rows, g.row.rows());
    int64_t blocks = steps / 8;
    if (blocks < sms) blocks = sms;
    const int64_t most = (int64_t)sms * g.per_sm;
    if (blocks > most) blocks = most;
    g.parts = (int)walking_blocks(steps, blocks);
    return g;
}

template <bool BF>
cudaError_t launch_backward(const LnParams& p, const GradShape& g, cudaStream_t stream) {
    const RowShape& s = g.row;
    if (!s.warps) {
        ln_backward_wide_kernel<BF><<<(unsigned)p.rows, 1024, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e
                                : launch_chained(ln_backward_wide_columns_kernel<BF>,
                                                 dim3((unsigned)cdiv(p.cols, 256), g.parts), 256, stream, p);
    }
#define TG_RING(COND, WARPS, NV, SHIFT)                                                              \
    if (s.ring && (COND) && s.packs == NV && (s.vec != 8) == SHIFT)                                  \
        return launch_ring<ln_backward_ring_kernel<BF, WARPS, NV, SHIFT>>(p, s, 2, g.per_sm, g.parts, stream);
    TG_RING(s.warps == 1, 1, 1, false)
    TG_RING(s.warps == 1, 1, 2, false)
    TG_RING(s.warps == 2, 2, 2, false)
    TG_RING(s.warps == 4, 4, 2, false)
    TG_RING(s.warps == 8, 8, 2, false)
    TG_RING(true, 0, 2, false)
    TG_RING(true, 0, 4, false)
    TG_RING(s.warps == 8, 8, 2, true)
    TG_RING(true, 0, 2, true)
    TG_RING(true, 0, 4, true)
#undef TG_RING
#define TG_REGS(WARPS, NV)                                                             \
    if (s.warps == WARPS && s.packs == NV) {                                           \
        ln_backward_kernel<BF, WARPS, NV><<<g.parts, s.threads(), 0, stream>>>(p);     \
        return cudaGetLastError();                                                     \
    }
    TG_REGS(1, 4)
    TG_REGS(1, 8)
    TG_REGS(2, 8)
    TG_REGS(4, 8)
#undef TG_REGS
    return cudaErrorInvalidValue;
}

int check_sizes(int64_t rows, int64_t cols, int dtype) {
    // (a column index plus a block's step stays within 32 bits)
    if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxSize) return TG_ERR_INVALID_ARG;
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
    PointerChecks check{dev};
    for (int i = 0; i < 6; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;
    LnParams p;
    std::memset(&p, 0, sizeof(p));
    p.rows = rows;
    p.cols = (int)cols;
    p.x = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.x_end = p.x + (rows - 1) * ldx + cols;
    p.weight = static_cast<const uint16_t*>(weight);
    p.bias = static_cast<const uint16_t*>(bias);
    p.eps = eps;
    p.out = static_cast<uint16_t*>(Y);
    p.ldo = ldy;
    p.mean = mean;
    p.rstd = rstd;
    const int vec = pack_of(cols, {X, weight, bias, Y}, {ldx, ldy});
    p.timeout_cycles = watchdog_timeout();
    p.status = info->status;
    if ((dtype == TG_BF16 ? launch_forward<true>(p, vec, info->sms, stream)
                          : launch_forward<false>(p, vec, info->sms, stream)) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}

extern "C" int tg_layernorm_grad_workspace_size(int64_t rows, int64_t cols, tg_dtype dtype,
                                                size_t* bytes) {
    int rc = check_sizes(rows, cols, (int)dtype);
    if (rc) return rc;
    if (!bytes) return TG_ERR_INVALID_ARG;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    // (the alignment of the rows does not change their number)
    *bytes = (size_t)grad_shape(rows, cols, 8, info->sms).parts * 2 * (size_t)pitch_of(cols) * sizeof(float);
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
    const size_t need = (size_t)s.parts * 2 * (size_t)pitch_of(cols) * sizeof(float);
    if (workspace_bytes < need) return TG_ERR_BUFFER;
    const Span work = span_bytes(workspace, need);
    for (const Span& o : outs)
        if (intersects(work, o)) return TG_ERR_OVERLAP;
    for (const Span& o : ins)
        if (intersects(work, o)) return TG_ERR_OVERLAP;
    const void* outp[3] = {dX, dweight, dbias};
    const void* inp[5] = {dY, X, weight, mean, rstd};
    PointerChecks check{dev};
    for (int i = 0; i < 3; ++i)
        if ((rc = check(outp[i], outs[i]))) return rc;
    for (int i = 0; i < 5; ++i)
        if ((rc = check(inp[i], ins[i]))) return rc;
    if ((rc = check(workspace, work))) return rc;
    LnParams p;
    std::memset(&p, 0, sizeof(p));
    p.rows = rows;
    p.cols = (int)cols;
    p.x = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.x_end = p.x + (rows - 1) * ldx + cols;
    p.dy = static_cast<const uint16_t*>(dY);
    p.lddy = lddy;
    p.dy_end = p.dy + (rows - 1) * lddy + cols;
    p.weight = static_cast<const uint16_t*>(weight);
    p.out = static_cast<uint16_t*>(dX);
    p.ldo = lddx;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.part = static_cast<float*>(workspace);
    p.pitch = pitch_of(cols);
    p.timeout_cycles = watchdog_timeout();
    p.status = info->status;
    cudaError_t e = dtype == TG_BF16 ? launch_backward<true>(p, s, stream)
                                     : launch_backward<false>(p, s, stream);
    if (e == cudaSuccess) {
        const bool bf = dtype == TG_BF16, few = s.parts <= 16;
        auto reduce = few ? (bf ? ln_reduce_kernel<true, 4> : ln_reduce_kernel<false, 4>)
                          : (bf ? ln_reduce_kernel<true, 32> : ln_reduce_kernel<false, 32>);
        e = launch_chained(reduce, dim3((unsigned)cdiv(cols, 32)), few ? 128 : 1024, stream, p.part, s.parts,
                           p.cols, p.pitch, s.row.ring && vec != 8 ? p.out : nullptr, p.ldo,
                           static_cast<uint16_t*>(dweight), static_cast<uint16_t*>(dbias));
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
