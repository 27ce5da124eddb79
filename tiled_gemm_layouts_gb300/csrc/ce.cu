// ce.cu -- linear cross entropy (tg_linear_ce, tg_linear_ce_grad): argument
// checks, the plan of pieces, tiles and workspace, the launches, and the
// small kernels around the tensor-core products of ce_kernel.cuh.
//
// Forward: one product kernel (CE_LSE) and a combination of its partial sums.
// Backward: the tokens whose target lies in the vocabulary are gathered into
// a dense copy of H first.  The others have no gradient, and a batch of
// prompts or padded texts has many; their rows of H may hold anything, and an
// infinity times G = 0 would put a NaN into dW.  (In fp16 dW's product has a
// copy of its own, whose rows carry the tokens' weights.)  Then, for each piece of the
// vocabulary, CE_GRAD and CE_PRODUCTS; at the end dH's fp32 planes are
// summed, scaled and scattered back to the tokens' rows.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>

#include "../../include/tilegemm.h"
#include "ce_launch.cuh"
#include "host_common.h"
#include "ring.cuh"
#include "stage.cuh"

namespace tg {

template <>
cudaError_t launch_ce_mode<CE_LSE>(const CeParams&, CeTile, int, bool, cudaStream_t);
template <>
cudaError_t launch_ce_mode<CE_GRAD>(const CeParams&, CeTile, int, bool, cudaStream_t);
template <>
cudaError_t launch_ce_mode<CE_PRODUCTS>(const CeParams&, CeTile, int, bool, cudaStream_t);

cudaError_t launch_ce(int mode, const CeParams& p, CeTile tile, int sms, bool chained,
                      cudaStream_t stream) {
    switch (mode) {
        case CE_LSE: return launch_ce_mode<CE_LSE>(p, tile, sms, chained, stream);
        case CE_GRAD: return launch_ce_mode<CE_GRAD>(p, tile, sms, chained, stream);
        default: return launch_ce_mode<CE_PRODUCTS>(p, tile, sms, chained, stream);
    }
}

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------ small kernels

// Copies of H and W, whichever a tensor map cannot describe, in one launch.
// Small ones run by run; large ones through rings of bulk copies, each warp its
// own: pieces of up to 2048 elements, several rows (with what lies between
// them) or a part of one, out of which windows of 8 are written aligned.  The
// columns that round a copied row up to whole windows hold anything; no tensor
// map reaches them.  (23 x 1911 x 65536: 136 us, run by run 159, without a copy
// 53; 500 MB moved at 5.9 TB/s.)
__global__ void __launch_bounds__(256) ce_stage_kernel(const CopyJob h, const CopyJob w) {
    allow_next_kernel();
    const long long thread = blockIdx.x * 256LL + threadIdx.x, threads = gridDim.x * 256LL;
    if (h.rows) copy_rows(h, thread, threads);
    if (w.rows) copy_rows(w, thread, threads);
}

constexpr int kCopyWarps = 16, kCopyStages = 3, kCopyPiece = 2048;
constexpr int kCopyStage = 33 * 128;  // the units around a piece, and one to read past it
constexpr int kCopySmem = kCopyWarps * kCopyStages * kCopyStage;
constexpr int64_t kRingCopyBytes = 16 << 20;  // from here on

struct CopyPieces {
    CopyJob job;
    int per, chunks, vecs;  // rows of a piece, pieces of a row, windows of a row
    int width;              // columns of a piece
    long long pieces;
};
CopyPieces copy_pieces(const CopyJob& j) {
    CopyPieces p{j, 1, 1, (int)cdiv(j.cols, 8), kCopyPiece, 0};
    if (!j.rows) return p;
    if (j.lds * 2 <= kCopyPiece) {
        p.per = (int)(kCopyPiece / j.lds);
    } else {
        p.chunks = (int)cdiv(j.cols, kCopyPiece);
        p.width = (int)up(cdiv(j.cols, p.chunks), 8);
    }
    p.pieces = cdiv(j.rows, p.per) * p.chunks;
    return p;
}

__global__ void __launch_bounds__(32 * kCopyWarps, 1)
ce_copy_kernel(const CopyPieces h, const CopyPieces w, long long timeout_cycles, int* status) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kCopyWarps][kCopyStages];
    allow_next_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* stages = ring + warp * kCopyStages * kCopyStage;
    const long long first = blockIdx.x * (long long)kCopyWarps + warp, step = gridDim.x * (long long)kCopyWarps;
    const long long total = h.pieces + w.pieces;
    struct Piece {
        long long row;  // first row, first column
        int col, rows, n;
        const uint16_t* src;
    };
    auto piece_of = [&](long long i, const CopyPieces& c) {
        Piece p;
        const long long g = c.chunks > 1 ? row_of(i, c.chunks) : i;
        p.row = g * c.per;
        p.col = (int)(i - g * c.chunks) * c.width;
        p.rows = (int)min((long long)c.per, c.job.rows - p.row);
        const int cols = (int)min((long long)c.width, c.job.cols - p.col);
        p.n = (int)((p.rows - 1) * c.job.lds) + cols;
        p.src = c.job.src + p.row * c.job.lds + p.col;
        return p;
    };
    auto issue = [&](long long i, int st) {
        const CopyPieces& c = i < h.pieces ? h : w;
        const Piece p = piece_of(i < h.pieces ? i : i - h.pieces, c);
        uint8_t* dst = stages + st * kCopyStage;
        const uint32_t bar = smem_addr(&full[warp][st]);
        const RowCopy x = row_copy(dst, p.src, c.job.src + (c.job.rows - 1) * c.job.lds + c.job.cols, p.n);
        mbar_arrive_expect_tx(bar, x.bytes);
        if (x.bytes) bulk_load(smem_addr(dst), x.src, x.bytes, bar);
    };
    if (lane == 0) {
        for (int st = 0; st < kCopyStages; ++st) mbar_init(smem_addr(&full[warp][st]), 1);
        fence_barrier_init();
        for (int st = 0; st < kCopyStages && first + st * step < total; ++st) issue(first + st * step, st);
    }
    __syncwarp();
    int st = 0;
    uint32_t phase = 0;
    for (long long i = first; i < total; i += step) {
        const CopyPieces& c = i < h.pieces ? h : w;
        const Piece p = piece_of(i < h.pieces ? i : i - h.pieces, c);
        const uint8_t* stage = stages + st * kCopyStage;
        if (!stage_ready(smem_addr(&full[warp][st]), phase, timeout_cycles, status)) return;
        const int shift = shift_of(p.src), lds = (int)c.job.lds;
        uint16_t* dst = c.job.dst + p.row * c.job.ldd + p.col;
        if (c.per == 1) {
            const int n = (p.n + 7) / 8;
#pragma unroll 4
            for (int k = lane; k < n; k += 32)
                *reinterpret_cast<uint4*>(dst + k * 8) = window(stage, k, shift);
        } else {
            const int n = p.rows * c.vecs;
#pragma unroll 4
            for (int k = lane; k < n; k += 32) {
                const int r = (uint32_t)k / (uint32_t)c.vecs, x = (k - r * c.vecs) * 8;
                *reinterpret_cast<uint4*>(dst + r * c.job.ldd + x) = window(stage, 0, shift + r * lds + x);
            }
        }
        __syncwarp();
        if (lane == 0 && i + kCopyStages * step < total) issue(i + kCopyStages * step, st);
        if (++st == kCopyStages) {
            st = 0;
            phase ^= 1;
        }
    }
}

cudaError_t launch_copy(const CopyJob& h, const CopyJob& w, const DeviceInfo* info, cudaStream_t stream) {
    const long long vecs = (std::max(h.rows ? h.cols : 0, w.rows ? w.cols : 0) + 7) / 8;
    if ((h.rows * h.cols + w.rows * w.cols) * 2 < kRingCopyBytes) {
        // (1216 blocks, what the SMs hold: 172 us for 23 x 1911 x 65536; 4096:
        // 160; a block per 4 KB: 202)
        const int64_t blocks = std::min<int64_t>(cdiv((h.rows + w.rows) * vecs, 256), 4096);
        ce_stage_kernel<<<(unsigned)blocks, 256, 0, stream>>>(h, w);
        return cudaGetLastError();
    }
    static std::atomic<unsigned long long> attr_set{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(attr_set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(ce_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopySmem);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit, std::memory_order_release);
    }
    ce_copy_kernel<<<(unsigned)info->sms, 32 * kCopyWarps, kCopySmem, stream>>>(
        copy_pieces(h), copy_pieces(w), watchdog_timeout(), info->status);
    return cudaGetLastError();
}

// (max in log2 units, sum of 2^(l - max)) of a set of logits.
struct LogSum {
    float m, s;
    __device__ __forceinline__ void merge(float m2, float s2) {
        const float mn = fmaxf(m, m2), base = mn == -INFINITY ? 0.0f : mn;
        s = s * pow2(m - base) + s2 * pow2(m2 - base);
        m = mn;
    }
    __device__ __forceinline__ void merge_warp() {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
            const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
            merge(m2, s2);
        }
    }
};

// loss and lse of a token from its tiles' partial sums: WARPS warps per token,
// 8 warps per block.
template <int WARPS>
__global__ void __launch_bounds__(256)
ce_combine_kernel(const float2* part, const float* hit,
                  const long long* __restrict__ target, int T, long long V, int tiles,
                  float* __restrict__ loss, float* __restrict__ lse) {
    wait_for_previous_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = WARPS == 1 ? (int)(blockIdx.x * 8 + warp) : (int)blockIdx.x;
    if (t >= T) return;
    const float2* row = part + (long long)t * tiles;
    LogSum a{-INFINITY, 0.0f};
#pragma unroll 4
    for (int i = (WARPS == 1 ? lane : (int)threadIdx.x); i < tiles; i += 32 * WARPS) {
        const float2 u = row[i];
        a.merge(u.x, u.y);
    }
    a.merge_warp();
    if constexpr (WARPS > 1) {
        __shared__ float2 all[WARPS];
        if (lane == 0) all[warp] = make_float2(a.m, a.s);
        __syncthreads();
        if (warp) return;
        a = lane < WARPS ? LogSum{all[lane].x, all[lane].y} : LogSum{-INFINITY, 0.0f};
        a.merge_warp();
    }
    if (lane == 0) {
        const float tail = logf(a.s);
        lse[t] = a.m * kLn2 + tail;
        const long long y = target[t];
        loss[t] = y >= 0 && y < V ? (a.m - hit[t]) * kLn2 + tail : 0.0f;
    }
}

// What the backward pass keeps per token and per compacted row.
struct CeRows {
    int* live;          // number of tokens whose target lies in the vocabulary
    float* alpha;       // factor that the products of the scaled G still need
    int* token;         // [T] compacted row -> token
    int* target;        // [T] compacted row -> target
    float2* scale;      // [T] compacted row -> (lse in log2 units, factor of G)
    float* down;        // [T] compacted row -> what H's row is scaled by in dW's product
    int* place;         // [T] token -> compacted row, or -1
};

// fp16 ends at 2^-14 (with full precision), a probability is about 1/V, and
// tokens may weigh very differently: G's rows are scaled by scale2, and those of
// tokens whose |dloss| is below 2^-kEven of the largest by a power of two `up`
// more, 2^kMostUp at most.  The scatter of dH takes it back from its row; dW sums
// over rows of different scale, so its product reads a second copy of H whose
// rows are scaled by 1 / up.  A token within 2^20 of the heaviest keeps full
// precision down to probabilities of 2^-18.  (2^-kMostUp of a norm's output is
// still exact but for elements below 2^-4, and those are off by 2^-15 at most.)  bf16
// has fp32's range and needs none of it.
constexpr float kScaleF16 = 16384.0f;  // fp16's largest number is four times that
constexpr int kEven = 6, kMostUp = 10;
// 1 / up of a token with dloss / (largest |dloss|) = x
__device__ __forceinline__ float row_down(float x) {
    const int e = (int)(__float_as_uint(x) >> 23 & 255u) - 127;  // 2^e <= |x| < 2^(e + 1)
    const int up = min(max(-e - 1 - kEven, 0), kMostUp);
    return __uint_as_float((uint32_t)(127 - up) << 23);
}

constexpr int kCompactThreads = 1024;
// Up to this many tokens every block of the gather does the compaction for
// itself (two passes over 12 bytes per token), which saves a launch.
constexpr int kCompactEverywhere = 2048;

// Stable compaction by one block: the largest finite |dloss|, then steps of 1024
// tokens; returns the number of tokens that count and, to every thread, the
// factors.  G is scaled by 2^shift / max|dloss|: with one dloss for all tokens
// its factor is then a power of two, and rounding G to 16 bits rounds
// (p - [hit]) itself instead of repeating one rounding of dloss in every row.
// `keep(row, token, target)` is called for each token that counts.
template <class Keep, class Drop>
__device__ __forceinline__ int compact(const long long* __restrict__ target, const float* __restrict__ dloss,
                                       int T, long long V, float& ref, Keep keep, Drop drop) {
    __shared__ float wmax[32];
    __shared__ int wsum[33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float top = 0.0f;
    for (int t = threadIdx.x; t < T; t += kCompactThreads) {
        const long long y = target[t];
        if (y >= 0 && y < V && fabsf(dloss[t]) < INFINITY) top = fmaxf(top, fabsf(dloss[t]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) wmax[warp] = top;
    __syncthreads();
    top = wmax[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    ref = top > 0.0f ? top : 1.0f;
    int total = 0;
    for (int base = 0; base < T; base += kCompactThreads) {
        const int t = base + threadIdx.x;
        const long long y = t < T ? target[t] : -1;
        const bool counts = y >= 0 && y < V;
        const unsigned votes = __ballot_sync(0xffffffffu, counts);
        if (lane == 0) wsum[warp] = __popc(votes);
        __syncthreads();
        if (warp == 0) {
            int v = wsum[lane], x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
            wsum[lane] = x - v;
            if (lane == 31) wsum[32] = x;
        }
        __syncthreads();
        if (counts)
            keep(total + wsum[warp] + __popc(votes & ((1u << lane) - 1)), t, (int)y);
        else if (t < T)
            drop(t);
        total += wsum[32];
        __syncthreads();
    }
    return total;
}

// Writes a compaction down.
struct CeKeep {
    CeRows r;
    const float *lse, *dloss;
    float scale2;
    bool f16;
    const float* ref;
    __device__ __forceinline__ void operator()(int j, int t, int y) const {
        r.place[t] = j;
        r.token[j] = t;
        r.target[j] = y;
        const float x = dloss[t] / *ref, down = f16 ? row_down(x) : 1.0f;
        r.scale[j] = make_float2(lse[t] * kLog2e, x / down * scale2);
        r.down[j] = down;
    }
};

__global__ void __launch_bounds__(kCompactThreads)
ce_compact_kernel(const long long* __restrict__ target, const float* __restrict__ lse,
                  const float* __restrict__ dloss, int T, long long V, float scale2, bool f16, CeRows r) {
    allow_next_kernel();
    float ref;
    const CeKeep keep{r, lse, dloss, scale2, f16, &ref};
    const int live = compact(target, dloss, T, V, ref, keep, [&](int t) { r.place[t] = -1; });
    if (threadIdx.x == 0) {
        *r.live = live;
        *r.alpha = ref / scale2;
    }
}

// Dense rows of H for the tokens that count: out[j] = H[token[j]], columns
// [D, ldo) and the rows up to the next multiple of 256 (max_rows at most) filled with zeros; and
// the same rows scaled, out2[j] = down[j] H[token[j]], if out2 is given (fp16).
// HERE: the blocks compact for themselves, and the first one writes it down.
// `w`: a copy of W, where a tensor map cannot describe it.
template <bool HERE>
__global__ void __launch_bounds__(kCompactThreads)
ce_gather_kernel(const uint16_t* __restrict__ H, long long ldh, int D, CeRows r,
                 uint16_t* __restrict__ out, uint16_t* __restrict__ out2, int ldo, long long max_rows,
                 const long long* __restrict__ target, const float* __restrict__ lse,
                 const float* __restrict__ dloss, int T, long long V, float scale2, bool f16,
                 const CopyJob w) {
    __shared__ int tokens[HERE ? kCompactEverywhere : 1];
    allow_next_kernel();
    if (w.rows)
        copy_rows(w, blockIdx.x * (long long)kCompactThreads + threadIdx.x,
                  (long long)gridDim.x * kCompactThreads);
    int live;
    float ref = 1.0f;
    if constexpr (HERE) {
        const bool first = blockIdx.x == 0;
        const CeKeep keep{r, lse, dloss, scale2, f16, &ref};
        live = compact(
            target, dloss, T, V, ref,
            [&](int j, int t, int y) {
                tokens[j] = t;
                if (first) keep(j, t, y);
            },
            [&](int t) {
                if (first) r.place[t] = -1;
            });
        if (first && threadIdx.x == 0) {
            *r.live = live;
            *r.alpha = ref / scale2;
        }
    } else {
        wait_for_previous_kernel();
        live = *r.live;
    }
    const long long rows = min(max_rows, (long long)max(256, (live + 255) / 256 * 256));
    const int vecs = ldo / 8;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < rows * vecs;
         i += (long long)gridDim.x * blockDim.x) {
        const long long j = row_of(i, vecs);
        const int c = (int)(i - j * vecs) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        float down = 1.0f;
        if (j < live && c < D) {
            const long long t = HERE ? tokens[j] : r.token[j];
            const uint16_t* s = H + t * ldh + c;
            if (c + 8 <= D && (reinterpret_cast<uintptr_t>(s) & 15u) == 0) {
                v = *reinterpret_cast<const uint4*>(s);
            } else {
                uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < D) e[k >> 1] |= (uint32_t)s[k] << (16 * (k & 1));
                v = make_uint4(e[0], e[1], e[2], e[3]);
            }
            if (out2) down = HERE ? row_down(dloss[t] / ref) : r.down[j];
        }
        *reinterpret_cast<uint4*>(out + j * ldo + c) = v;
        if (out2) {
            const __half2 s = __float2half2_rn(down);
            __half2* x = reinterpret_cast<__half2*>(&v);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __hmul2(x[k], s);
            *reinterpret_cast<uint4*>(out2 + j * ldo + c) = v;
        }
    }
}

// dH rows: the sum of the fp32 planes' rows, scaled and rounded once; zeros
// for tokens without a gradient.
template <bool BF>
__global__ void ce_scatter_kernel(const float* planes, int splits, long long plane,
                                  int ldp, CeRows r, int T, int D, uint16_t* __restrict__ dH,
                                  long long ldd) {
    wait_for_previous_kernel();
    const float alpha = *r.alpha;
    const int vecs = (D + 7) / 8;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < (long long)T * vecs;
         i += (long long)gridDim.x * blockDim.x) {
        const long long t = row_of(i, vecs);
        const int c = (int)(i - t * vecs) * 8;
        const int j = r.place[t];
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (j >= 0) {
            const float* s = planes + (long long)j * ldp + c;
#pragma unroll 8
            for (int k = 0; k < splits; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(s + k * plane);
                const float4 b = *reinterpret_cast<const float4*>(s + k * plane + 4);
                y[0] += a.x; y[1] += a.y; y[2] += a.z; y[3] += a.w;
                y[4] += b.x; y[5] += b.y; y[6] += b.z; y[7] += b.w;
            }
            const float back = alpha * r.down[j];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] *= back;
        }
        uint16_t* o = dH + t * ldd + c;
        if (c + 8 <= D && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
            *reinterpret_cast<uint4*>(o) = make_uint4(pack2t<BF>(y[0], y[1]), pack2t<BF>(y[2], y[3]),
                                                      pack2t<BF>(y[4], y[5]), pack2t<BF>(y[6], y[7]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < D) o[k] = from_f32(y[k], BF);
        }
    }
}

unsigned blocks_for(int64_t threads, int sms) {
    const int64_t blocks = cdiv(threads, 256), most = (int64_t)sms * 8;
    return (unsigned)(blocks < most ? blocks : most);
}

// --------------------------------------------------------------- plans

bool tma_rows(const void* p, int64_t ld) { return aligned16(p) && (ld * 2) % 16 == 0; }

// Rows of whole 32-byte sectors.
bool sector_rows(const void* p, int64_t ld) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld * 2) & 31) == 0;
}
int64_t copied_ld(int64_t D) { return up(D, 64); }  // of a copy: whole lines

// Places regions one after another, 256-byte aligned.
struct Cursor {
    size_t at = 0;
    size_t take(u128 bytes) {
        const size_t here = at;
        at += ((size_t)bytes + 255) / 256 * 256;
        return here;
    }
};

// Tile of the logits' products.  CTA pairs' 256 x 256 tiles feed the tensor
// cores best.  For up to 128 tokens a pair's second half would multiply rows
// that do not exist, and reading W bounds the time; and where such tiles are
// fewer than the pairs, 128 x 128 tiles of single CTAs keep more SMs busy.
constexpr int kPairs = 76;  // of a GB300's 152 SMs (only the choice of a tile depends on it)

CeTile logits_tile(int64_t T, int64_t V) {
    return T > 128 && cdiv(T, 256) * cdiv(V, 256) >= kPairs ? CeTile{256, 1} : CeTile{128, 0};
}

// Tile of the gradients' products.  For up to 128 tokens a pair would read W
// at half the rate, for rows of dH that do not exist (with dH's contraction
// split over all workers: 16 x 4096 x 32768 189 us with pairs and 162 with
// single CTAs, 64 x 1024 x 65536 97 and 93, 128 x 512 x 4096 25.2 and 23.0);
// beyond, the same rule on the tiles of dH and dW together (200 x 1024 x
// 65536: 112 and 121).  A narrow D does not fill 256 columns.
CeTile products_tile(int64_t T, int64_t cols, int64_t D) {
    if (T <= 128) return CeTile{128, 0};
    const int bn = D > 128 ? 256 : 128;
    const int64_t tiles = (cdiv(T, 256) + cdiv(cols, 256)) * cdiv(D, bn);
    return tiles >= kPairs ? CeTile{bn, 1} : CeTile{128, 0};
}

struct FwdPlan {
    bool copy_h, copy_w;
    CeTile tile;
    int64_t tiles_n;
    size_t part, hit, h, w, bytes;
};

FwdPlan forward_plan(int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh, const void* W,
                     int64_t ldw) {
    FwdPlan f;
    f.tile = logits_tile(T, V);
    f.tiles_n = cdiv(V, f.tile.bn);
    // Every worker reads H again for each of its tiles, and rows that start
    // inside a sector cost a request more per 128 bytes.  A copy of H pays from
    // two rounds of tiles on, and not for a few rows (rows 16 bytes off in H and
    // W: 1000 x 512 x 117936 109 us, 89 with it; 102 x 1024 x 50000 32.2, 28.9; 32 x
    // 512 x 117936 31.6 as it is, 29.4 with aligned rows).
    const int64_t rounds = cdiv(T, f.tile.rows()) * f.tiles_n / (f.tile.pair ? kPairs : 2 * kPairs);
    f.copy_h = !tma_rows(H, ldh) || (T > 64 && rounds >= 2 && !sector_rows(H, ldh));
    f.copy_w = !tma_rows(W, ldw);
    Cursor c;
    f.part = c.take((u128)T * f.tiles_n * 2 * sizeof(float2));
    f.hit = c.take((u128)T * sizeof(float));
    f.h = c.take(f.copy_h ? (u128)T * copied_ld(D) * 2 : 0);
    f.w = c.take(f.copy_w ? (u128)V * copied_ld(D) * 2 : 0);
    f.bytes = c.at;
    return f;
}

// Bytes that a piece of G may take.  Each piece costs two launches, whose first
// and last tiles leave SMs idle; a larger one costs memory only (64, 128, 256
// and 512 MiB at 4096 x 4096 x 65536: 3783, 3674, 3673 and 3632 us).
constexpr int64_t kPieceBytes = 512LL << 20;

struct BwdPlan {
    bool copy_w;
    int64_t rows;        // of G and of the gathered H: T rounded up to whole tiles
    int64_t ldh;         // columns of the gathered H: D rounded up to whole K-blocks
    int64_t piece;       // columns of a piece of G, a multiple of 256
    int64_t pieces;
    int64_t ldp;         // columns of dH's planes
    CeTile grad, products;
    int64_t dh_kb;       // K-blocks of one split of dH's contraction
    int splits;
    bool scaled_h;       // dW's product has a copy of H of its own
    size_t live, token, target, scale, down, place, h, h2, g, planes, w, bytes;
};

BwdPlan backward_plan(int64_t T, int64_t V, int64_t D, const void* W, int64_t ldw, bool dw, int dtype,
                      int sms) {
    BwdPlan b;
    b.scaled_h = dw && dtype == TG_F16;
    b.copy_w = !tma_rows(W, ldw);
    // up to 128 tokens only K-blocks of dW's contraction count (rows of a 128-row
    // tile beyond them are not stored): 16 MiB of G for one token and V = 131072
    b.rows = up(T, T <= 128 ? 64 : 256);
    b.ldh = up(D, 64);
    const int64_t tiles_v = cdiv(V, 256);
    int64_t most = kPieceBytes / (b.rows * 512);
    if (most < 1) most = 1;
    b.pieces = cdiv(tiles_v, most);
    b.piece = cdiv(tiles_v, b.pieces) * 256;
    b.pieces = cdiv(V, b.piece);
    b.ldp = up(D, 8);
    b.grad = logits_tile(T, V < b.piece ? V : b.piece);
    // A tile of dH contracts over the whole piece.  Where that is longer than
    // an equal share of all the products, split it into fp32 planes that the
    // last kernel adds, each at least 8 K-blocks deep.  For up to 128 tokens
    // those planes are small beside W, which dH's workers have to read: split
    // until every worker has a share of it, 24 K-blocks or more (8 x 856 x
    // 54155: 87 us by the first rule, 75 by this; 128 x 300 x 20000 with
    // shares of 12: 46.5 instead of 43.8).
    const int64_t cols = V < b.piece ? V : b.piece, kb = cdiv(cols, 64);
    b.products = products_tile(T, cols, D);
    const int64_t workers = b.products.pair ? sms / 2 : sms, bm = b.products.rows();
    const int64_t n = cdiv(T, bm) * cdiv(D, b.products.bn);
    const int64_t n_dw = cdiv(cols, bm) * cdiv(D, b.products.bn);
    const int64_t share = (n * std::max<int64_t>(kb, kCeTileBlocks) +
                           n_dw * std::max<int64_t>(cdiv(T, 64), kCeTileBlocks)) / workers + 1;
    int64_t splits = cdiv(kb, share);
    if (T <= 128) splits = std::max(splits, std::min(workers / n, kb / 24));
    if (splits > kb / 8) splits = kb / 8;
    if (splits < 1) splits = 1;
    b.dh_kb = up(cdiv(kb, splits), 2);
    b.splits = (int)cdiv(kb, b.dh_kb);
    Cursor c;
    b.live = c.take(8);
    b.token = c.take((u128)T * 4);
    b.target = c.take((u128)T * 4);
    b.scale = c.take((u128)T * 8);
    b.down = c.take((u128)T * 4);
    b.place = c.take((u128)T * 4);
    b.h = c.take((u128)b.rows * b.ldh * 2);
    b.h2 = c.take(b.scaled_h ? (u128)b.rows * b.ldh * 2 : 0);
    b.g = c.take((u128)b.rows * b.piece * 2);
    b.planes = c.take((u128)b.splits * T * b.ldp * 4);
    b.w = c.take(b.copy_w ? (u128)V * copied_ld(D) * 2 : 0);
    b.bytes = c.at;
    return b;
}

// ------------------------------------------------------ argument checks

int check_sizes(int64_t T, int64_t V, int64_t D, int dtype) {
    if (T <= 0 || V <= 0 || D <= 0 || T > kMaxSize || V > kMaxSize || D > kMaxSize)
        return TG_ERR_INVALID_ARG;
    // tiles are counted in 32 bits
    if (cdiv(T, 128) * cdiv(V, 64) > INT_MAX || cdiv(T, 128) * cdiv(D, 64) > INT_MAX ||
        cdiv(V, 128) * cdiv(D, 64) > INT_MAX)
        return TG_ERR_INVALID_ARG;
    if (dtype != TG_F16 && dtype != TG_BF16) return TG_ERR_DTYPE;
    return TG_OK;
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Every output (and the workspace) disjoint from every other operand.
template <int N>
int check_disjoint(const Span (&s)[N], int outputs) {
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < N; ++j)
            if (intersects(s[i], s[j])) return TG_ERR_OVERLAP;
    return TG_OK;
}

void common_params(CeParams* p, int dtype, const DeviceInfo* info) {
    std::memset(p, 0, sizeof(*p));
    p->bf16 = dtype == TG_BF16;
    p->splits = 1;
    p->timeout_cycles = watchdog_timeout();
    p->status = info->status;
}

// K-major operand: `rows` x `k`, `box` rows of it per CTA; `two` may be null.
bool k_major(CUtensorMap* one, CUtensorMap* two, int* pairs, int dtype, const void* base, int64_t rows,
             int64_t k, int64_t ld, int box) {
    const int64_t whole = k & ~int64_t(63);
    *pairs = two && encode_k_pairs(two, dtype, base, rows, whole, ld, (uint32_t)box) ? (int)(whole / 64) : 0;
    return encode_2d(one, dtype, base, k, rows, ld, 64, (uint32_t)box);
}

// The logits' product: P = H (or its gathered rows) and Q = W^T, both K-major.
bool logits_side(CeParams* p, int dtype, CeTile tile, int64_t T, const void* H, int64_t h_rows,
                 int64_t h_cols, int64_t ldh, const void* W, int64_t V, int64_t D, int64_t ldw) {
    CeSide& s = p->side[0];
    // For few tokens the box holds only the rows there are, in whole groups of
    // 8: one token's K-block is then 1 KB of copies instead of 16.  (The rest
    // of the stage keeps old bytes, which reach only accumulator rows that
    // nobody reads.)
    const int64_t box = h_rows >= 128 ? 128 : up(h_rows, 8);
    s.p_bytes = (uint32_t)box * 128;
    // (two K-blocks of a smaller box would not land where two stages are)
    if (!k_major(&s.map_p, box == 128 ? &s.map_p2 : nullptr, &s.p_pairs, dtype, H, h_rows, h_cols, ldh,
                 (int)box) ||
        !k_major(&s.map_q, &s.map_q2, &s.q_pairs, dtype, W, V, D, ldw, tile.pair ? tile.bn / 2 : tile.bn))
        return false;
    s.num_kb = (int)cdiv(D, 64);
    s.tiles_m = (int)cdiv(T, tile.rows());
    s.tiles_n = (int)cdiv(V, tile.bn);
    s.group_m = std::min(s.tiles_m, 16);
    s.idesc = make_idesc(dtype, false, false, tile.bn, tile.rows());
    p->rows = (int)T;
    p->cols = (int)V;
    return true;
}

// MN-major Q: `cols` columns contiguous, `k` rows of them.
bool mn_major_q(CeSide* s, int dtype, CeTile tile, const void* base, int64_t cols, int64_t k,
                int64_t ld) {
    const int atoms = (tile.pair ? tile.bn / 2 : tile.bn) / 64;
    const int64_t whole = cols & ~int64_t(63), k_whole = k & ~int64_t(63);
    s->q_whole = encode_mn_atoms(&s->map_q3, dtype, base, whole, k, ld, (uint32_t)atoms) ? (int)whole : 0;
    s->q_pairs = s->q_whole && encode_mn_atom_pairs(&s->map_q2, dtype, base, whole, k_whole, ld, (uint32_t)atoms)
                     ? (int)(k_whole / 64)
                     : 0;
    return encode_2d(&s->map_q, dtype, base, cols, k, ld, 64, 64);
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_linear_ce_workspace_size(int64_t T, int64_t V, int64_t D, const void* H,
                                           int64_t ldh, const void* W, int64_t ldw, tg_dtype dtype,
                                           size_t* bytes) {
    const int rc = check_sizes(T, V, D, (int)dtype);
    if (rc) return rc;
    if (!bytes) return TG_ERR_INVALID_ARG;
    if (ldh < D || ldw < D || ldh > kMaxLd || ldw > kMaxLd) return TG_ERR_STRIDE;
    *bytes = forward_plan(T, V, D, H, ldh, W, ldw).bytes;
    return TG_OK;
}

extern "C" int tg_linear_ce(int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
                            const void* W, int64_t ldw, const int64_t* target, float* loss,
                            float* lse, tg_dtype dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
    int rc = check_sizes(T, V, D, (int)dtype);
    if (rc) return rc;
    if (!H || !W || !target || !loss || !lse || !workspace) return TG_ERR_INVALID_ARG;
    if (ldh < D || ldw < D || ldh > kMaxLd || ldw > kMaxLd) return TG_ERR_STRIDE;
    if (off(H, 2) || off(W, 2) || off(target, 8) || off(loss, 4) || off(lse, 4) || off(workspace, 256))
        return TG_ERR_ALIGN;
    const FwdPlan f = forward_plan(T, V, D, H, ldh, W, ldw);
    if (workspace_bytes < f.bytes) return TG_ERR_BUFFER;
    const Span spans[6] = {span_bytes(workspace, f.bytes), span_bytes(loss, (u128)T * 4),
                           span_bytes(lse, (u128)T * 4), span_of(H, T, D, ldh),
                           span_of(W, V, D, ldw), span_bytes(target, (u128)T * 8)};
    if ((rc = check_disjoint(spans, 3))) return rc;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (!load_driver_entry_points()) return TG_ERR_CUDA;
    const void* ptrs[6] = {workspace, loss, lse, H, W, target};
    PointerChecks check{dev};
    for (int i = 0; i < 6; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;

    char* ws = static_cast<char*>(workspace);
    bool ok = true;
    const bool staged = f.copy_h || f.copy_w;
    if (staged) {
        const int64_t wide = copied_ld(D);
        CopyJob h{static_cast<const uint16_t*>(H), ldh, reinterpret_cast<uint16_t*>(ws + f.h), wide,
                  f.copy_h ? T : 0, D};
        CopyJob w{static_cast<const uint16_t*>(W), ldw, reinterpret_cast<uint16_t*>(ws + f.w), wide,
                  f.copy_w ? V : 0, D};
        ok = launch_copy(h, w, info, stream) == cudaSuccess;
        if (f.copy_h) {
            H = h.dst;
            ldh = wide;
        }
        if (f.copy_w) {
            W = w.dst;
            ldw = wide;
        }
    }
    CeParams p;
    common_params(&p, (int)dtype, info);
    ok = ok && logits_side(&p, (int)dtype, f.tile, T, H, T, D, ldh, W, V, D, ldw);
    p.target = reinterpret_cast<const long long*>(target);
    p.part = reinterpret_cast<float2*>(ws + f.part);
    p.hit = reinterpret_cast<float*>(ws + f.hit);
    ok = ok && launch_ce(CE_LSE, p, f.tile, info->sms, staged, stream) == cudaSuccess;
    if (ok) {
        // few tokens: a block for each, so that hundreds of partial sums are
        // not one warp's serial chain (1024 of them: 6.9 us by one warp)
        const bool few = T <= info->sms;
        ok = launch_chained(few ? ce_combine_kernel<8> : ce_combine_kernel<1>,
                            dim3((unsigned)(few ? T : cdiv(T, 8))), 256, stream, p.part, p.hit, p.target,
                            (int)T, (long long)V, (int)f.tiles_n * 2, loss, lse) == cudaSuccess;
    }
    if (!ok) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}

extern "C" int tg_linear_ce_grad_workspace_size(int64_t T, int64_t V, int64_t D, const void* H,
                                                int64_t ldh, const void* W, int64_t ldw,
                                                const void* dH, int64_t lddh, const void* dW,
                                                int64_t lddw, tg_dtype dtype, size_t* bytes) {
    int rc = check_sizes(T, V, D, (int)dtype);
    if (rc) return rc;
    if (!bytes || (!dH && !dW)) return TG_ERR_INVALID_ARG;
    if (ldh < D || ldw < D || ldh > kMaxLd || ldw > kMaxLd) return TG_ERR_STRIDE;
    if ((dH && (lddh < D || lddh > kMaxLd)) || (dW && (lddw < D || lddw > kMaxLd))) return TG_ERR_STRIDE;
    (void)H;  // copied in any case
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    *bytes = backward_plan(T, V, D, W, ldw, dW != nullptr, (int)dtype, info->sms).bytes;
    return TG_OK;
}

extern "C" int tg_linear_ce_grad(int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
                                 const void* W, int64_t ldw, const int64_t* target,
                                 const float* lse, const float* dloss, void* dH, int64_t lddh,
                                 void* dW, int64_t lddw, tg_dtype dtype, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    int rc = check_sizes(T, V, D, (int)dtype);
    if (rc) return rc;
    if (!H || !W || !target || !lse || !dloss || (!dH && !dW) || !workspace) return TG_ERR_INVALID_ARG;
    if (ldh < D || ldw < D || ldh > kMaxLd || ldw > kMaxLd) return TG_ERR_STRIDE;
    if ((dH && (lddh < D || lddh > kMaxLd)) || (dW && (lddw < D || lddw > kMaxLd))) return TG_ERR_STRIDE;
    if (off(H, 2) || off(W, 2) || off(dH, 2) || off(dW, 2) || off(target, 8) || off(lse, 4) ||
        off(dloss, 4) || off(workspace, 256))
        return TG_ERR_ALIGN;
    const Span outs[2] = {span_of(dH, T, D, lddh), span_of(dW, V, D, lddw)};
    const Span ins[5] = {span_of(H, T, D, ldh), span_of(W, V, D, ldw), span_bytes(target, (u128)T * 8),
                         span_bytes(lse, (u128)T * 4), span_bytes(dloss, (u128)T * 4)};
    {
        const Span all[7] = {outs[0], outs[1], ins[0], ins[1], ins[2], ins[3], ins[4]};
        if ((rc = check_disjoint(all, 2))) return rc;
    }
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (!load_driver_entry_points()) return TG_ERR_CUDA;
    const BwdPlan b = backward_plan(T, V, D, W, ldw, dW != nullptr, (int)dtype, info->sms);
    if (workspace_bytes < b.bytes) return TG_ERR_BUFFER;
    const Span work = span_bytes(workspace, b.bytes);
    for (const Span& s : outs)
        if (intersects(work, s)) return TG_ERR_OVERLAP;
    for (const Span& s : ins)
        if (intersects(work, s)) return TG_ERR_OVERLAP;
    PointerChecks check{dev};
    if ((rc = check(workspace, work)) || (rc = check(dH, outs[0])) || (rc = check(dW, outs[1])) ||
        (rc = check(H, ins[0])) || (rc = check(W, ins[1])) || (rc = check(target, ins[2])) ||
        (rc = check(lse, ins[3])) || (rc = check(dloss, ins[4])))
        return rc;

    char* ws = static_cast<char*>(workspace);
    const int dt = (int)dtype, sms = info->sms;
    bool ok = true;
    CopyJob copy_w{static_cast<const uint16_t*>(W), ldw, reinterpret_cast<uint16_t*>(ws + b.w), copied_ld(D),
                   b.copy_w ? V : 0, D};
    if (b.copy_w) {
        W = copy_w.dst;
        ldw = copy_w.ldd;
        if (V * D * 2 >= kRingCopyBytes) {  // a small copy is part of the gather below
            ok = launch_copy(CopyJob{}, copy_w, info, stream) == cudaSuccess;
            copy_w.rows = 0;
        }
    }
    CeRows rows;
    rows.live = reinterpret_cast<int*>(ws + b.live);
    rows.alpha = reinterpret_cast<float*>(ws + b.live) + 1;
    rows.token = reinterpret_cast<int*>(ws + b.token);
    rows.target = reinterpret_cast<int*>(ws + b.target);
    rows.scale = reinterpret_cast<float2*>(ws + b.scale);
    rows.down = reinterpret_cast<float*>(ws + b.down);
    rows.place = reinterpret_cast<int*>(ws + b.place);
    uint16_t* h = reinterpret_cast<uint16_t*>(ws + b.h);
    uint16_t* h2 = b.scaled_h ? reinterpret_cast<uint16_t*>(ws + b.h2) : nullptr;
    uint16_t* g = reinterpret_cast<uint16_t*>(ws + b.g);
    float* planes = reinterpret_cast<float*>(ws + b.planes);
    const bool f16 = dt == TG_F16;
    const float scale2 = f16 ? kScaleF16 : 1.0f;
    const long long* tgt = reinterpret_cast<const long long*>(target);
    const bool here = T <= kCompactEverywhere;
    const unsigned gather_blocks = (unsigned)std::min<int64_t>(
        cdiv(b.rows * (b.ldh / 8) + copy_w.rows * (up(D, 8) / 8), kCompactThreads), sms * 2);
    if (here) {
        ce_gather_kernel<true><<<gather_blocks, kCompactThreads, 0, stream>>>(
            static_cast<const uint16_t*>(H), ldh, (int)D, rows, h, h2, (int)b.ldh, b.rows, tgt, lse, dloss,
            (int)T, V, scale2, f16, copy_w);
        ok = ok && cudaGetLastError() == cudaSuccess;
    } else {
        ce_compact_kernel<<<1, kCompactThreads, 0, stream>>>(tgt, lse, dloss, (int)T, V, scale2, f16, rows);
        ok = ok && cudaGetLastError() == cudaSuccess &&
             launch_chained(ce_gather_kernel<false>, dim3(gather_blocks), kCompactThreads, stream,
                            static_cast<const uint16_t*>(H), (long long)ldh, (int)D, rows, h, h2, (int)b.ldh,
                            (long long)b.rows, tgt, lse, dloss, (int)T, (long long)V, scale2, f16,
                            copy_w) == cudaSuccess;
    }

    // Raster groups: 16 tile rows of the logits (12, 20 and 24 cost 1 to 4 % of
    // the loss at 8192 x 4096 x 131072), 4 of dH and 8 of dW (16 of each: 3712
    // us against 3568 at 4096 x 4096 x 65536).
    const int bm = b.products.rows();
    for (int64_t i = 0; ok && i < b.pieces; ++i) {
        const int64_t v0 = i * b.piece, cols = V - v0 < b.piece ? V - v0 : b.piece;
        const uint16_t* w = static_cast<const uint16_t*>(W) + v0 * ldw;
        CeParams p;
        // a piece of G, scaled, from the gathered rows
        common_params(&p, dt, info);
        ok = logits_side(&p, dt, b.grad, T, h, b.rows, b.ldh, b.ldh, w, cols, D, ldw) &&
             encode_2d(&p.side[0].map_c, dt, g, b.piece, b.rows, b.piece, 64, 32);
        p.live = rows.live;
        p.col0 = v0;
        p.row_target = rows.target;
        p.row_scale = rows.scale;
        ok = ok && launch_ce(CE_GRAD, p, b.grad, sms, true, stream) == cudaSuccess;
        if (!ok) break;
        common_params(&p, dt, info);
        p.live = rows.live;
        p.alpha = rows.alpha;
        if (dH) {
            CeSide& s = p.side[0];
            p.all_kb = (int)cdiv(cols, 64);
            p.splits = (int)cdiv(p.all_kb, b.dh_kb);
            p.accumulate = i > 0;
            // a K-block past `cols` meets G's zero columns and W rows that the
            // map fills with zeros
            // one CTA's tiles need only the rows of G that there are
            const int64_t box = b.products.pair || T >= 128 ? 128 : up(T, 8);
            s.p_bytes = (uint32_t)box * 128;
            ok = k_major(&s.map_p, box == 128 ? &s.map_p2 : nullptr, &s.p_pairs, dt, g, b.rows,
                         (int64_t)p.all_kb * 64, b.piece, (int)box) &&
                 mn_major_q(&s, dt, b.products, w, D, cols, ldw) &&
                 encode_f32_planes(&s.map_c, planes, b.ldp, T, b.splits, b.ldp);
            s.num_kb = (int)b.dh_kb;
            s.tiles_m = (int)cdiv(T, bm);
            s.tiles_n = (int)cdiv(D, b.products.bn);
            s.group_m = std::min(s.tiles_m, 4);
            s.idesc = make_idesc(dt, false, true, b.products.bn, bm);
            s.out_rows = (int)T;
            s.out_cols = (int)D;
        }
        if (ok && dW) {
            CeSide& s = p.side[1];
            uint16_t* out = static_cast<uint16_t*>(dW) + v0 * lddw;
            const bool tensor = tma_rows(dW, lddw) && D >= 8;
            p.n_tma = tensor ? (int)(D & ~int64_t(7)) : 0;
            ok = encode_mn_atoms(&s.map_p, dt, g, b.piece, b.rows, b.piece, 2) &&
                 mn_major_q(&s, dt, b.products, h2 ? h2 : h, b.ldh, b.rows, b.ldh) &&
                 encode_2d(&s.map_c, dt, tensor ? out : g, tensor ? p.n_tma : 8, cols,
                           tensor ? lddw : b.piece, 64, 32);
            s.p_pairs = encode_mn_atom_pairs(&s.map_p2, dt, g, b.piece, b.rows, b.piece, 2)
                            ? (int)(b.rows / 64)
                            : 0;
            s.num_kb = (int)(b.rows / 64);
            s.p_bytes = 128 * 128;
            s.tiles_m = (int)cdiv(cols, bm);
            s.tiles_n = (int)cdiv(D, b.products.bn);
            s.group_m = std::min(s.tiles_m, 8);
            s.idesc = make_idesc(dt, true, true, b.products.bn, bm);
            s.out_rows = (int)cols;
            s.out_cols = (int)D;
            p.out = out;
            p.ldo = lddw;
        }
        ok = ok && launch_ce(CE_PRODUCTS, p, b.products, sms, true, stream) == cudaSuccess;
    }
    if (ok && dH)
        ok = launch_chained(dt == TG_BF16 ? ce_scatter_kernel<true> : ce_scatter_kernel<false>,
                            dim3(blocks_for(T * ((D + 7) / 8), sms)), 256, stream, planes, b.splits,
                            (long long)T * b.ldp, (int)b.ldp, rows, (int)T, (int)D,
                            static_cast<uint16_t*>(dH), (long long)lddh) == cudaSuccess;
    if (!ok) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
