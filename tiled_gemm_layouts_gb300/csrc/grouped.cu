// grouped.cu -- host side of tg_grouped_gemm and tg_grouped_gemm_grad: argument
// checks, tile choice, tensor maps and the single launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "../../include/tilegemm.h"
#include "gemm_params.h"
#include "grouped.h"
#include "grouped_launch.cuh"

namespace tg {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

bool encode(CUtensorMap* map, int dtype, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    EncodeTiledFn fn = encode_fn();
    return fn &&
           fn(map, dtype == TG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `groups` matrices of `outer` rows of `inner` elements, ld and stride elements
// apart, in boxes of 64 x box_outer x 1.
bool encode_stack(CUtensorMap* map, int dtype, const void* base, int64_t inner, int64_t outer, int64_t groups,
                  int64_t ld, int64_t stride, uint32_t box_outer) {
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)groups};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, box_outer, 1};
    return encode(map, dtype, 3, base, dims, strides, box);
}

// The same in boxes of two neighbouring runs of 64: 64 x box_outer x 2 x 1.  Only
// the whole runs of a row (`runs`, two at least).
bool encode_stack_pairs(CUtensorMap* map, int dtype, const void* base, int64_t runs, int64_t outer, int64_t groups,
                        int64_t ld, int64_t stride, uint32_t box_outer) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)outer, (cuuint64_t)runs, (cuuint64_t)groups};
    const cuuint64_t strides[3] = {(cuuint64_t)ld * 2, 128, (cuuint64_t)stride * 2};
    const cuuint32_t box[4] = {64, box_outer, 2, 1};
    return encode(map, dtype, 4, base, dims, strides, box);
}

// Rows of a matrix: by `row`, a list, divided by per_row; or, without one, the maps
// of boxes of 64 columns x 128 rows (and two of them), and of gathered rows.
bool encode_rows(GroupedRows* rows, int dtype, const void* base, int64_t count, int64_t cols, int64_t ld,
                 const int32_t* row, int64_t per_row) {
    rows->count = (int)count;
    rows->base = base;
    rows->ld = ld;
    rows->cols = (int)cols;
    rows->row = row;
    // r / d for 0 <= r < 2^31: with d <= 2^b and m = floor(2^(31+b) / d) + 1, r m / 2^(31+b) is
    // above r / d by less than r / 2^(31+b) < 1 / d
    int b = 0;
    while (((int64_t)1 << b) < per_row) ++b;
    rows->shift = 31 + b;
    rows->magic = (uint32_t)(((u128)1 << (31 + b)) / (u128)per_row + 1);
    rows->pairs = cols >= 128 ? (int)(cols / 64) : 0;
    if (row) return true;  // fetched without maps
    return encode_2d(&rows->box, dtype, base, (uint64_t)cols, (uint64_t)count, ld, 64, 128) &&
           encode_2d(&rows->gather, dtype, base, (uint64_t)cols, (uint64_t)count, ld, 64, 1) &&
           (!rows->pairs || encode_k_pairs(&rows->box2, dtype, base, count, cols / 64 * 64, ld, 128));
}

}  // namespace

cudaError_t launch_grouped(int mode, const GroupedParams& p, GroupedTile tile, long long tiles, int sms, cudaStream_t stream) {
    switch (mode) {
        case GROUPED_ROWS: return launch_grouped_mode<GROUPED_ROWS>(p, tile, tiles, sms, stream);
        case GROUPED_WEIGHT: return launch_grouped_mode<GROUPED_WEIGHT>(p, tile, tiles, sms, stream);
    }
    return cudaErrorInvalidValue;
}

namespace {

bool odd_bytes(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Bytes of `groups` matrices of `rows` x `width`.
Span span_stack(const void* p, int64_t groups, int64_t rows, int64_t width, int64_t ld, int64_t stride) {
    return span_bytes(p, ((u128)(groups - 1) * (u128)stride + (u128)(rows - 1) * (u128)ld + (u128)width) * 2u);
}

struct GroupedArgs {
    int64_t R, N, K, G;
    const void* X;
    int64_t x_rows, ldx;
    const int32_t* row;
    int64_t per_row;
    const void* B;
    int64_t ldb, stride_b;
    int perm;
    const int32_t* offset;
    const void* Y;  // or dY
    int64_t ldy;
    int dtype;

    int64_t b_rows() const { return perm == TG_OP_N ? K : N; }
    int64_t b_width() const { return perm == TG_OP_N ? N : K; }
    Span x_span() const { return span_of(X, x_rows, K, ldx); }
    Span b_span() const { return span_stack(B, G, b_rows(), b_width(), ldb, stride_b); }
    Span y_span() const { return span_of(Y, R, N, ldy); }
    Span row_span() const { return span_bytes(row, (u128)R * 4); }
    Span offset_span() const { return span_bytes(offset, (u128)(G + 1) * 4); }
};

int check_args(const GroupedArgs& a) {
    if (a.R <= 0 || a.N <= 0 || a.K <= 0 || a.G <= 0 || a.x_rows <= 0 || a.R > kMaxSize || a.N > kMaxSize ||
        a.K > kMaxSize || a.x_rows > kMaxSize || a.G > kMaxRowGroups || a.per_row <= 0 || a.per_row > kMaxSize)
        return TG_ERR_INVALID_ARG;
    if (a.perm != TG_OP_N && a.perm != TG_OP_T) return TG_ERR_INVALID_ARG;
    if (a.dtype != TG_F16 && a.dtype != TG_BF16) return TG_ERR_DTYPE;
    if (!a.X || !a.B || !a.offset || !a.Y) return TG_ERR_INVALID_ARG;
    if (a.ldx < a.K || a.ldx > kMaxLd || a.ldy < a.N || a.ldy > kMaxLd || a.ldb < a.b_width() || a.ldb > kMaxLd)
        return TG_ERR_STRIDE;
    // (matrices of several groups do not overlap)
    if (a.G > 1 && (a.stride_b > kMaxLd || (u128)a.stride_b < (u128)(a.b_rows() - 1) * (u128)a.ldb + (u128)a.b_width() ||
                    a.stride_b < 0))
        return TG_ERR_STRIDE;
    if (!aligned16(a.X) || !aligned16(a.B) || !aligned16(a.Y) || a.ldx % 8 || a.ldy % 8 || a.ldb % 8 ||
        (a.G > 1 && a.stride_b % 8) || odd_bytes(a.row, 4) || odd_bytes(a.offset, 4))
        return TG_ERR_ALIGN;
    return TG_OK;
}

// The most tiles of `rows` rows that R rows in G groups can make, times tiles_n.
long long most_tiles(int64_t R, int64_t G, int rows, int64_t tiles_n) {
    return (std::min(R, G) + R / rows) * tiles_n;
}

// Tiles of 16 rows (grouped_few.cu) against tiles of 128: up to four rows per group
// that may have any, and up to 16 where the large tiles would not fill the GPU.
// N = 2048, K = 4096, us: 64 groups, 8 rows 31 to 50, 128 rows 119 to 138, 256 rows 158
// to 166, 512 rows 199 to 189; 8 groups, 16 rows 31 to 50, 128 rows 44 to 52, 256 rows
// 68 to 42.
bool few_rows(int64_t R, int64_t N, int64_t G, int perm, int sms) {
    const int64_t used = std::min(R, G);
    return perm == TG_OP_T && (R <= 4 * used || (R <= 16 * used && most_tiles(R, G, 128, (N + 127) / 128) <= sms));
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_grouped_gemm(int64_t R, int64_t N, int64_t K, int64_t G, const void* X, int64_t x_rows,
                               int64_t ldx, const int32_t* row, int64_t per_row, const void* B, int64_t ldb,
                               int64_t stride_b, tg_perm permB, const int32_t* offset, void* Y, int64_t ldy,
                               tg_dtype dtype, const tg_group_epilogue* epi, cudaStream_t stream) {
    const GroupedArgs a{R, N, K, G, X, x_rows, ldx, row, per_row, B, ldb, stride_b, (int)permB, offset, Y, ldy, (int)dtype};
    int rc = check_args(a);
    if (rc) return rc;
    if (!row && x_rows < R) return TG_ERR_INVALID_ARG;
    const void* bias = epi ? epi->bias : nullptr;
    const void* relu_of = epi ? epi->relu_of : nullptr;
    if (epi && epi->relu != 0 && epi->relu != 1) return TG_ERR_INVALID_ARG;
    if ((bias && (epi->ld_bias < N || epi->ld_bias > kMaxLd)) || (relu_of && (epi->ld_relu < N || epi->ld_relu > kMaxLd)))
        return TG_ERR_STRIDE;
    if (odd_bytes(bias, 2) || (relu_of && (!aligned16(relu_of) || epi->ld_relu % 8))) return TG_ERR_ALIGN;
    const void* ptrs[7] = {Y, X, B, row, offset, bias, relu_of};
    const Span spans[7] = {a.y_span(), a.x_span(), a.b_span(), a.row_span(), a.offset_span(),
                           bias ? span_of(bias, G, N, epi->ld_bias) : Span{},
                           relu_of ? span_of(relu_of, R, N, epi->ld_relu) : Span{}};
    for (int j = 1; j < 7; ++j)
        if (intersects(spans[0], spans[j])) return TG_ERR_OVERLAP;
    // tiles are counted in 32 bits
    if (most_tiles(R, G, 128, (N + 63) / 64) > kMaxSize) return TG_ERR_INVALID_ARG;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (!load_driver_entry_points()) return TG_ERR_CUDA;
    PointerChecks check{dev};
    for (int i = 0; i < 7; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;

    if (few_rows(R, N, G, permB, info->sms)) {
        FewRowsParams f = {};
        f.offset = offset;
        f.groups = (int)G;
        f.rows = (int)R;
        f.x_rows = (int)(row ? x_rows : R);
        f.per_row = (int)per_row;
        f.n = (int)N;
        f.k = (int)K;
        f.x = static_cast<const uint16_t*>(X);
        f.ldx = ldx;
        f.row = row;
        f.b = static_cast<const uint16_t*>(B);
        f.ldb = ldb;
        f.stride_b = G > 1 ? stride_b : 0;
        f.y = static_cast<uint16_t*>(Y);
        f.ldy = ldy;
        f.bias = static_cast<const uint16_t*>(bias);
        f.ld_bias = bias ? epi->ld_bias : 0;
        f.relu = epi ? epi->relu : 0;
        f.relu_of = static_cast<const uint16_t*>(relu_of);
        f.ld_relu = relu_of ? epi->ld_relu : 0;
        if (launch_few_rows(f, dtype == TG_BF16, most_tiles(R, G, kFewTileRows, 1), info->sms, stream) != cudaSuccess) {
            cudaGetLastError();
            return TG_ERR_CUDA;
        }
        return TG_OK;
    }
    // A pair's tiles for full groups, if they are enough for all pairs; else as many
    // columns as still leave a tile for every SM.  (Two groups of 150 rows, 1000 x 1000:
    // 19 us by pairs, 15 by 64 columns; eight of 100, 1024 x 2048, by a list 31 by 64
    // columns; 16 of 4096, 2048 to 192: 64 by pairs, 95 by 128 columns.)
    GroupedTile tile{64, 0, row != nullptr};
    if (R >= 128 * G && most_tiles(R, G, 256, (N + 255) / 256) >= info->sms / 2)
        tile = GroupedTile{256, 1, row != nullptr};
    else if (most_tiles(R, G, 128, (N + 127) / 128) >= info->sms)
        tile = GroupedTile{128, 0, row != nullptr};
    GroupedParams p;
    std::memset(&p, 0, sizeof(p));
    const int bnc = tile.pair ? tile.bn / 2 : tile.bn;
    p.q_mn = permB == TG_OP_N;
    bool ok = encode_rows(&p.p, dtype, X, row ? x_rows : R, K, ldx, row, per_row);
    const int64_t stride = G > 1 ? stride_b : ldb;  // (of one matrix: none)
    p.q_pairs = !p.q_mn && K >= 128 ? (int)(K / 64) : 0;
    ok = ok && (p.q_mn ? encode_stack(&p.map_q, dtype, B, N, K, G, ldb, stride, 64u * (uint32_t)tile.blocks_rows())
                       : encode_stack(&p.map_q, dtype, B, K, N, G, ldb, stride, (uint32_t)bnc));
    ok = ok && (!p.q_pairs || encode_stack_pairs(&p.map_q2, dtype, B, p.q_pairs, N, G, ldb, stride, (uint32_t)bnc));
    if (!ok) return TG_ERR_CUDA;
    p.offset = offset;
    p.groups = (int)G;
    p.rows = (int)R;
    p.num_kb = (int)((K + 63) / 64);
    p.tiles_n = (int)((N + tile.bn - 1) / tile.bn);
    p.group_m = 2048 / tile.rows();
    p.n = (int)N;
    p.idesc = make_idesc(dtype, false, p.q_mn != 0, tile.bn, tile.rows());
    p.bf16 = dtype == TG_BF16;
    p.out = Y;
    p.ldo = ldy;
    p.bias = bias;
    p.ld_bias = bias ? epi->ld_bias : 0;
    p.relu = epi ? epi->relu : 0;
    p.relu_of = relu_of;
    p.ld_relu = relu_of ? epi->ld_relu : 0;
    p.timeout_cycles = watchdog_timeout();
    p.status = info->status;
    if (launch_grouped(GROUPED_ROWS, p, tile, most_tiles(R, G, tile.rows(), p.tiles_n), info->sms, stream) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}

extern "C" int tg_grouped_gemm_grad(int64_t R, int64_t N, int64_t K, int64_t G, const void* dY, int64_t lddy,
                                    const void* X, int64_t x_rows, int64_t ldx, const int32_t* row, int64_t per_row,
                                    const int32_t* offset, void* dB, int64_t lddb, int64_t stride_db, tg_perm permB,
                                    tg_dtype dtype, cudaStream_t stream) {
    const GroupedArgs a{R, N, K, G, X, x_rows, ldx, row, per_row, dB, lddb, stride_db, (int)permB, offset, dY, lddy, (int)dtype};
    int rc = check_args(a);
    if (rc) return rc;
    if (!row && x_rows < R) return TG_ERR_INVALID_ARG;
    const void* ptrs[5] = {dB, X, dY, row, offset};
    const Span spans[5] = {a.b_span(), a.x_span(), a.y_span(), a.row_span(), a.offset_span()};
    for (int j = 1; j < 5; ++j)
        if (intersects(spans[0], spans[j])) return TG_ERR_OVERLAP;
    // dB's rows and columns: K x N, or N x K
    const int64_t m = a.b_rows(), n = a.b_width();
    if ((u128)G * (u128)((m + 127) / 128) * (u128)((n + 127) / 128) > (u128)kMaxSize) return TG_ERR_INVALID_ARG;
    int dev;
    DeviceInfo* info;
    if ((rc = current_device(&dev, &info))) return rc;
    if (!load_driver_entry_points()) return TG_ERR_CUDA;
    PointerChecks check{dev};
    for (int i = 0; i < 5; ++i)
        if ((rc = check(ptrs[i], spans[i]))) return rc;

    GroupedTile tile{128, 0, row != nullptr};
    if (G * ((m + 255) / 256) * ((n + 255) / 256) >= info->sms / 2) tile = GroupedTile{256, 1, row != nullptr};
    GroupedParams p;
    std::memset(&p, 0, sizeof(p));
    GroupedRows &x = permB == TG_OP_N ? p.p : p.q, &y = permB == TG_OP_N ? p.q : p.p;
    if (!encode_rows(&x, dtype, X, row ? x_rows : R, K, ldx, row, per_row) ||
        !encode_rows(&y, dtype, dY, R, N, lddy, nullptr, 1))
        return TG_ERR_CUDA;
    p.offset = offset;
    p.groups = (int)G;
    p.rows = (int)R;
    p.tiles_m = (int)((m + tile.rows() - 1) / tile.rows());
    p.tiles_n = (int)((n + tile.bn - 1) / tile.bn);
    p.group_m = 2048 / tile.rows();
    p.m = (int)m;
    p.n = (int)n;
    p.q_mn = 1;
    p.idesc = make_idesc(dtype, true, true, tile.bn, tile.rows());
    p.bf16 = dtype == TG_BF16;
    p.out = dB;
    p.ldo = lddb;
    p.out_stride = G > 1 ? stride_db : 0;
    p.timeout_cycles = watchdog_timeout();
    p.status = info->status;
    const long long tiles = (long long)G * p.tiles_m * p.tiles_n;
    if (launch_grouped(GROUPED_WEIGHT, p, tile, tiles, info->sms, stream) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_CUDA;
    }
    return TG_OK;
}
