// host_common.h -- what every host entry point of the library shares: the
// checked current device, byte spans and the proofs that a call stays inside
// its caller's memory, and the tensor maps of GEMM operands.  Defined in
// api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

constexpr int64_t kMaxDim = 2147483647LL;
// Sizes whose kernels step past the end in 32 bits.
constexpr int64_t kMaxSize = 1LL << 30;
// Leading dimensions stay below the tensor-map stride limit of 2^40 bytes.
constexpr int64_t kMaxLd = (1LL << 39) - 8;

struct DeviceInfo {
    bool ready = false;
    bool supported = false;
    int sms = 0;
    int* status = nullptr;  // device address of the watchdog's status word
};

// Current device, checked for compute capability 10.3 once; a TG_* status.
int current_device(int* dev_out, DeviceInfo** info_out);

// Looks the driver's tensor-map and address-range calls up once; false if the
// tensor-map call is missing.
bool load_driver_entry_points();

// Watchdog limit and test hook set by tg_debug_configure.
long long watchdog_timeout();
int watchdog_skip_kblock();

typedef unsigned __int128 u128;

struct Span {
    uintptr_t lo = 0;
    u128 hi = 0;  // exclusive
    bool present = false;
};

// Bytes [p, p + ((rows-1)*ld + width) * 2) of a row-strided 16-bit matrix.
Span span_of(const void* p, int64_t rows, int64_t width, int64_t ld);
// Bytes [p, p + bytes); absent for a null p.
Span span_bytes(const void* p, u128 bytes);
bool intersects(const Span& a, const Span& b);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// TG_OK if the span is absent or lies inside one allocation of device `dev`
// (whose bytes then are *inside, if given).
int check_pointer(const void* p, const Span& s, int dev, Span* inside = nullptr);

// The same for the many operands of one call: tensors often lie in one
// allocation after another, and what was proven for it is asked for once.
struct PointerChecks {
    int dev;
    Span last = {};
    int operator()(const void* p, const Span& s) {
        if (s.present && last.present && last.lo <= s.lo && s.hi <= last.hi) return 0;
        return check_pointer(p, s, dev, &last);
    }
};

// Tensor maps of a 16-bit matrix (see the definitions for the box shapes).
bool encode_2d(CUtensorMap* map, int dtype, const void* base, uint64_t inner, uint64_t outer,
               int64_t ld, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);
bool encode_mn_atoms(CUtensorMap* map, int dtype, const void* base, int64_t rows, int64_t k,
                     int64_t ld, uint32_t atoms);
bool encode_k_pairs(CUtensorMap* map, int dtype, const void* base, int64_t rows, int64_t k,
                    int64_t ld, uint32_t box_rows);
bool encode_mn_atom_pairs(CUtensorMap* map, int dtype, const void* base, int64_t rows, int64_t k,
                          int64_t ld, uint32_t atoms);
// fp32 planes x rows x cols (row stride ld elements, planes rows*ld apart),
// box 32 columns x 32 rows, 128-byte swizzle.
bool encode_f32_planes(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                       uint64_t planes, int64_t ld);

// tcgen05 instruction descriptor: 16-bit operands, fp32 accumulation.
uint32_t make_idesc(int dtype, bool p_mn, bool q_mn, int n, int m);

// Copies rows x cols 16-bit elements between strided buffers (stage.cu).
cudaError_t launch_copy_rows(const void* src, long long lds, void* dst, long long ldd,
                             long long rows, long long cols, cudaStream_t stream);

}  // namespace tg
