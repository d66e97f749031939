// Shared by the matrix kernels (newton_schulz.hip, mx4.hip): 16-bit formats,
// the tiled product on the matrix cores, launches and argument checks.
//
// The product.  A workgroup computes a TILE x TILE tile of A B^T, both
// operands stored row-major along k, from "slabs" of 128 bytes of every row
// (64 fp16 or 256 4-bit elements).  A slab of both operands is copied to LDS by
// direct global-to-LDS loads of 16 bytes per lane, double-buffered, while the
// previous one feeds the matrix cores: one barrier per slab.  A fragment of
// the 32x32 matrix instructions is 16 bytes per lane, so fp16 (k = 16) and
// 4-bit (k = 64) operands move alike and share this code; which 16-byte
// pieces of a slab meet in one instruction does not matter as long as both
// operands agree, and lane group h takes pieces 4h..4h+3 (for the 4-bit
// operands its four block scales are then one dword).  Direct loads write LDS
// in lane order, so the bank swizzle is put into the addresses they read:
// piece q of row r sits in slot q ^ (r mod 8).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "zero_internal.h"
#include "zero_shard.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- formats
template <int DT>
struct Elem {
    typedef uint16_t type;
};
template <>
struct Elem<ZERO_F32> {
    typedef float type;
};

template <int DT>
__device__ __forceinline__ float to_float(typename Elem<DT>::type x) {
    if constexpr (DT == ZERO_F32) {
        return x;
    } else if constexpr (DT == ZERO_F16) {
        return (float)__builtin_bit_cast(_Float16, x);
    } else {
        return __builtin_bit_cast(float, (uint32_t)x << 16);
    }
}

// Rounded to nearest even; NaN stays NaN.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::type from_float(float x) {
    if constexpr (DT == ZERO_F32) {
        return x;
    } else if constexpr (DT == ZERO_F16) {
        return __builtin_bit_cast(uint16_t, (_Float16)x);
    } else {
        return __builtin_bit_cast(uint16_t, (__bf16)x);
    }
}

// ---------------------------------------------------------------- the product
constexpr int kSlab = 128;  // bytes of every row per slab

// A tile of TILE x TILE outputs by waves of WM x WN outputs each.
template <int TILE_, int WM_, int WN_>
struct Shape {
    static constexpr int TILE = TILE_, WM = WM_, WN = WN_;
    static constexpr int WAVES = (TILE / WM) * (TILE / WN);
    static constexpr int THREADS = WAVES * 64;
    static constexpr int MT = WM / 32, NT = WN / 32;
    static constexpr int LOADS = 2 * TILE / 8 / WAVES;  // direct loads (8 rows each) per wave and slab
    static constexpr int BUFFER = 2 * TILE * kSlab;     // bytes of one slab of both operands
    static constexpr int LDS = 2 * BUFFER;
};

// Rows of an operand from a tile's first row on: row r starts at base + r * ld
// bytes; rows from `rows` (>= 1) on repeat the last one.
struct Operand {
    const char* base;
    uint32_t ld;
    int rows;
};

struct Lane {
    int lane, wave, h, c;  // lane, wave, lane / 32, lane % 32
    __device__ Lane()
        : lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), h(lane >> 5),
          c(lane & 31) {}
};

__device__ __forceinline__ void load_to_lds(const char* from, char* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// fp16 operands: four k = 16 instructions a slab.
struct MmF16 {
    static constexpr bool kHalfSlabs = false;
    __device__ void begin(int, int) {}
    __device__ void next(int) {}
    template <int KK>
    __device__ __forceinline__ f32x16 mma(const i32x4& a, const i32x4& b, f32x16 c, int, int) const {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                      c, 0, 0, 0);
    }
};

template <class S, class MM, int KK>
__device__ __forceinline__ void slab_step(MM& mm, f32x16 (&acc)[S::MT][S::NT], const char* ra, const char* rb,
                                          int slot) {
    const int at = (slot ^ KK) << 4;
    i32x4 a[S::MT], b[S::NT];
#pragma unroll
    for (int i = 0; i < S::MT; ++i) a[i] = *(const i32x4*)(ra + i * 32 * kSlab + at);
#pragma unroll
    for (int j = 0; j < S::NT; ++j) b[j] = *(const i32x4*)(rb + j * 32 * kSlab + at);
#pragma unroll
    for (int i = 0; i < S::MT; ++i)
#pragma unroll
        for (int j = 0; j < S::NT; ++j) acc[i][j] = mm.template mma<KK>(a[i], b[j], acc[i][j], i, j);
}

// acc = the wave's part of the tile over `slabs` whole slabs, then (4-bit
// operands) half a slab if `half`.  Element r of acc[i][j] is output row
// wm * WM + 32 i + 8 (r / 4) + 4 h + r % 4, column wn * WN + 32 j + c.
// lds: S::LDS bytes.
template <class S, class MM>
__device__ __forceinline__ void tile_product(const Operand& A, const Operand& B, int slabs, bool half, MM& mm,
                                             char* lds, f32x16 (&acc)[S::MT][S::NT]) {
    const Lane L;
    const int wm = L.wave / (S::TILE / S::WN), wn = L.wave % (S::TILE / S::WN);
#pragma unroll
    for (int i = 0; i < S::MT; ++i)
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int total = slabs + (half ? 1 : 0);
    if (total == 0) return;
    // this wave's direct loads: groups of 8 rows, all of one operand
    const int g0 = L.wave * S::LOADS;
    const bool is_a = g0 < S::TILE / 8;
    const char* base = is_a ? A.base : B.base;
    const uint32_t ld = is_a ? A.ld : B.ld;
    const int last = (is_a ? A.rows : B.rows) - 1;
    const int row0 = (is_a ? g0 : g0 - S::TILE / 8) * 8 + (L.lane >> 3);
    const uint32_t piece = (L.lane & 7) ^ (L.lane >> 3);
    uint32_t off[S::LOADS];
#pragma unroll
    for (int i = 0; i < S::LOADS; ++i) {
        const int row = row0 + i * 8;
        off[i] = (uint32_t)(row < last ? row : last) * ld + piece * 16;
    }
    auto stage = [&](int slab, int buf) {
        const char* from = base + (int64_t)slab * kSlab;
        // past a half slab lies the next row: its second half is not read
        const uint32_t back = MM::kHalfSlabs && slab >= slabs ? (piece & 4) * 16 : 0;
        char* to = lds + buf * S::BUFFER + g0 * 1024;
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i) load_to_lds(from + (off[i] - back), to + i * 1024);
    };
    const int fa = (wm * S::WM + L.c) * kSlab, fb = (S::TILE + wn * S::WN + L.c) * kSlab;
    const int slot = (4 * L.h) ^ (L.c & 7);

    stage(0, 0);
    mm.begin(wm, wn);
    for (int s = 0; s < slabs; ++s) {
        __syncthreads();  // slab s has landed; the other buffer's readers are done
        const char* buf = lds + (s & 1) * S::BUFFER;
        if (s + 1 < total) stage(s + 1, (s + 1) & 1);
        mm.next(s + 1 < total ? s + 1 : s);
        const char *ra = buf + fa, *rb = buf + fb;
        slab_step<S, MM, 0>(mm, acc, ra, rb, slot);
        slab_step<S, MM, 1>(mm, acc, ra, rb, slot);
        slab_step<S, MM, 2>(mm, acc, ra, rb, slot);
        slab_step<S, MM, 3>(mm, acc, ra, rb, slot);
    }
    if constexpr (MM::kHalfSlabs) {
        if (!half) return;
        __syncthreads();
        const char* buf = lds + (slabs & 1) * S::BUFFER;
        mm.half();
        const char *ra = buf + fa, *rb = buf + fb;
        const int hslot = (2 * L.h) ^ (L.c & 7);
        slab_step<S, MM, 0>(mm, acc, ra, rb, hslot);
        slab_step<S, MM, 1>(mm, acc, ra, rb, hslot);
    }
}

// Workgroup number -> tile number: consecutive workgroups go to different XCDs,
// each with its own L2, so every XCD gets a contiguous range of tiles.
constexpr int kXcds = 8;
__device__ __forceinline__ int xcd_tile(int wg, int tiles) {
    const int xcd = wg % kXcds, k = wg / kXcds, per = tiles / kXcds, rest = tiles % kXcds;
    return xcd * per + (xcd < rest ? xcd : rest) + k;
}

// Tile number -> (row, column) of a tm x tn grid, walked in bands of 8 rows so
// that neighbours in time share operand rows.
__device__ __forceinline__ void band_tile(int t, int tm, int tn, int& i, int& j) {
    const int band = t / (8 * tn), first = band * 8;
    const int high = tm - first < 8 ? tm - first : 8, k = t - first * tn;
    i = first + k % high;
    j = k / high;
}

// ---------------------------------------------------------------- host side
int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(zero_error_text(), kErrorText, fmt, ap);
    va_end(ap);
    return code;
}

int ok() {
    zero_error_text()[0] = '\0';
    return ZERO_OK;
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool valid_dtype(int32_t dt, bool f32) { return dt == ZERO_F16 || dt == ZERO_BF16 || (f32 && dt == ZERO_F32); }

size_t elem_bytes(int32_t dt) { return dt == ZERO_F32 ? 4 : 2; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

template <class Args>
int launch(void (*kernel)(Args), dim3 grid, int block, hipStream_t s, const Args& args, const char* what) {
    void* params[] = {const_cast<Args*>(&args)};
    const hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(block), params, 0, s);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(ZERO_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    }
    return ok();
}

}  // namespace
