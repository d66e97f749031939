// Shared by the kernels on microscaled operands and on rows (mx4.hip, mx8.hip, rows.hip,
// tokens.hip): sizes, eight elements of a row at a time, block scales, places.
#pragma once

#include <initializer_list>

#include "matrix_common.h"

namespace {

constexpr int kMxBlock = 32;
constexpr int kMxPad = 128;
constexpr int kThreads = 256;
constexpr int64_t kMaxSide = int64_t(1) << 24;

__device__ __host__ __forceinline__ int64_t padded(int64_t cols) { return (cols + kMxPad - 1) / kMxPad * kMxPad; }

// ---------------------------------------------------------------- quantisation
__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }

// Scale byte of a block whose largest magnitude has these bits: 2 below its
// exponent (6 = 1.5 * 2^2 is the largest code), not below 0; 255 for inf or NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255 ? 255u : e < 2 ? 0u : e - 2;
}

// 1 / scale, exactly: 2^(127 - s), a normal number for every s that a block gets.
__device__ __forceinline__ float inverse_scale(uint32_t s) {
    return __builtin_bit_cast(float, (254u - (s < 253 ? s : 253u)) << 23);
}

// Eight values times 1 / scale as 4-bit codes, the first in the low bits:
// nearest, ties to even, saturating (what the conversion instructions do).
__device__ __forceinline__ uint32_t codes8(const float* x, float inv) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0] * inv, x[1] * inv, 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2] * inv, x[3] * inv, 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4] * inv, x[5] * inv, 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6] * inv, x[7] * inv, 1.0f, 3);
    return c;
}

// The same from four dwords of 16-bit values under a scale.  bf16: not for scales near
// the smallest numbers, where a value below the normal ones is more than half a code.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kLowScale = 16;
template <int DT>
__device__ __forceinline__ uint32_t codes8_16(const uint32_t* v, float scale) {
    uint32_t c = 0;
    if constexpr (DT == ZERO_BF16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[3]), scale, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v[3]), scale, 3);
    }
    return c;
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t v) {  // v of another lane of this group of four
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest magnitude, as fp32 bits, of 16-bit values in dwords.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <int DT, int N>
__device__ __forceinline__ uint32_t top16(const uint32_t* v) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
    const uint16_t top = m[0] > m[1] ? m[0] : m[1];
    return __builtin_bit_cast(uint32_t, to_float<DT>(top));
}

// Eight elements of a row from column c on; past the row's end zeros.
template <int DT>
struct Eight {
    typedef typename Elem<DT>::type T;
    static constexpr int kVecs = (int)sizeof(T) / 2;
    u32x4 v[kVecs];

    // Whole vectors at any alignment of the elements: the memory pipeline takes them.
    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t cols) {
        if (c + 8 <= cols) {
            __builtin_memcpy(v, row + c, sizeof(v));
        } else {
            T x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = c + i < cols ? row[c + i] : (T)0;
            __builtin_memcpy(v, x, sizeof(v));
        }
    }
    // The same with a row's last elements taken from its last whole vector, moved down: one load instead of
    // eight, whose registers every kernel that holds several such vectors would pay for.  WHOLE: cols is a
    // multiple of eight.
    template <bool WHOLE = false>
    __device__ __forceinline__ void fetch(const T* row, int64_t c, int64_t cols) {
        if (WHOLE || c + 8 <= cols) {
            __builtin_memcpy(v, row + c, sizeof(v));
        } else if (c >= cols) {
            zero();
        } else if (cols >= 8) {
            __builtin_memcpy(v, row + cols - 8, sizeof(v));
            down((int)(c + 8 - cols));
        } else {  // rows of fewer than eight
            zero();
#pragma unroll 1
            for (int64_t i = cols - 1; i >= c; --i) up(row[i]);
        }
    }
    // values() from whole dwords: two elements each, without 16-bit pieces in registers of their own.
    __device__ __forceinline__ void floats(float* x) const {
        if constexpr (DT == ZERO_BF16) {
            uint32_t d[4];
            __builtin_memcpy(d, v, sizeof(d));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __builtin_bit_cast(float, d[i] << 16);
                x[2 * i + 1] = __builtin_bit_cast(float, d[i] & 0xFFFF0000u);
            }
        } else {
            values(x);
        }
    }
    // The elements `by` (1 to 7) places lower, zeros behind them.
    __device__ __forceinline__ void down(int by) {
        if constexpr (kVecs == 1) {
            unsigned __int128 w;
            __builtin_memcpy(&w, v, sizeof(w));
            w >>= 16 * by;
            __builtin_memcpy(v, &w, sizeof(w));
        } else {
            uint32_t d[8];
            __builtin_memcpy(d, v, sizeof(d));
#pragma unroll
            for (int step = 1; step <= 4; step *= 2)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = by & step ? (i + step < 8 ? d[i + step] : 0u) : d[i];
            __builtin_memcpy(v, d, sizeof(d));
        }
    }
    // x first, the elements one place higher.
    __device__ __forceinline__ void up(T x) {
        T d[8];
        __builtin_memcpy(d, v, sizeof(d));
#pragma unroll
        for (int i = 7; i > 0; --i) d[i] = d[i - 1];
        d[0] = x;
        __builtin_memcpy(v, d, sizeof(d));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = u32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void values(float* x) const {
        T t[8];
        __builtin_memcpy(t, v, sizeof(v));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_float<DT>(t[i]);
    }
    // The largest magnitude of the block that four neighbouring lanes hold, as fp32 bits.
    __device__ __forceinline__ uint32_t block_top() const {
        uint32_t top = 0;
        if constexpr (DT == ZERO_F32) {
            float x[8];
            values(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = umax(top, magnitude(x[i]));
        } else {
            uint32_t d[4];
            __builtin_memcpy(d, v, sizeof(d));
            top = top16<DT, 4>(d);
        }
        top = umax(top, quad<0xB1>(top));  // lanes 1 0 3 2
        return umax(top, quad<0x4E>(top));  // lanes 2 3 0 1
    }
    __device__ __forceinline__ uint32_t codes(uint32_t s) const {
        if (s == 255) return 0;
        if constexpr (DT != ZERO_F32) {
            if (s >= kLowScale) {
                uint32_t d[4];
                __builtin_memcpy(d, v, sizeof(d));
                return codes8_16<DT>(d, __builtin_bit_cast(float, s << 23));
            }
        }
        float x[8];
        values(x);
        return codes8(x, inverse_scale(s));
    }
};

// Eight values, rounded to the type, to a row from column c on; nothing past the row's end.
template <int DT, bool WHOLE = false>
__device__ __forceinline__ void put8(typename Elem<DT>::type* row, int64_t c, int64_t cols, const float* x) {
    typedef typename Elem<DT>::type T;
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = from_float<DT>(x[i]);
    if (WHOLE || c + 8 <= cols) {  // whole vectors at any alignment
        u32x4 w[sizeof(v) / 16];
        __builtin_memcpy(w, v, sizeof(v));
#pragma unroll
        for (int k = 0; k < (int)sizeof(v) / 16; ++k) {
            asm volatile("" : "+v"(w[k]));  // one store, not the pieces it was made of
            __builtin_memcpy((char*)(row + c) + 16 * k, &w[k], 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = v[i];
    }
}

// ---------------------------------------------------------------- MXFP8
// Scale byte of a block of E4M3 codes whose largest magnitude has these bits: the smallest
// power of two (not below 2^-127) that brings it to 448 = 1.75 * 2^8, the largest code, or
// below: 8 below its exponent, 7 where its fraction is above 1.75.  Nothing saturates, and a
// floating code loses no precision by it.  255 for inf or NaN.
__device__ __forceinline__ uint32_t scale_byte8(uint32_t top) {
    if (top >> 23 == 255) return 255u;
    const uint32_t e = (top + 0x1FFFFFu) >> 23;
    return e < 8 ? 0u : e - 8;
}

// Eight values under a block's scale as E4M3 codes, the first in the low byte: nearest, ties to even.
__device__ __forceinline__ u32x2 codes8_e4m3(const float* x, uint32_t s) {
    if (s == 255) return u32x2{0, 0};
    const float inv = inverse_scale(s);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * inv, x[5] * inv, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * inv, x[7] * inv, hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
}

// The largest magnitude of the block of 32 that four neighbouring lanes hold, as fp32 bits.
__device__ __forceinline__ uint32_t block_top8(const float* x) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = umax(top, magnitude(x[i]));
    top = umax(top, quad<0xB1>(top));
    return umax(top, quad<0x4E>(top));
}

// ---------------------------------------------------------------- host side
inline int check_sides(int64_t rows, int64_t cols, const char* what) {
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return fail(ZERO_ERANGE, "%s: %lld x %lld out of range", what, (long long)rows, (long long)cols);
    return ZERO_OK;
}

// Places of values (rows x cols, row stride ld) and of an operand's codes and scales.
inline Place values_at(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
    const int64_t size = (int64_t)elem_bytes(dtype);
    return Place(p, rows, cols * size, ld * size);
}
inline Place codes_at(const void* p, int64_t rows, int64_t cols) { return Place(p, rows * (padded(cols) / 2)); }
inline Place codes8_at(const void* p, int64_t rows, int64_t cols) { return Place(p, rows * padded(cols)); }
inline Place scales_at(const void* p, int64_t rows, int64_t cols) { return Place(p, rows * (padded(cols) / kMxBlock)); }

// Whether a place shares memory with one of the others.
inline bool meets(const Place& p, std::initializer_list<Place> others) {
    for (const Place& o : others)
        if (overlap(p, o)) return true;
    return false;
}

}  // namespace
