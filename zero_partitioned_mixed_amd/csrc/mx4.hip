// MXFP4 operands: quantisation along rows and columns, the values back, and
// the product on the scaled matrix instructions of gfx950.
//
// An operand is [rows][P / 2] codes and [rows][P / 32] scales, P = cols rounded up
// to 128: rows start on 64 bytes, the four block scales of 128 elements are a
// dword, and the product needs no test for a ragged k (the padding is zero
// codes under the smallest scale).
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
// nearest, ties to even, saturating (what the conversion instruction does).
__device__ __forceinline__ uint32_t codes8(const float* x, float inv) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0] * inv, x[1] * inv, 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2] * inv, x[3] * inv, 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4] * inv, x[5] * inv, 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6] * inv, x[7] * inv, 1.0f, 3);
    return c;
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t v) {  // v of another lane of this group of four
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest magnitude of the 32 values that four neighbouring lanes hold.
__device__ __forceinline__ uint32_t block_top(const float* x) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = umax(top, magnitude(x[i]));
    top = umax(top, quad<0xB1>(top));  // lanes 1 0 3 2
    return umax(top, quad<0x4E>(top));  // lanes 2 3 0 1
}

// Eight elements of a row from column c on; past the row's end zeros.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* row, int64_t c, int64_t cols, float* x) {
    typedef typename Elem<DT>::type T;
    T v[8];
    if (VEC && c + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(v) / 16; ++i) ((u32x4*)v)[i] = *((const u32x4*)(row + c) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? row[c + i] : (T)0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float<DT>(v[i]);
}

struct QuantArgs {
    const void* src;
    int64_t rows, cols, ld;
    uint8_t *codes, *scales, *codes_t, *scales_t;
};

// Codes and scale of this lane's eight elements of a row (four lanes a block).
__device__ __forceinline__ void put_row8(const QuantArgs& a, int64_t r, int64_t c, int64_t p, const float* x) {
    const uint32_t s = scale_byte(block_top(x));
    *(uint32_t*)(a.codes + r * (p / 2) + c / 2) = s == 255 ? 0u : codes8(x, inverse_scale(s));
    if ((threadIdx.x & 3) == 0) a.scales[r * (p / kMxBlock) + c / kMxBlock] = (uint8_t)s;
}

// Along rows: eight elements per thread.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) mx4_rows_kernel(QuantArgs a) {
    const int64_t p = padded(a.cols), pieces = p / 8;
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = t / pieces, c = (t - r * pieces) * 8;
    if (r >= a.rows) return;  // whole groups of 16 lanes
    float x[8];
    load8<DT, VEC>((const typename Elem<DT>::type*)a.src + r * a.ld, c, a.cols, x);
    put_row8(a, r, c, p, x);
}

// Along columns, and along rows too where asked, from one read: a 128 x 128
// patch through LDS.  A thread then takes 32 elements of a column; four
// neighbouring lanes write 64 contiguous bytes of codes.  Every 32 rows start
// 16 columns further on, which keeps those four lanes on different banks.
constexpr int kPatch = 128;
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) mx4_cols_kernel(QuantArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr int kLd = kPatch + 16 / (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) T patch[kPatch * kLd + 3 * 16];
    const int64_t r0 = (int64_t)blockIdx.y * kPatch, c0 = (int64_t)blockIdx.x * kPatch;
    const int64_t p = padded(a.cols), pt = padded(a.rows);
    const int tid = threadIdx.x;
    auto at = [](int r, int c) { return r * kLd + (r / kMxBlock) * 16 + c; };
#pragma unroll
    for (int i = 0; i < kPatch; i += kThreads / 16) {
        const int r = i + tid / 16, c = (tid % 16) * 8;
        float x[8];
        if (r0 + r < a.rows) {
            load8<DT, VEC>((const T*)a.src + (r0 + r) * a.ld, c0 + c, a.cols, x);
            if (a.codes != nullptr) put_row8(a, r0 + r, c0 + c, p, x);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = 0.0f;
        }
        T v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = from_float<DT>(x[k]);
#pragma unroll
        for (int k = 0; k < (int)sizeof(v) / 16; ++k) *((u32x4*)(patch + at(r, c)) + k) = ((u32x4*)v)[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 64 + tid / 4, block = tid % 4;
        if (c0 + c >= a.cols) continue;
        float x[kMxBlock];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kMxBlock; ++k) {
            x[k] = to_float<DT>(patch[at(block * kMxBlock, c) + k * kLd]);
            top = umax(top, magnitude(x[k]));
        }
        const uint32_t s = scale_byte(top);
        const float inv = inverse_scale(s);
        u32x4 q;
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = s == 255 ? 0u : codes8(x + 8 * k, inv);
        const int64_t row = c0 + c, blk = r0 / kMxBlock + block;
        *(u32x4*)(a.codes_t + row * (pt / 2) + blk * (kMxBlock / 2)) = q;
        a.scales_t[row * (pt / kMxBlock) + blk] = (uint8_t)s;
    }
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    int64_t rows, cols, ld;
    void* dst;
};

__device__ __forceinline__ float code_value(uint32_t c) {  // 0 .5 1 1.5 2 3 4 6
    const uint32_t m = c & 1, e = (c >> 1) & 3;
    const float v = e == 0 ? 0.5f * (float)m : __builtin_bit_cast(float, ((e + 126) << 23) | (m << 22));
    return c & 8 ? -v : v;
}

// value * 2^(s - 127) with one rounding, in two exact-or-final steps.
__device__ __forceinline__ float scaled(float v, uint32_t s) {
    return s == 255 ? __builtin_nanf("") : ldexpf(v, (int)s - 127);
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) mx4_values_kernel(DequantArgs a) {
    typedef typename Elem<DT>::type T;
    const int64_t p = padded(a.cols), pieces = p / 8;
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = t / pieces, c = (t - r * pieces) * 8;
    if (r >= a.rows || c >= a.cols) return;
    const uint32_t q = *(const uint32_t*)(a.codes + r * (p / 2) + c / 2);
    const uint32_t s = a.scales[r * (p / kMxBlock) + c / kMxBlock];
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = from_float<DT>(scaled(code_value(q >> (4 * i)), s));
    T* dst = (T*)a.dst + r * a.ld + c;
    if (VEC && c + 8 <= a.cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(v) / 16; ++i) ((u32x4*)dst)[i] = ((u32x4*)v)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < a.cols) dst[i] = v[i];
    }
}

// ---------------------------------------------------------------- the product
struct MatmulArgs {
    const uint8_t *a, *sa, *b, *sb;
    int64_t m, n, p;  // p: padded k
    void* c;
    int64_t ldc;
    int tiles_m, tiles_n;
    int accumulate;
    int vector;  // rows of c aligned to four elements
};

template <class S, int DT>
__global__ void __launch_bounds__(S::THREADS) mx4_matmul_kernel(MatmulArgs g) {
    __shared__ __attribute__((aligned(16))) char lds[product_lds<S, MmFp4>()];
    int ti, tj;
    band_tile(xcd_tile(blockIdx.x, gridDim.x), g.tiles_m, g.tiles_n, ti, tj);
    const int64_t i0 = (int64_t)ti * S::TILE, j0 = (int64_t)tj * S::TILE;
    const int64_t left_m = g.m - i0, left_n = g.n - j0;
    const int rows_a = (int)(left_m < S::TILE ? left_m : S::TILE), rows_b = (int)(left_n < S::TILE ? left_n : S::TILE);
    const uint32_t ld = (uint32_t)(g.p / 2), ls = (uint32_t)(g.p / kMxBlock);
    const Operand A{(const char*)g.a + i0 * ld, ld, rows_a}, B{(const char*)g.b + j0 * ld, ld, rows_b};
    const Operand SA{(const char*)g.sa + i0 * ls, ls, rows_a}, SB{(const char*)g.sb + j0 * ls, ls, rows_b};
    f32x16 acc[S::MT][S::NT];
    if (!tile_product<S, MmFp4>(A, B, SA, SB, (int)(g.p / 256), g.p % 256 != 0, lds, acc)) return;

    typedef typename Elem<DT>::type T;
    const Lane L(S::WAVES);
    const int64_t iw = i0 + L.wave / (S::TILE / S::WN) * S::WM, jw = j0 + L.wave % (S::TILE / S::WN) * S::WN;
#pragma unroll
    for (int ii = 0; ii < S::MT; ++ii)
#pragma unroll
        for (int jj = 0; jj < S::NT; ++jj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[ii][jj][4 * q + r];
                quad_turn(v);  // four columns of one row
                const int64_t i = iw + ii * 32 + 8 * q + 4 * L.h + (L.c & 3), j = jw + jj * 32 + (L.c & ~3);
                if (i >= g.m || j >= g.n) continue;
                T* out = (T*)g.c + i * g.ldc + j;
                if (g.vector && j + 4 <= g.n) {
                    typedef T T4 __attribute__((ext_vector_type(4)));
                    T4 w;
                    if constexpr (DT == ZERO_F32) {
                        if (g.accumulate) {
                            w = *(const T4*)out;
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] += w[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = from_float<DT>(v[e]);
                    *(T4*)out = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (j + e >= g.n) break;
                        if constexpr (DT == ZERO_F32) {
                            if (g.accumulate) v[e] += out[e];
                        }
                        out[e] = from_float<DT>(v[e]);
                    }
                }
            }
}

// ---------------------------------------------------------------- host side
int check_sides(int64_t rows, int64_t cols, const char* what) {
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return fail(ZERO_ERANGE, "%s: %lld x %lld out of range", what, (long long)rows, (long long)cols);
    return ZERO_OK;
}

bool vector_rows(const void* p, int64_t ld, int32_t dtype) {
    return aligned(p, 16) && (ld * (int64_t)elem_bytes(dtype)) % 16 == 0;
}

template <int DT>
int quantize_with(const QuantArgs& a, hipStream_t s, const char* what) {
    const bool vec = vector_rows(a.src, a.ld, DT);
    if (a.codes_t == nullptr) {
        const int64_t wgs = ceil_div(a.rows * (padded(a.cols) / 8), kThreads);
        if (wgs > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
        return launch(vec ? mx4_rows_kernel<DT, true> : mx4_rows_kernel<DT, false>, dim3((unsigned)wgs), kThreads, s,
                      a, what);
    }
    const int64_t gx = ceil_div(a.cols, kPatch), gy = ceil_div(a.rows, kPatch);
    if (gy > 65535) return fail(ZERO_ERANGE, "%s: too many rows to quantise along columns", what);
    return launch(vec ? mx4_cols_kernel<DT, true> : mx4_cols_kernel<DT, false>, dim3((unsigned)gx, (unsigned)gy),
                  kThreads, s, a, what);
}

int quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void* codes, void* scales,
             void* codes_t, void* scales_t, hipStream_t s, const char* what) {
    const QuantArgs a{src, rows, cols, ld, (uint8_t*)codes, (uint8_t*)scales, (uint8_t*)codes_t, (uint8_t*)scales_t};
    switch (dtype) {
        case ZERO_F16: return quantize_with<ZERO_F16>(a, s, what);
        case ZERO_BF16: return quantize_with<ZERO_BF16>(a, s, what);
        default: return quantize_with<ZERO_F32>(a, s, what);
    }
}

template <class S>
int matmul_with(MatmulArgs g, int32_t c_dtype, hipStream_t s, const char* what) {
    const int64_t tm = ceil_div(g.m, S::TILE), tn = ceil_div(g.n, S::TILE);
    if (tm * tn > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many tiles for one launch", what);
    g.tiles_m = (int)tm;
    g.tiles_n = (int)tn;
    g.vector = aligned(g.c, 4 * elem_bytes(c_dtype)) && g.ldc % 4 == 0;
    const dim3 grid((unsigned)(tm * tn));
    switch (c_dtype) {
        case ZERO_F16: return launch(mx4_matmul_kernel<S, ZERO_F16>, grid, S::THREADS, s, g, what);
        case ZERO_BF16: return launch(mx4_matmul_kernel<S, ZERO_BF16>, grid, S::THREADS, s, g, what);
        default: return launch(mx4_matmul_kernel<S, ZERO_F32>, grid, S::THREADS, s, g, what);
    }
}

int matmul(const MatmulArgs& g, int32_t c_dtype, hipStream_t s, const char* what) {
    const int pick = pick_tile([&](int64_t t) { return ceil_div(g.m, t) * ceil_div(g.n, t); });
    return with_tile(pick, [&](auto shape) { return matmul_with<decltype(shape)>(g, c_dtype, s, what); });
}

// The checks shared by the products; 1: nothing to do.
int check_matmul(const void* b, const void* sb, int64_t m, int64_t n, int64_t k, const void* c, int32_t c_dtype,
                 int64_t ldc, const char* what) {
    if (!valid_dtype(c_dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    int rc;
    if ((rc = check_sides(m, n, what)) != ZERO_OK || (rc = check_sides(k, k, what)) != ZERO_OK) return rc;
    if (m == 0 || n == 0) return 1;
    if (c == nullptr || (k > 0 && (b == nullptr || sb == nullptr)))
        return fail(ZERO_EINVAL, "%s: null operand or result", what);
    if (!aligned(b, 16) || !aligned(sb, 16)) return fail(ZERO_EALIGN, "%s: operands not 16-byte aligned", what);
    if (!aligned(c, elem_bytes(c_dtype))) return fail(ZERO_EALIGN, "%s: result not aligned to its elements", what);
    if (ldc < n) return fail(ZERO_ERANGE, "%s: row stride below n", what);
    return ZERO_OK;
}

size_t quantized_bytes(int64_t rows, int64_t cols) {
    return (size_t)(round_up(rows * (padded(cols) / 2), 256) + round_up(rows * (padded(cols) / kMxBlock), 256));
}

}  // namespace

extern "C" {

int64_t zero_mx4_padded(int64_t cols) { return cols <= 0 ? 0 : padded(cols); }

size_t zero_mx4_code_bytes(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 ? 0 : (size_t)(rows * (padded(cols) / 2));
}

size_t zero_mx4_scale_bytes(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 ? 0 : (size_t)(rows * (padded(cols) / kMxBlock));
}

int zero_mx4_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void* codes,
                      void* scales, void* codes_t, void* scales_t, void* stream) {
    const char* what = "zero_mx4_quantize";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_sides(rows, cols, what)) != ZERO_OK) return rc;
    if (ld < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
        return fail(ZERO_EINVAL, "%s: codes and scales come in pairs", what);
    if (codes == nullptr && codes_t == nullptr) return fail(ZERO_EINVAL, "%s: no output", what);
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(codes_t, 16) || !aligned(scales_t, 16))
        return fail(ZERO_EALIGN, "%s: outputs not 16-byte aligned", what);
    if (rows == 0 || cols == 0) return ok();
    if (src == nullptr) return fail(ZERO_EINVAL, "%s: null source", what);
    if (!aligned(src, elem_bytes(dtype))) return fail(ZERO_EALIGN, "%s: source not aligned to its elements", what);
    return quantize(src, dtype, rows, cols, ld, codes, scales, codes_t, scales_t, (hipStream_t)stream, what);
}

int zero_mx4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, void* dst, int32_t dtype,
                        int64_t ld, void* stream) {
    const char* what = "zero_mx4_dequantize";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_sides(rows, cols, what)) != ZERO_OK) return rc;
    if (ld < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (rows == 0 || cols == 0) return ok();
    if (codes == nullptr || scales == nullptr || dst == nullptr) return fail(ZERO_EINVAL, "%s: null buffer", what);
    if (!aligned(codes, 16) || !aligned(scales, 16)) return fail(ZERO_EALIGN, "%s: operand not 16-byte aligned", what);
    if (!aligned(dst, elem_bytes(dtype))) return fail(ZERO_EALIGN, "%s: result not aligned to its elements", what);
    const DequantArgs a{(const uint8_t*)codes, (const uint8_t*)scales, rows, cols, ld, dst};
    const int64_t wgs = ceil_div(rows * (padded(cols) / 8), kThreads);
    if (wgs > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    const dim3 grid((unsigned)wgs);
    const hipStream_t s = (hipStream_t)stream;
    const bool vec = vector_rows(dst, ld, dtype);
    switch (dtype) {
        case ZERO_F16:
            return launch(vec ? mx4_values_kernel<ZERO_F16, true> : mx4_values_kernel<ZERO_F16, false>, grid, kThreads, s, a, what);
        case ZERO_BF16:
            return launch(vec ? mx4_values_kernel<ZERO_BF16, true> : mx4_values_kernel<ZERO_BF16, false>, grid, kThreads, s, a, what);
        default:
            return launch(vec ? mx4_values_kernel<ZERO_F32, true> : mx4_values_kernel<ZERO_F32, false>, grid, kThreads, s, a, what);
    }
}

size_t zero_mx4_matmul_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

int zero_mx4_matmul(const void* a, const void* sa, const void* b, const void* sb, int64_t m, int64_t n, int64_t k,
                    void* c, int32_t c_dtype, int64_t ldc, int32_t accumulate, void*, size_t, void* stream) {
    const char* what = "zero_mx4_matmul";
    if (accumulate != 0 && (accumulate != 1 || c_dtype != ZERO_F32))
        return fail(ZERO_EINVAL, "%s: accumulate is 0, or 1 with an fp32 result", what);
    const int rc = check_matmul(b, sb, m, n, k, c, c_dtype, ldc, what);
    if (rc == 1) return ok();
    if (rc != ZERO_OK) return rc;
    if (k > 0 && (a == nullptr || sa == nullptr)) return fail(ZERO_EINVAL, "%s: null operand", what);
    if (!aligned(a, 16) || !aligned(sa, 16)) return fail(ZERO_EALIGN, "%s: operands not 16-byte aligned", what);
    const MatmulArgs g{(const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b, (const uint8_t*)sb,
                       m, n, padded(k), c, ldc, 0, 0, accumulate, 0};
    return matmul(g, c_dtype, (hipStream_t)stream, what);
}

size_t zero_mx4_matmul_rows_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m <= 0 || n <= 0 || k <= 0 || m > ZERO_MX4_ROWS_MAX || n > kMaxSide || k > kMaxSide) return 0;
    return quantized_bytes(m, k);
}

int zero_mx4_matmul_rows(const void* a, int32_t a_dtype, int64_t lda, const void* b, const void* sb, int64_t m,
                         int64_t n, int64_t k, void* c, int32_t c_dtype, int64_t ldc, void* ws, size_t ws_bytes,
                         void* stream) {
    const char* what = "zero_mx4_matmul_rows";
    if (!valid_dtype(a_dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    int rc = check_matmul(b, sb, m, n, k, c, c_dtype, ldc, what);
    if (m > ZERO_MX4_ROWS_MAX) return fail(ZERO_ERANGE, "%s: %lld rows, at most %d", what, (long long)m, ZERO_MX4_ROWS_MAX);
    if (rc == 1) return ok();
    if (rc != ZERO_OK) return rc;
    if (k > 0 && a == nullptr) return fail(ZERO_EINVAL, "%s: null operand", what);
    if (!aligned(a, elem_bytes(a_dtype))) return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    if (lda < k) return fail(ZERO_ERANGE, "%s: row stride below k", what);
    const size_t need = zero_mx4_matmul_rows_workspace_bytes(m, n, k);
    if (need > 0) {
        if (ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
        if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
        if (ws_bytes < need) return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
    }
    uint8_t* codes = (uint8_t*)ws;
    uint8_t* scales = codes + round_up(m * (padded(k) / 2), 256);
    if (k > 0 && (rc = quantize(a, a_dtype, m, k, lda, codes, scales, nullptr, nullptr, (hipStream_t)stream, what)) != ZERO_OK)
        return rc;
    const MatmulArgs g{codes, scales, (const uint8_t*)b, (const uint8_t*)sb, m, n, padded(k), c, ldc, 0, 0, 0, 0};
    return matmul(g, c_dtype, (hipStream_t)stream, what);
}

}  // extern "C"
