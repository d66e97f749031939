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

struct QuantArgs {
    const void* src;
    int64_t rows, cols, ld;
    uint8_t *codes, *scales, *codes_t, *scales_t;
};

// One or two matrices in one launch: workgroups from `second` on take the second.
struct QuantJobs {
    QuantArgs job[2];
    uint32_t across[2];  // patches in a row of patches
    uint32_t second;
};

// Codes and scale of this lane's eight elements of a row (four lanes a block).
template <int DT>
__device__ __forceinline__ void put_row8(const QuantArgs& a, int64_t r, int64_t c, int64_t p, const Eight<DT>& e) {
    const uint32_t s = scale_byte(e.block_top());
    *(uint32_t*)(a.codes + r * (p / 2) + c / 2) = e.codes(s);
    if ((threadIdx.x & 3) == 0) a.scales[r * (p / kMxBlock) + c / kMxBlock] = (uint8_t)s;
}

// A patch of ROWS x 128 elements per workgroup, sixteen lanes to a row, all its loads
// before the first use.  Along rows four lanes hold a block.  Along columns (COLS)
// the patch goes through LDS and a thread takes 32 elements of a column.  A row is
// eight banks further on than the one before and every 32 rows another 32, so
// the four rows that sixteen lanes read, and their neighbours', differ.  Bound
// by memory: both directions of 8192 x 8192 bf16 read and write 205 MB.
template <int DT, int ROWS, bool COLS>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(QuantJobs jobs) {
    typedef typename Elem<DT>::type T;
    constexpr int kCols = kMxPad, kLd = kCols + (DT == ZERO_F32 ? 4 : 16), kSkip = DT == ZERO_F32 ? 16 : 64, kLoads = ROWS / 16;
    __shared__ __attribute__((aligned(16))) T patch[COLS ? ROWS * kLd + (ROWS / 32 - 1) * kSkip : 8];
    const bool other = blockIdx.x >= jobs.second;
    const QuantArgs& a = jobs.job[other];
    const uint32_t wg = other ? blockIdx.x - jobs.second : blockIdx.x, across = jobs.across[other];
    const int64_t r0 = (int64_t)(wg / across) * ROWS, c0 = (int64_t)(wg % across) * kCols;
    const int64_t p = padded(a.cols), pt = padded(a.rows);
    const int tid = threadIdx.x, r = tid / 16, c = tid % 16 * 8;
    auto at = [](int row, int col) { return row * kLd + row / kMxBlock * kSkip + col; };
    Eight<DT> e[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t row = r0 + r + 16 * i;
        if (row < a.rows)
            e[i].load((const T*)a.src + row * a.ld, c0 + c, a.cols);
        else
            e[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = r + 16 * i;
        if constexpr (COLS) {
#pragma unroll
            for (int k = 0; k < Eight<DT>::kVecs; ++k) *((u32x4*)(patch + at(row, c)) + k) = e[i].v[k];
        }
        if ((!COLS || a.codes != nullptr) && r0 + row < a.rows) put_row8<DT>(a, r0 + row, c0 + c, p, e[i]);
    }
    if constexpr (COLS) {
        __syncthreads();
        // sixteen lanes a block of 32 rows and sixteen columns, a column each
        constexpr int kBlocks = ROWS / kMxBlock, kGroups = kThreads / 16;
#pragma unroll
        for (int t = tid / 16; t < kCols / 16 * kBlocks; t += kGroups) {
            const int col0 = t / kBlocks * 16, col = col0 + tid % 16, block = t % kBlocks;
            uint32_t s;
            u32x4 q;
            if constexpr (DT == ZERO_F32) {
                float x[kMxBlock];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < kMxBlock; ++k) {
                    x[k] = patch[at(block * kMxBlock, col) + k * kLd];
                    top = umax(top, magnitude(x[k]));
                }
                s = scale_byte(top);
                const float inv = inverse_scale(s);
#pragma unroll
                for (int k = 0; k < 4; ++k) q[k] = s == 255 ? 0u : codes8(x + 8 * k, inv);
            } else {
                // LDS reads that turn 4 rows x 16 columns: four values of the lane's column
                typedef int16_t s16x4 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) s16x4* Place;
                const T* from = patch + at(block * kMxBlock + tid % 16 / 4, col0 + tid % 4 * 4);
                uint32_t d[kMxBlock / 2];
#pragma unroll
                for (int k = 0; k < kMxBlock / 4; ++k) {
                    const u32x2 w =
                        __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Place)(from + 4 * k * kLd)));
                    d[2 * k] = w[0];
                    d[2 * k + 1] = w[1];
                }
                s = scale_byte(top16<DT, kMxBlock / 2>(d));
                if (s >= kLowScale) {
                    const float scale = __builtin_bit_cast(float, s << 23);
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = s == 255 ? 0u : codes8_16<DT>(d + 4 * k, scale);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        Eight<DT> e;
                        __builtin_memcpy(e.v, d + 4 * k, sizeof(e.v));
                        q[k] = e.codes(s);
                    }
                }
            }
            if (c0 + col < a.cols) {
                const int64_t row = c0 + col, blk = r0 / kMxBlock + block;
                *(u32x4*)(a.codes_t + row * (pt / 2) + blk * (kMxBlock / 2)) = q;
                a.scales_t[row * (pt / kMxBlock) + blk] = (uint8_t)s;
            }
        }
    }
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    int64_t rows, cols, ld;
    void* dst;
};

// Eight codes times 2^(s - 127), the scaling with one rounding for results below the
// normal numbers.
__device__ __forceinline__ void values8(uint32_t q, uint32_t s, float* x) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3)};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s == 255 ? __builtin_nanf("") : ldexpf(v[i / 2][i % 2], (int)s - 127);
}

// 64 rows x 128 columns per workgroup, sixteen lanes to a row.
constexpr int kValueRows = 64;
template <int DT>
__global__ void __launch_bounds__(kThreads) mx4_values_kernel(DequantArgs a) {
    typedef typename Elem<DT>::type T;
    const int64_t p = padded(a.cols);
    const uint32_t across = (uint32_t)(p / kMxPad);
    const int64_t r0 = (int64_t)(blockIdx.x / across) * kValueRows + threadIdx.x / 16;
    const int64_t c = (int64_t)(blockIdx.x % across) * kMxPad + threadIdx.x % 16 * 8;
    if (c >= a.cols) return;
    constexpr int kEach = kValueRows / 16;
    uint32_t q[kEach], s[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t r = r0 + 16 * i < a.rows ? r0 + 16 * i : a.rows - 1;
        q[i] = *(const uint32_t*)(a.codes + r * (p / 2) + c / 2);
        s[i] = a.scales[r * (p / kMxBlock) + c / kMxBlock];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (r0 + 16 * i >= a.rows) return;
        float x[8];
        values8(q[i], s[i], x);
        T v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = from_float<DT>(x[k]);
        T* dst = (T*)a.dst + (r0 + 16 * i) * a.ld + c;
        if (c + 8 <= a.cols) {  // whole vectors at any alignment
            u32x4 w[sizeof(v) / 16];
            __builtin_memcpy(w, v, sizeof(v));
#pragma unroll
            for (int k = 0; k < (int)sizeof(v) / 16; ++k) {
                asm volatile("" : "+v"(w[k]));  // one store, not the pieces it was made of
                __builtin_memcpy((char*)dst + 16 * k, &w[k], 16);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < a.cols) dst[k] = v[k];
        }
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
    Product<S, MmFp4> product(lds, (int)(g.p / 256), g.p % 256 != 0);
    product.tile(Operand{(const char*)g.a + i0 * ld, ld, rows_a}, Operand{(const char*)g.b + j0 * ld, ld, rows_b},
                 Operand{(const char*)g.sa + i0 * ls, ls, rows_a}, Operand{(const char*)g.sb + j0 * ls, ls, rows_b});
    product.ahead();
    f32x16 acc[S::MT][S::NT];
    if (!product.run(acc)) return;

    // A lane's place in the tile: 32-bit offsets from the tile's first element.
    typedef typename Elem<DT>::type T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    const Lane& L = product.L;
    const int iw = L.wave / (S::TILE / S::WN) * S::WM + 4 * L.h + (L.c & 3);
    const int jw = L.wave % (S::TILE / S::WN) * S::WN + (L.c & ~3);
    T* const out = (T*)g.c + i0 * g.ldc + j0;
    const bool whole = g.vector && rows_a == S::TILE && rows_b == S::TILE;
#pragma unroll
    for (int ii = 0; ii < S::MT; ++ii)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = iw + ii * 32 + 8 * q;
            T* const row = out + i * g.ldc + jw;
#pragma unroll
            for (int jj = 0; jj < S::NT; ++jj) {
                const int j = jw + jj * 32;
                T* const at = row + jj * 32;
                const bool vector = whole || (g.vector && i < rows_a && j + 4 <= rows_b);
                T4 w;  // four columns of one row
                if constexpr (DT == ZERO_F32) {
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = acc[ii][jj][4 * q + r];
                    quad_turn(v);
                    if (g.accumulate) {
                        if (vector) {
                            w = *(const T4*)at;
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] += w[e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (i < rows_a && j + e < rows_b) v[e] += at[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = v[e];
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[r] = from_float<DT>(acc[ii][jj][4 * q + r]);
                    w = __builtin_bit_cast(T4, quad_turn16(__builtin_bit_cast(u32x2, w)));
                }
                if (vector) {
                    *(T4*)at = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i < rows_a && j + e < rows_b) at[e] = w[e];
                }
            }
        }
}

// Few rows (m <= 32, as single tokens bring): bound by reading B once.  A workgroup
// takes 32 of B's rows, its eight waves an eighth of k each: a wave brings its own
// slabs to its own part of LDS (whole lines; 16 bytes per lane straight to
// registers touch a line per lane), waits for nobody, and the waves' sums meet in LDS.
// One token, 11008 x 4096: 5.9 us, where reading B takes 5; the waves wait for 57% of their
// cycles, 3% for LDS.
// VALUES (m k up to kFewValues): A comes as values, and every workgroup quantises
// all of it to LDS first, which saves a launch.
constexpr int kFewWaves = 8;
constexpr int kFewValues = 16384;
constexpr int kFewSlabs = 2;   // slabs of a wave on their way at once

struct FewArgs {
    MatmulArgs g;
    int64_t lda, k;  // values of A: row stride, length
};

template <int DTA, int DT, bool VALUES>
__global__ void __launch_bounds__(kFewWaves * 64) mx4_few_kernel(FewArgs f) {
    const MatmulArgs& g = f.g;
    constexpr int kCodes = VALUES ? kFewValues / 2 : 16, kScales = kCodes / 16;
    __shared__ __attribute__((aligned(16))) uint8_t codes[kCodes];
    __shared__ __attribute__((aligned(16))) uint8_t scales[VALUES ? kScales : 16];
    constexpr int kRing = kFewWaves * kFewSlabs * 32 * kSlab, kSums = kFewWaves * 32 * 33 * 4;
    __shared__ __attribute__((aligned(16))) char lds[kRing > kSums ? kRing : kSums];
    float(*sums)[32][33] = (float(*)[32][33])lds;  // after the products
    const Lane L;
    const uint32_t p = (uint32_t)g.p, half_row = p / 2, scale_row = p / kMxBlock;
    const int64_t j = (int64_t)blockIdx.x * 32 + L.c;
    const int64_t jc = j < g.n ? j : g.n - 1;
    const uint8_t *b = g.b + jc * half_row + 64 * L.h, *sb = g.sb + jc * scale_row + 4 * L.h;
    const int slabs = (int)(p / 256);

    // A wave fetches only slabs that it then waits for: the waves' sums overwrite the ring.
    char* const ring = lds + L.wave * kFewSlabs * 32 * kSlab;
    const bool any = L.wave < slabs;
    uint32_t bs[kFewSlabs];
    auto fetch = [&](int first) {
#pragma unroll
        for (int u = 0; u < kFewSlabs; ++u) {
            const int s = first + u * kFewWaves < slabs ? first + u * kFewWaves : slabs - 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // eight rows each
                const int r = 8 * q + (L.lane >> 3);
                const int64_t row = (int64_t)blockIdx.x * 32 + r;
                const uint32_t piece = (L.lane & 7) ^ ((r >> 1) & 7);
                load_to_lds16((const char*)g.b + (row < g.n ? row : g.n - 1) * half_row + (int64_t)s * kSlab + piece * 16,
                              ring + u * 32 * kSlab + q * 1024);
            }
            bs[u] = *(const uint32_t*)(sb + (int64_t)s * 8);
        }
    };
    if constexpr (VALUES) {
        typedef typename Elem<DTA>::type T;
        const int pieces = (int)(g.m * p / 8);
        auto read = [&](int t, Eight<DTA>& e) {
            const uint32_t r = (uint32_t)t / (p / 8), c = ((uint32_t)t - r * (p / 8)) * 8;
            e.load((const T*)g.a + r * f.lda, c, f.k);
        };
        auto put = [&](int t, const Eight<DTA>& e) {  // whole groups of four lanes
            const uint32_t r = (uint32_t)t / (p / 8), c = ((uint32_t)t - r * (p / 8)) * 8;
            const uint32_t s = scale_byte(e.block_top());
            *(uint32_t*)(codes + r * half_row + c / 2) = e.codes(s);
            if ((t & 3) == 0) scales[r * scale_row + c / kMxBlock] = (uint8_t)s;
        };
        // loads return in order: the first of A go out before B's, so that A is ready while B is on its way
        constexpr int kFirst = 2;
        const int tid = threadIdx.x;
        Eight<DTA> e[kFirst];
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
            if (tid + i * kFewWaves * 64 < pieces) read(tid + i * kFewWaves * 64, e[i]);
        if (any) fetch(L.wave);
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
            if (tid + i * kFewWaves * 64 < pieces) put(tid + i * kFewWaves * 64, e[i]);
        for (int t = tid + kFirst * kFewWaves * 64; t < pieces; t += kFewWaves * 64) {
            read(t, e[0]);
            put(t, e[0]);
        }
        __syncthreads();
    } else {
        if (any) fetch(L.wave);
    }
    const uint8_t *a = VALUES ? codes : g.a, *sa = VALUES ? scales : g.sa;
    const uint32_t row = (uint32_t)(L.c < g.m ? L.c : g.m - 1);
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;

    for (int first = L.wave; first < slabs; first += kFewWaves * kFewSlabs) {
        if (first != L.wave) fetch(first);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's slabs are in its part of LDS
#pragma unroll
        for (int u = 0; u < kFewSlabs; ++u) {
            const int s = first + u * kFewWaves;
            if (s >= slabs) break;
            const char* from = ring + u * 32 * kSlab + L.c * kSlab;
            i32x4 bw[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) bw[q] = *(const i32x4*)(from + (((4 * L.h + q) ^ ((L.c >> 1) & 7)) << 4));
            const uint32_t as = *(const uint32_t*)(sa + row * scale_row + s * 8 + 4 * L.h);
            const i32x4* aw = (const i32x4*)(a + row * half_row + s * 128 + 64 * L.h);
            acc = MmFp4::mma<0>(aw[0], bw[0], acc, as, bs[u]);
            acc = MmFp4::mma<1>(aw[1], bw[1], acc, as, bs[u]);
            acc = MmFp4::mma<2>(aw[2], bw[2], acc, as, bs[u]);
            acc = MmFp4::mma<3>(aw[3], bw[3], acc, as, bs[u]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next slabs come
    }
    if (p % 256 != 0 && L.wave == 0) {  // half a slab: group h takes blocks 2h and 2h + 1 of four
        const int64_t at = (int64_t)slabs * 128 - 32 * L.h, sat = (int64_t)slabs * 8 - 4 * L.h;
        const uint32_t bsh = *(const uint32_t*)(sb + sat) >> (16 * L.h);
        const i32x4 b0 = *(const i32x4*)(b + at), b1 = *(const i32x4*)(b + at + 16);
        const uint32_t as = *(const uint32_t*)(sa + row * scale_row + slabs * 8) >> (16 * L.h);
        const i32x4* aw = (const i32x4*)(a + row * half_row + slabs * 128 + 32 * L.h);
        acc = MmFp4::mma<0>(aw[0], b0, acc, as, bsh);
        acc = MmFp4::mma<1>(aw[1], b1, acc, as, bsh);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no slab is on its way
    __syncthreads();                                  // nor has one a reader any more
#pragma unroll
    for (int r = 0; r < 16; ++r) sums[L.wave][8 * (r / 4) + 4 * L.h + r % 4][L.c] = acc[r];
    __syncthreads();
    typedef typename Elem<DT>::type T;
    for (int t = threadIdx.x; t < (int)g.m * 32; t += kFewWaves * 64) {
        const int i = t / 32, c = t % 32;
        const int64_t col = (int64_t)blockIdx.x * 32 + c;
        if (col >= g.n) continue;
        float v = sums[0][i][c];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += sums[w][i][c];
        T* out = (T*)g.c + i * g.ldc + col;
        if constexpr (DT == ZERO_F32) {
            if (g.accumulate) v += *out;
        }
        *out = from_float<DT>(v);
    }
}

// ---------------------------------------------------------------- host side
int check_sides(int64_t rows, int64_t cols, const char* what) {
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return fail(ZERO_ERANGE, "%s: %lld x %lld out of range", what, (long long)rows, (long long)cols);
    return ZERO_OK;
}

// One or two matrices of one type (the second may be absent: rows 0), along rows or,
// where the first asks for its transpose, along columns too.
template <int DT>
int quantize_with(const QuantArgs* jobs, int count, hipStream_t s, const char* what) {
    QuantJobs q{};
    for (int i = 0; i < count; ++i) {
        q.job[i] = jobs[i];
        q.across[i] = (uint32_t)(padded(jobs[i].cols) / kMxPad);
    }
    const bool cols = jobs[0].codes_t != nullptr;
    auto patches = [&](int i, int64_t rows) -> int64_t {  // along columns the padding of the rows too
        return i < count ? ceil_div(cols ? padded(jobs[i].rows) : jobs[i].rows, rows) * q.across[i] : 0;
    };
    // Patches of 32 rows where those of 128 would leave CUs without work: 500 x 768 and
    // 1024 x 768 together, 5 against 7 us; at 8192 x 8192 they write the transposed
    // codes in runs of 16 bytes, not 64.
    const int high = !cols ? 64 : patches(0, 128) + patches(1, 128) >= 512 ? 128 : 32;
    const int64_t first = patches(0, high), all = first + patches(1, high);
    if (all > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    q.second = (uint32_t)first;
    const dim3 grid((unsigned)all);
    if (high == 64) return launch(mx4_quantize_kernel<DT, 64, false>, grid, kThreads, s, q, what);
    if (high == 128) return launch(mx4_quantize_kernel<DT, 128, true>, grid, kThreads, s, q, what);
    return launch(mx4_quantize_kernel<DT, 32, true>, grid, kThreads, s, q, what);
}

// Places of values (rows x cols, row stride ld) and of an operand's codes and scales.
Place values_at(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
    const int64_t size = (int64_t)elem_bytes(dtype);
    return Place(p, rows, cols * size, ld * size);
}
Place codes_at(const void* p, int64_t rows, int64_t cols) { return Place(p, rows * (padded(cols) / 2)); }
Place scales_at(const void* p, int64_t rows, int64_t cols) { return Place(p, rows * (padded(cols) / kMxBlock)); }

int quantize(const QuantArgs* jobs, int count, int32_t dtype, hipStream_t s, const char* what) {
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j) {
            const Place from = values_at(jobs[i].src, dtype, jobs[i].rows, jobs[i].cols, jobs[i].ld);
            const int64_t rows = jobs[j].rows, cols = jobs[j].cols;
            if (overlap(from, codes_at(jobs[j].codes, rows, cols)) || overlap(from, scales_at(jobs[j].scales, rows, cols)) ||
                overlap(from, codes_at(jobs[j].codes_t, cols, rows)) || overlap(from, scales_at(jobs[j].scales_t, cols, rows)))
                return fail(ZERO_EINVAL, "%s: codes or scales overlap the values", what);
        }
    switch (dtype) {
        case ZERO_F16: return quantize_with<ZERO_F16>(jobs, count, s, what);
        case ZERO_BF16: return quantize_with<ZERO_BF16>(jobs, count, s, what);
        default: return quantize_with<ZERO_F32>(jobs, count, s, what);
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

template <int DTA, bool VALUES>
int few_with(const FewArgs& f, int32_t c_dtype, hipStream_t s, const char* what) {
    const dim3 grid((unsigned)ceil_div(f.g.n, 32));
    switch (c_dtype) {
        case ZERO_F16: return launch(mx4_few_kernel<DTA, ZERO_F16, VALUES>, grid, kFewWaves * 64, s, f, what);
        case ZERO_BF16: return launch(mx4_few_kernel<DTA, ZERO_BF16, VALUES>, grid, kFewWaves * 64, s, f, what);
        default: return launch(mx4_few_kernel<DTA, ZERO_F32, VALUES>, grid, kFewWaves * 64, s, f, what);
    }
}

// Values of A quantised in the product's own kernel.
bool few_values(int64_t m, int64_t k) { return m <= 32 && m * padded(k) <= kFewValues; }

int few_of_values(const FewArgs& f, int32_t a_dtype, int32_t c_dtype, hipStream_t s, const char* what) {
    switch (a_dtype) {
        case ZERO_F16: return few_with<ZERO_F16, true>(f, c_dtype, s, what);
        case ZERO_BF16: return few_with<ZERO_BF16, true>(f, c_dtype, s, what);
        default: return few_with<ZERO_F32, true>(f, c_dtype, s, what);
    }
}

int matmul(const MatmulArgs& g, int32_t c_dtype, hipStream_t s, const char* what) {
    const Place c = values_at(g.c, c_dtype, g.m, g.n, g.ldc);
    if (overlap(c, codes_at(g.a, g.m, g.p)) || overlap(c, scales_at(g.sa, g.m, g.p)) || overlap(c, codes_at(g.b, g.n, g.p)) ||
        overlap(c, scales_at(g.sb, g.n, g.p)))
        return fail(ZERO_EINVAL, "%s: the result overlaps an operand", what);
    // Few rows against tiles of 64, us of operands in a replayed graph: 11008 x 4096, 8 rows 6.7, 9 to 32 rows by
    // tiles 7.5; where the tiles leave half of the CUs out, 4096 x 11008, 1 row 7.2, 32 rows 10.6, 33 to 64 rows by
    // tiles 13.6.  Where both fill the CUs tiles win from 9 rows on (11008 x 4096, 16 rows: 9.8 and 9.1, whole calls).
    if (g.m <= 8 || (g.m <= 32 && g.n <= 64 * 128)) return few_with<ZERO_F32, false>(FewArgs{g, 0, 0}, c_dtype, s, what);
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

// Where an operand's codes and scales are in one buffer of zero_mx4_operand_bytes.
struct Operand2 {
    uint8_t *codes, *scales;
    Operand2(void* at, int64_t rows, int64_t cols)
        : codes((uint8_t*)at),
          scales(at == nullptr ? nullptr : (uint8_t*)at + round_up(rows * (padded(cols) / 2), 256)) {}
};

int check_operands(const void* x_t, const void* w_t, const void* ws, size_t ws_bytes, size_t need, const char* what) {
    if (!aligned(x_t, 16) || !aligned(w_t, 16)) return fail(ZERO_EALIGN, "%s: operands not 16-byte aligned", what);
    if (ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
    if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
    if (ws_bytes < need) return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
    return ZERO_OK;
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
    const QuantArgs job{src, rows, cols, ld, (uint8_t*)codes, (uint8_t*)scales, (uint8_t*)codes_t, (uint8_t*)scales_t};
    return quantize(&job, 1, dtype, (hipStream_t)stream, what);
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
    const Place to = values_at(dst, dtype, rows, cols, ld);
    if (overlap(to, codes_at(codes, rows, cols)) || overlap(to, scales_at(scales, rows, cols)))
        return fail(ZERO_EINVAL, "%s: the result overlaps the operand", what);
    const DequantArgs a{(const uint8_t*)codes, (const uint8_t*)scales, rows, cols, ld, dst};
    const int64_t wgs = ceil_div(rows, kValueRows) * (padded(cols) / kMxPad);
    if (wgs > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    const dim3 grid((unsigned)wgs);
    const hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
        case ZERO_F16:
            return launch(mx4_values_kernel<ZERO_F16>, grid, kThreads, s, a, what);
        case ZERO_BF16:
            return launch(mx4_values_kernel<ZERO_BF16>, grid, kThreads, s, a, what);
        default:
            return launch(mx4_values_kernel<ZERO_F32>, grid, kThreads, s, a, what);
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
    return few_values(m, k) ? 0 : quantized_bytes(m, k);
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
    const Place to = values_at(c, c_dtype, m, n, ldc);
    if (overlap(to, values_at(a, a_dtype, m, k, lda)) || overlap(to, codes_at(b, n, k)) || overlap(to, scales_at(sb, n, k)))
        return fail(ZERO_EINVAL, "%s: the result overlaps an operand", what);
    MatmulArgs g{(const uint8_t*)a, nullptr, (const uint8_t*)b, (const uint8_t*)sb, m, n, padded(k), c, ldc, 0, 0, 0, 0};
    if (few_values(m, k)) return few_of_values(FewArgs{g, lda, k}, a_dtype, c_dtype, (hipStream_t)stream, what);
    if (k == 0) return matmul(g, c_dtype, (hipStream_t)stream, what);  // nothing to quantise
    const Operand2 q(ws, m, k);
    const QuantArgs job{a, m, k, lda, q.codes, q.scales, nullptr, nullptr};
    if ((rc = quantize(&job, 1, a_dtype, (hipStream_t)stream, what)) != ZERO_OK) return rc;
    g.a = q.codes;
    g.sa = q.scales;
    return matmul(g, c_dtype, (hipStream_t)stream, what);
}

size_t zero_mx4_operand_bytes(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 || rows > kMaxSide || cols > kMaxSide ? 0 : quantized_bytes(rows, cols);
}

size_t zero_mx4_linear_workspace_bytes(int64_t tokens, int64_t n, int64_t k) {
    return zero_mx4_operand_bytes(tokens, k) + zero_mx4_operand_bytes(n, k);
}

int zero_mx4_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t dtype, int64_t tokens, int64_t n,
                    int64_t k, void* y, int64_t ldy, void* x_t, void* w_t, void* ws, size_t ws_bytes, void* stream) {
    const char* what = "zero_mx4_linear";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_sides(tokens, n, what)) != ZERO_OK || (rc = check_sides(k, k, what)) != ZERO_OK) return rc;
    if (tokens == 0 || n == 0 || k == 0) return fail(ZERO_ERANGE, "%s: an empty product", what);
    if (x == nullptr || w == nullptr || y == nullptr) return fail(ZERO_EINVAL, "%s: null matrix", what);
    if (!aligned(x, elem_bytes(dtype)) || !aligned(w, elem_bytes(dtype)) || !aligned(y, elem_bytes(dtype)))
        return fail(ZERO_EALIGN, "%s: matrices not aligned to their elements", what);
    if (ldx < k || ldw < k || ldy < n) return fail(ZERO_ERANGE, "%s: row stride below the row", what);
    if ((rc = check_operands(x_t, w_t, ws, ws_bytes, zero_mx4_linear_workspace_bytes(tokens, n, k), what)) != ZERO_OK)
        return rc;
    const hipStream_t s = (hipStream_t)stream;
    const Operand2 xr(ws, tokens, k), wr((char*)ws + quantized_bytes(tokens, k), n, k);
    const Operand2 xt(x_t, k, tokens), wt(w_t, k, n);
    const QuantArgs jobs[2] = {{x, tokens, k, ldx, xr.codes, xr.scales, xt.codes, xt.scales},
                               {w, n, k, ldw, wr.codes, wr.scales, wt.codes, wt.scales}};
    if ((x_t == nullptr) == (w_t == nullptr))
        rc = quantize(jobs, 2, dtype, s, what);
    else if ((rc = quantize(jobs, 1, dtype, s, what)) == ZERO_OK)
        rc = quantize(jobs + 1, 1, dtype, s, what);
    if (rc != ZERO_OK) return rc;
    return matmul(MatmulArgs{xr.codes, xr.scales, wr.codes, wr.scales, tokens, n, padded(k), y, ldy, 0, 0, 0, 0}, dtype, s,
                  what);
}

size_t zero_mx4_linear_grad_workspace_bytes(int64_t tokens, int64_t n) {
    return zero_mx4_operand_bytes(tokens, n) + zero_mx4_operand_bytes(n, tokens);
}

int zero_mx4_linear_grad(const void* dy, int64_t lddy, int32_t dtype, int64_t tokens, int64_t n, int64_t k,
                         const void* x_t, const void* w_t, void* dx, int64_t lddx, void* dw, int64_t lddw, void* ws,
                         size_t ws_bytes, void* stream) {
    const char* what = "zero_mx4_linear_grad";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_sides(tokens, n, what)) != ZERO_OK || (rc = check_sides(k, k, what)) != ZERO_OK) return rc;
    if (tokens == 0 || n == 0 || k == 0) return fail(ZERO_ERANGE, "%s: an empty product", what);
    if (dx == nullptr && dw == nullptr) return ok();
    if (dy == nullptr || (dx != nullptr && w_t == nullptr) || (dw != nullptr && x_t == nullptr))
        return fail(ZERO_EINVAL, "%s: null matrix or operand", what);
    if (!aligned(dy, elem_bytes(dtype)) || !aligned(dx, elem_bytes(dtype)) || !aligned(dw, elem_bytes(dtype)))
        return fail(ZERO_EALIGN, "%s: matrices not aligned to their elements", what);
    if (lddy < n || (dx != nullptr && lddx < k) || (dw != nullptr && lddw < k))
        return fail(ZERO_ERANGE, "%s: row stride below the row", what);
    if ((rc = check_operands(x_t, w_t, ws, ws_bytes, zero_mx4_linear_grad_workspace_bytes(tokens, n), what)) != ZERO_OK)
        return rc;
    // dx is written before dw's product reads x_t
    if (dw != nullptr && overlap(values_at(dx, dtype, tokens, k, lddx), Place(x_t, (int64_t)quantized_bytes(k, tokens))))
        return fail(ZERO_EINVAL, "%s: dx overlaps x_t", what);
    const hipStream_t s = (hipStream_t)stream;
    const Operand2 r(ws, tokens, n), c((char*)ws + quantized_bytes(tokens, n), n, tokens);
    const Operand2 xt(const_cast<void*>(x_t), k, tokens), wt(const_cast<void*>(w_t), k, n);
    QuantArgs job{dy, tokens, n, lddy, r.codes, r.scales, c.codes, c.scales};
    if (dx == nullptr) job.codes = job.scales = nullptr;
    if (dw == nullptr) job.codes_t = job.scales_t = nullptr;
    if ((rc = quantize(&job, 1, dtype, s, what)) != ZERO_OK) return rc;
    if (dx != nullptr &&
        (rc = matmul(MatmulArgs{r.codes, r.scales, wt.codes, wt.scales, tokens, k, padded(n), dx, lddx, 0, 0, 0, 0}, dtype,
                     s, what)) != ZERO_OK)
        return rc;
    if (dw != nullptr)
        return matmul(MatmulArgs{c.codes, c.scales, xt.codes, xt.scales, n, k, padded(tokens), dw, lddw, 0, 0, 0, 0}, dtype,
                      s, what);
    return ok();
}

}  // extern "C"
