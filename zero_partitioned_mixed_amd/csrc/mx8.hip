// MXFP8 rows (E4M3 codes under E8M0 block scales) as the left operand of products with MXFP4
// operands: quantisation, the values back, and the product on the scaled matrix instructions,
// which take the two formats together at the rate of 8-bit operands.
//
// Rows are [rows][P] codes and [rows][P / 32] scales, P = cols rounded up to 128, the padding zero.
#include "mx_common.h"

namespace {

// ---------------------------------------------------------------- quantisation and values
struct Quant8Args {
    const void* src;
    int64_t rows, cols, ld;
    uint8_t *codes, *scales;
};

// Eight elements a lane, four lanes a block.  Bound by memory: the values of 4000 x 8192 back in bf16, 17 us for 99 MB.
template <int DT>
__device__ __forceinline__ void quantize8(const Eight<DT>& e, uint8_t* codes, uint8_t* scale) {
    float x[8];
    e.values(x);
    const uint32_t s = scale_byte8(block_top8(x));
    *(u32x2*)codes = codes8_e4m3(x, s);
    if ((threadIdx.x & 3) == 0) *scale = (uint8_t)s;
}

constexpr int kValueRows8 = 64;  // rows of a workgroup, 128 columns wide
template <int DT>
__global__ void __launch_bounds__(kThreads) mx8_quantize_kernel(Quant8Args a) {
    typedef typename Elem<DT>::type T;
    const int64_t p = padded(a.cols);
    const uint32_t across = (uint32_t)(p / kMxPad);
    const int64_t r0 = (int64_t)(blockIdx.x / across) * kValueRows8 + threadIdx.x / 16;
    const int64_t c = (int64_t)(blockIdx.x % across) * kMxPad + threadIdx.x % 16 * 8;
    constexpr int kEach = kValueRows8 / 16;
    Eight<DT> e[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (r0 + 16 * i < a.rows) e[i].fetch((const T*)a.src + (r0 + 16 * i) * a.ld, c, a.cols);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < a.rows) quantize8<DT>(e[i], a.codes + r * p + c, a.scales + r * (p / kMxBlock) + c / kMxBlock);
    }
}

struct Dequant8Args {
    const uint8_t *codes, *scales;
    int64_t rows, cols, ld;
    void* dst;
};

// Four codes times 2^(s - 127), the scaling with one rounding for results below the normal numbers.
__device__ __forceinline__ void values4_e4m3(uint32_t q, uint32_t s, float* x) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 v[2] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)q, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)q, true)};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = s == 255 ? __builtin_nanf("") : ldexpf(v[i / 2][i % 2], (int)s - 127);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) mx8_values_kernel(Dequant8Args a) {
    typedef typename Elem<DT>::type T;
    const int64_t p = padded(a.cols);
    const uint32_t across = (uint32_t)(p / kMxPad);
    const int64_t r0 = (int64_t)(blockIdx.x / across) * kValueRows8 + threadIdx.x / 16;
    const int64_t c = (int64_t)(blockIdx.x % across) * kMxPad + threadIdx.x % 16 * 8;
    if (c >= a.cols) return;
    constexpr int kEach = kValueRows8 / 16;
    u32x2 q[kEach];
    uint32_t s[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t r = r0 + 16 * i < a.rows ? r0 + 16 * i : a.rows - 1;
        q[i] = *(const u32x2*)(a.codes + r * p + c);
        s[i] = a.scales[r * (p / kMxBlock) + c / kMxBlock];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (r0 + 16 * i >= a.rows) return;
        float x[8];
        values4_e4m3(q[i][0], s[i], x);
        values4_e4m3(q[i][1], s[i], x + 4);
        put8<DT>((T*)a.dst + (r0 + 16 * i) * a.ld, c, a.cols, x);
    }
}

// ---------------------------------------------------------------- the product
struct Matmul8Args {
    const uint8_t *a, *sa, *b, *sb;
    int64_t m, n, p;  // p: padded k
    void* c;
    int64_t ldc;
    int tiles_m, tiles_n;
    int accumulate;
    int vector;  // rows of c aligned to four elements
};

// Of a 32x32x64 instruction, lane group h (lane / 32) holds of the 4-bit operand's row the block of
// 32 that is its half of k, but of the 8-bit operand's row sixteen elements of either block: bytes
// 16 h .. 16 h + 15 of the first in registers 0..3, of the second in 4..7 (measured).  Group h's
// scales are those of block h for both.
//
// The instruction adds eight neighbouring products on a grid of 2^(E - 13), E the largest sum of
// their exponents, and cuts what lies below it (measured; a subnormal code counts with the smallest
// normal exponent).  Sums have to be fp32 for results of 16 bits too: cut like that they are off by 2e-5 of
// a result's norm for activations, and by more where few columns are large.  So A is split by its codes'
// highest exponent bit: products of codes from 2 on are multiples of 2^(E - 13), and those of the codes below
// too, so that nothing is cut, at twice the instructions (8192 x 8192 x 8192 418 us with one, 694 with two).
template <class K>
__device__ __forceinline__ f32x16 mma8(const i32x8& a, const i32x4& b, f32x16 c, int sa, int sb, K) {
    const i32x8 v = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, v, c, 0, 4, K::value, sa, K::value, sb);
}
__device__ __forceinline__ i32x8 joined(const i32x4& a0, const i32x4& a1) {
    return __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
}
// 255 in the bytes of codes from 2 on: the permutation takes the signs of 16-bit halves, to which the bits are moved.
__device__ __forceinline__ uint32_t high_codes(int u) {
    return __builtin_amdgcn_perm((uint32_t)u << 1, (uint32_t)u << 9, 0x0B090A08u);
}
template <class K>
__device__ __forceinline__ f32x16 mma8_split(const i32x4& a0, const i32x4& a1, const i32x4& b, f32x16 c, int sa, int sb, K k) {
    const i32x8 u = joined(a0, a1);
    i32x8 low, high;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        high[i] = u[i] & (int)high_codes(u[i]);
        low[i] = u[i] ^ high[i];
    }
    return mma8(high, b, mma8(low, b, c, sa, sb, k), sa, sb, k);
}

template <int K>
using Step = std::integral_constant<int, K>;

// A tile of TM x TN outputs by waves of WM x WN outputs each.  A slab is 128 elements of every
// row: 128 bytes of A's and 64 of B's, and a dword of block scales; STAGES slabs in LDS,
// copied by direct loads, STAGES - 1 on their way while one is used.  A dword of scales costs as much
// of the memory pipeline as a line, so where their rows are multiples of 16 bytes (WIDE) those of four
// slabs come together.  Piece q (16 bytes) of A's
// row r sits in slot q ^ (r / 2 mod 8), of B's in q ^ (r / 4 mod 4): 16 lanes then read all banks.
template <int TM_, int TN_, int WM_, int WN_, int STAGES_>
struct Mixed {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr int WAVES = (TM / WM) * (TN / WN), THREADS = WAVES * 64;
    static constexpr int MT = WM / 32, NT = WN / 32;
    static constexpr int LA = TM / 8 / WAVES, LB = TN / 16 / WAVES;         // direct loads per wave and slab
    static constexpr int SETS = (TM + TN) / 64, LS = (SETS + WAVES - 1) / WAVES;  // and of scales
    static constexpr int B_AT = TM * 128, STAGE = B_AT + TN * 64;
    // behind the stages the scales: two groups of four slabs, or STAGES slabs
    static constexpr int S_AT = STAGES * STAGE, SCALES = 2 * (TM + TN) * 16;
    static_assert(LA * 8 * WAVES == TM && LB * 16 * WAVES == TN && LA >= 1 && LB >= 1, "whole loads per wave");
    static_assert(S_AT + SCALES <= 160 * 1024 && STAGES * 4 <= 2 * 16, "LDS");
};

template <class S, int DT, bool WIDE>
__global__ void __launch_bounds__(S::THREADS) mx8_matmul_kernel(Matmul8Args g) {
    __shared__ __attribute__((aligned(16))) char lds[S::S_AT + S::SCALES];
    int ti, tj;
    band_tile(xcd_tile(blockIdx.x, gridDim.x), g.tiles_m, g.tiles_n, ti, tj);
    const int64_t i0 = (int64_t)ti * S::TM, j0 = (int64_t)tj * S::TN;
    const int64_t left_m = g.m - i0, left_n = g.n - j0;
    const int rows_a = (int)(left_m < S::TM ? left_m : S::TM), rows_b = (int)(left_n < S::TN ? left_n : S::TN);
    const Lane L;
    const uint32_t p = (uint32_t)g.p, ps = p / kMxBlock;
    const char *const a = (const char*)g.a + i0 * g.p, *const b = (const char*)g.b + j0 * (g.p / 2);
    const char *const sa = (const char*)g.sa + i0 * ps, *const sb = (const char*)g.sb + j0 * ps;
    const int slabs = (int)(g.p / 128);

    // Where this wave's direct loads read: rows past the operand's end repeat its last one.
    uint32_t at_a[S::LA], at_b[S::LB], at_s[S::LS];
    const char* from_s[S::LS];
#pragma unroll
    for (int i = 0; i < S::LA; ++i) {
        const int r = (L.wave * S::LA + i) * 8 + (L.lane >> 3);
        at_a[i] = (uint32_t)(r < rows_a ? r : rows_a - 1) * p + ((L.lane & 7) ^ ((r >> 1) & 7)) * 16;
    }
#pragma unroll
    for (int i = 0; i < S::LB; ++i) {
        const int r = (L.wave * S::LB + i) * 16 + (L.lane >> 2);
        at_b[i] = (uint32_t)(r < rows_b ? r : rows_b - 1) * (p / 2) + ((L.lane & 3) ^ ((r >> 2) & 3)) * 16;
    }
    auto set_of = [&](int i) { return (L.wave * S::LS + i) % S::SETS; };  // fewer sets than waves: some are loaded twice
#pragma unroll
    for (int i = 0; i < S::LS; ++i) {
        const int r = set_of(i) * 64;
        const bool of_a = r < S::TM;
        const int row = (of_a ? r : r - S::TM) + L.lane, rows = of_a ? rows_a : rows_b;
        from_s[i] = of_a ? sa : sb;
        at_s[i] = (uint32_t)(row < rows ? row : rows - 1) * ps;
    }
    // half q of a slab's loads (q = 2: all)
    auto stage = [&](int slab, char* buf, int q) {
        const int64_t k = (int64_t)slab * 128;
        if (q != 1) {
#pragma unroll
            for (int i = 0; i < S::LA; ++i) load_to_lds16(a + k + at_a[i], buf + (L.wave * S::LA + i) * 1024);
        }
        if (q != 0) {
#pragma unroll
            for (int i = 0; i < S::LB; ++i)
                load_to_lds16(b + k / 2 + at_b[i], buf + S::B_AT + (L.wave * S::LB + i) * 1024);
            if constexpr (WIDE) {
                if (slab % 4 == 0) {
                    char* const to = lds + S::S_AT + (slab / 4 & 1) * ((S::TM + S::TN) * 16);
#pragma unroll
                    for (int i = 0; i < S::LS; ++i) load_to_lds16(from_s[i] + k / 32 + at_s[i], to + set_of(i) * 1024);
                }
            } else {
                char* const to = lds + S::S_AT + slab % S::STAGES * ((S::TM + S::TN) * 4);
#pragma unroll
                for (int i = 0; i < S::LS; ++i) load_to_lds4(from_s[i] + k / 32 + at_s[i], to + set_of(i) * 256);
            }
        }
    };
    auto scale = [&](int slab, int row) {  // of a row of A's, or of B's behind them
        const uint32_t* const from = (const uint32_t*)(lds + S::S_AT);
        const uint32_t v = WIDE ? from[(slab / 4 & 1) * ((S::TM + S::TN) * 4) + row * 4 + slab % 4]
                                : from[slab % S::STAGES * (S::TM + S::TN) + row];
        return (int)(v >> (8 * L.h));
    };

    f32x16 acc[S::MT][S::NT];
#pragma unroll
    for (int i = 0; i < S::MT; ++i)
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int wm = L.wave / (S::TN / S::WN), wn = L.wave % (S::TN / S::WN);
    const int ra = (wm * S::WM + L.c) * 128, rb = S::B_AT + (wn * S::WN + L.c) * 64;
    const int turn_a = (L.c >> 1) & 7, turn_b = (L.c >> 2) & 3;
    struct Frags {
        i32x4 a[S::MT][2], b[S::NT];
    };
    auto fragments = [&](const char* buf, int s, Frags& f) {
        const int a0 = ((4 * s + L.h) ^ turn_a) << 4, a1 = ((4 * s + 2 + L.h) ^ turn_a) << 4, b0 = ((2 * s + L.h) ^ turn_b) << 4;
#pragma unroll
        for (int i = 0; i < S::MT; ++i) {
            f.a[i][0] = *(const i32x4*)(buf + ra + i * 32 * 128 + a0);
            f.a[i][1] = *(const i32x4*)(buf + ra + i * 32 * 128 + a1);
        }
#pragma unroll
        for (int j = 0; j < S::NT; ++j) f.b[j] = *(const i32x4*)(buf + rb + j * 32 * 64 + b0);
    };
    int va[S::MT], vb[S::NT];
    auto multiply = [&](const Frags& f, auto kk) {
#pragma unroll
        for (int i = 0; i < S::MT; ++i)
#pragma unroll
            for (int j = 0; j < S::NT; ++j) acc[i][j] = mma8_split(f.a[i][0], f.a[i][1], f.b[j], acc[i][j], va[i], vb[j], kk);
    };

#pragma unroll
    for (int t = 0; t < S::STAGES - 1; ++t)
        if (t < slabs) stage(t, lds + t * S::STAGE, 2);
    char *buf = lds, *fill = lds + (S::STAGES - 1) * S::STAGE;
    char* const end = lds + S::STAGES * S::STAGE;
    auto after = [&](char* x) { return x + S::STAGE == end ? lds : x + S::STAGE; };
    for (int t = 0; t < slabs; ++t) {
        // this slab has landed in every wave's part, and the buffer used before it is free
        // (of the slabs after it those with scales have more loads: counted without, a few of them are waited for)
        constexpr int kLoads = S::LA + S::LB + (WIDE ? 0 : S::LS);
        if (t + S::STAGES - 2 < slabs)
            wait_and_meet<(S::STAGES - 2) * kLoads>();
        else
            wait_and_meet<0>();
        const int next = t + S::STAGES - 1;
        const bool more = next < slabs;
#pragma unroll
        for (int i = 0; i < S::MT; ++i) va[i] = scale(t, wm * S::WM + 32 * i + L.c);
#pragma unroll
        for (int j = 0; j < S::NT; ++j) vb[j] = scale(t, S::TM + wn * S::WN + 32 * j + L.c);
        Frags f[2];
        fragments(buf, 0, f[0]);
        if (more) stage(next, fill, 0);
        fragments(buf, 1, f[1]);
        multiply(f[0], Step<0>());
        if (more) stage(next, fill, 1);
        multiply(f[1], Step<2>());
        buf = after(buf);
        fill = after(fill);
    }

    // Four columns of a row per lane and store.
    typedef typename Elem<DT>::type T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    const int iw = wm * S::WM + 4 * L.h + (L.c & 3), jw = wn * S::WN + (L.c & ~3);
    T* const out = (T*)g.c + i0 * g.ldc + j0;
    const bool whole = g.vector && rows_a == S::TM && rows_b == S::TN;
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
                T4 w;
                if constexpr (DT == ZERO_F32) {
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = acc[ii][jj][4 * q + r];
                    quad_turn(v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (g.accumulate && i < rows_a && j + e < rows_b) v[e] += at[e];
                        w[e] = v[e];
                    }
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

// Few rows (m <= 32, as single tokens bring): bound by reading B once (one token 11008 x 4096: 7.5 us,
// where reading B takes 4.7; its waves wait for 53% of their cycles).  A workgroup takes 32 of B's
// rows, its eight waves an eighth of k each: a wave brings slabs of 256 elements of them to its own
// part of LDS in whole lines, waits for nobody, and the waves' sums meet in LDS.
// VALUES (m times the padded k up to kFew8): A comes as values, and every workgroup quantises all
// of it to LDS first, which saves a launch.
// HALVES (m <= 16): the low codes of row i are the instruction's row 2i and the high ones its row 2i + 1, so
// that one instruction is enough.
constexpr int kFewWaves = 8;
constexpr int kFew8 = 8192;  // two workgroups on a CU: one token 11008 x 4096 6.2 us, 7.5 with one, with codes unsplit
constexpr int kFewSlabs = 2;  // slabs of a wave on their way at once

struct Few8Args {
    Matmul8Args g;
    const void* values;
    int64_t lda, k;
};

template <int DTA, int DT, bool VALUES, bool HALVES>
__global__ void __launch_bounds__(kFewWaves * 64) mx8_few_kernel(Few8Args f) {
    const Matmul8Args& g = f.g;
    __shared__ __attribute__((aligned(16))) uint8_t codes[VALUES ? kFew8 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t scales[VALUES ? kFew8 / kMxBlock : 16];
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
            e.fetch((const T*)f.values + r * f.lda, c, f.k);
        };
        auto put = [&](int t, const Eight<DTA>& e) {  // whole groups of four lanes
            const uint32_t r = (uint32_t)t / (p / 8), c = ((uint32_t)t - r * (p / 8)) * 8;
            quantize8<DTA>(e, codes + r * p + c, scales + r * scale_row + c / kMxBlock);
        };
        // loads return in order: A's go out before B's, so that A is ready while B is on its way
        constexpr int kFirst = kFew8 / (8 * kFewWaves * 64);  // pieces a lane
        static_assert(kFirst * 8 * kFewWaves * 64 == kFew8, "all of A");
        const int tid = threadIdx.x;
        Eight<DTA> e[kFirst];
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
            if (tid + i * kFewWaves * 64 < pieces) read(tid + i * kFewWaves * 64, e[i]);
        if (any) fetch(L.wave);
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
            if (tid + i * kFewWaves * 64 < pieces) put(tid + i * kFewWaves * 64, e[i]);
        __syncthreads();
    } else {
        if (any) fetch(L.wave);
    }
    const int of = HALVES ? L.c >> 1 : L.c;
    const uint32_t other = HALVES && (L.c & 1) == 0 ? ~0u : 0u;  // even lanes take the low codes
    const uint32_t row = (uint32_t)(of < g.m ? of : g.m - 1);
    const uint8_t* const a = (VALUES ? codes : g.a) + (int64_t)row * p + 16 * L.h;
    const uint8_t* const sa = (VALUES ? scales : g.sa) + (int64_t)row * scale_row;
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    // blocks q and q + apart (of the slab's) meet in a step
    auto step = [&](const uint8_t* at, int apart, const i32x4& bw, uint32_t as, uint32_t bs_, auto kk) {
        const int q = decltype(kk)::value;
        const i32x4 a0 = *(const i32x4*)(at + q * 32), a1 = *(const i32x4*)(at + (q + apart) * 32);
        if constexpr (HALVES) {
            i32x8 part = joined(a0, a1);
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i] &= (int)(high_codes(part[i]) ^ other);
            acc = mma8(part, bw, acc, (int)as, (int)bs_, kk);
        } else {
            acc = mma8_split(a0, a1, bw, acc, (int)as, (int)bs_, kk);
        }
    };

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
            const uint32_t as = *(const uint32_t*)(sa + s * 8 + 4 * L.h);
            const uint8_t* const at = a + (int64_t)s * 256;
            step(at, 4, bw[0], as, bs[u], Step<0>());
            step(at, 4, bw[1], as, bs[u], Step<1>());
            step(at, 4, bw[2], as, bs[u], Step<2>());
            step(at, 4, bw[3], as, bs[u], Step<3>());
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next slabs come
    }
    if (p % 256 != 0 && L.wave == 0) {  // half a slab: group h takes blocks 2h and 2h + 1 of four
        const int64_t at = (int64_t)slabs * 128 - 32 * L.h, sat = (int64_t)slabs * 8 - 4 * L.h;
        const uint32_t bsh = *(const uint32_t*)(sb + sat) >> (16 * L.h);
        const i32x4 b0 = *(const i32x4*)(b + at), b1 = *(const i32x4*)(b + at + 16);
        const uint32_t as = *(const uint32_t*)(sa + slabs * 8) >> (16 * L.h);
        step(a + (int64_t)slabs * 256, 2, b0, as, bsh, Step<0>());
        step(a + (int64_t)slabs * 256, 2, b1, as, bsh, Step<1>());
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
        constexpr int kRows = HALVES ? 2 : 1;  // of the sums
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
            for (int u = 0; u < kRows; ++u) v += sums[w][kRows * i + u][c];
        T* out = (T*)g.c + i * g.ldc + col;
        if constexpr (DT == ZERO_F32) {
            if (g.accumulate) v += *out;
        }
        *out = from_float<DT>(v);
    }
}

// ---------------------------------------------------------------- host side
template <class F>
int with_dtype(int32_t dt, F f) {
    switch (dt) {
        case ZERO_F16: return f(Step<ZERO_F16>());
        case ZERO_BF16: return f(Step<ZERO_BF16>());
        default: return f(Step<ZERO_F32>());
    }
}

int quantize(const Quant8Args& a, int32_t dtype, hipStream_t s, const char* what) {
    const int64_t wgs = ceil_div(a.rows, kValueRows8) * (padded(a.cols) / kMxPad);
    if (wgs > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    return with_dtype(dtype, [&](auto t) {
        return launch(mx8_quantize_kernel<decltype(t)::value>, dim3((unsigned)wgs), kThreads, s, a, what);
    });
}

template <class S>
int matmul_with(Matmul8Args g, int32_t c_dtype, hipStream_t s, const char* what) {
    const int64_t tm = ceil_div(g.m, S::TM), tn = ceil_div(g.n, S::TN);
    if (tm * tn > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many tiles for one launch", what);
    g.tiles_m = (int)tm;
    g.tiles_n = (int)tn;
    return with_dtype(c_dtype, [&](auto t) {
        const dim3 grid((unsigned)(tm * tn));
        if (g.p % 512 == 0) return launch(mx8_matmul_kernel<S, decltype(t)::value, true>, grid, S::THREADS, s, g, what);
        return launch(mx8_matmul_kernel<S, decltype(t)::value, false>, grid, S::THREADS, s, g, what);
    });
}

// 8192 x 8192 x 8192 690 us (1600 TFLOP/s, 3200 of instructions; from registers they reach 4212), 4096 x 11008 x 4096 262.
// Chosen with one instruction a step, 8192 x 8192 x 8192, us: eight waves with 64 x 128 each 474, four with 128 x 128
// 490; with the scales of four slabs at once 446.  Without the loads to LDS 404, without the matrix instructions 362:
// both keep the waves waiting for their turn to issue, and together they lower the clock.  Fragments read ahead of the
// barrier, loads spread between the matrix instructions, another first slab for each row of tiles: no faster.
typedef Mixed<256, 256, 64, 128, 3> Mixed256;
typedef Mixed<128, 128, 64, 64, 3> Mixed128;  // up to two workgroups on a CU
typedef Mixed<64, 64, 32, 32, 4> Mixed64;     // up to three

// The shape that a product takes: microseconds a slab as measured (256 CUs, k = 4096), a part of it however few the
// tiles and a part for each tile that the busiest CU gets.  us by tiles of 64, 128 and 256: 64 x 4096 15, 33, 83; 512 x
// 4096 23, 33, 84; 1024 x 4096 41, 36, 87; 300 x 11008 41, 55, 89; 1024 x 11008 103, 83, 93; 2048 x 11008 201, 152, 175;
// 4096 x 4096 148, 105, 93; 4096 x 11008 391, 278, 262.
int pick_mixed(int64_t t256, int64_t t128, int64_t t64) {
    const double c256 = 0.10 + 2.70 * (double)ceil_div(t256, 256);
    const double c128 = 0.20 + 0.79 * (double)ceil_div(t128, 256);
    const double c64 = 0.20 + 0.28 * (double)ceil_div(t64, 256);
    return c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
}

// Values of A quantised in the product's own kernel.
bool few_values(int64_t m, int64_t k) { return m <= 32 && m * padded(k) <= kFew8; }

template <class F>
int with_halves(int64_t m, F f) {
    return m <= 16 ? f(std::true_type()) : f(std::false_type());
}

int matmul(Matmul8Args g, int32_t c_dtype, hipStream_t s, const char* what) {
    g.vector = aligned(g.c, 4 * elem_bytes(c_dtype)) && g.ldc % 4 == 0;
    // Few rows against tiles, us: 4096 x 4096, 8 rows 5.8 and 15.2, 32 rows 7.6 and 15.3; 11008 x 4096, 8 rows 8.9 and
    // 16.2, 24 rows 12.8 and 15.5, 32 rows 15.7 and 15.5.
    if (g.m <= 32) {
        const Few8Args f{g, nullptr, 0, 0};
        return with_halves(g.m, [&](auto h) {
            return with_dtype(c_dtype, [&](auto t) {
                return launch(mx8_few_kernel<ZERO_F32, decltype(t)::value, false, decltype(h)::value>,
                              dim3((unsigned)ceil_div(g.n, 32)), kFewWaves * 64, s, f, what);
            });
        });
    }
    auto tiles = [&](int64_t t) { return ceil_div(g.m, t) * ceil_div(g.n, t); };
    switch (pick_mixed(tiles(256), tiles(128), tiles(64))) {
        case 256: return matmul_with<Mixed256>(g, c_dtype, s, what);
        case 128: return matmul_with<Mixed128>(g, c_dtype, s, what);
        default: return matmul_with<Mixed64>(g, c_dtype, s, what);
    }
}

int few_of_values(const Few8Args& f, int32_t a_dtype, int32_t c_dtype, hipStream_t s, const char* what) {
    return with_halves(f.g.m, [&](auto h) {
        return with_dtype(a_dtype, [&](auto ta) {
            return with_dtype(c_dtype, [&](auto tc) {
                return launch(mx8_few_kernel<decltype(ta)::value, decltype(tc)::value, true, decltype(h)::value>,
                              dim3((unsigned)ceil_div(f.g.n, 32)), kFewWaves * 64, s, f, what);
            });
        });
    });
}

// The checks shared by the products; 1: nothing to do.
int check_matmul(const void* b, const void* sb, int64_t m, int64_t n, int64_t k, const void* c, int32_t c_dtype,
                 int64_t ldc, int32_t accumulate, const char* what) {
    if (!valid_dtype(c_dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if (accumulate != 0 && (accumulate != 1 || c_dtype != ZERO_F32))
        return fail(ZERO_EINVAL, "%s: accumulate is 0, or 1 with an fp32 result", what);
    int rc;
    if ((rc = check_sides(m, n, what)) != ZERO_OK || (rc = check_sides(k, k, what)) != ZERO_OK) return rc;
    if (m == 0 || n == 0) return 1;
    if (c == nullptr || (k > 0 && (b == nullptr || sb == nullptr)))
        return fail(ZERO_EINVAL, "%s: null operand or result", what);
    if (!aligned(b, 16) || !aligned(sb, 16)) return fail(ZERO_EALIGN, "%s: operands not 16-byte aligned", what);
    if (!aligned(c, elem_bytes(c_dtype))) return fail(ZERO_EALIGN, "%s: result not aligned to its elements", what);
    if (ldc < n) return fail(ZERO_ERANGE, "%s: row stride below n", what);
    const Place to = values_at(c, c_dtype, m, n, ldc);
    if (overlap(to, codes_at(b, n, k)) || overlap(to, scales_at(sb, n, k)))
        return fail(ZERO_EINVAL, "%s: the result overlaps an operand", what);
    return ZERO_OK;
}

}  // namespace

extern "C" {

size_t zero_mx8_code_bytes(int64_t rows, int64_t cols) { return rows <= 0 || cols <= 0 ? 0 : (size_t)(rows * padded(cols)); }

int zero_mx8_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void* codes, void* scales,
                      void* stream) {
    const char* what = "zero_mx8_quantize";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_sides(rows, cols, what)) != ZERO_OK) return rc;
    if (ld < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (rows == 0 || cols == 0) return ok();
    if (src == nullptr || codes == nullptr || scales == nullptr) return fail(ZERO_EINVAL, "%s: null buffer", what);
    if (!aligned(codes, 16) || !aligned(scales, 16)) return fail(ZERO_EALIGN, "%s: outputs not 16-byte aligned", what);
    if (!aligned(src, elem_bytes(dtype))) return fail(ZERO_EALIGN, "%s: source not aligned to its elements", what);
    const Place from = values_at(src, dtype, rows, cols, ld);
    if (overlap(from, codes8_at(codes, rows, cols)) || overlap(from, scales_at(scales, rows, cols)))
        return fail(ZERO_EINVAL, "%s: codes or scales overlap the values", what);
    if (overlap(codes8_at(codes, rows, cols), scales_at(scales, rows, cols)))
        return fail(ZERO_EINVAL, "%s: codes and scales overlap", what);
    return quantize(Quant8Args{src, rows, cols, ld, (uint8_t*)codes, (uint8_t*)scales}, dtype, (hipStream_t)stream, what);
}

int zero_mx8_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, void* dst, int32_t dtype,
                        int64_t ld, void* stream) {
    const char* what = "zero_mx8_dequantize";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_sides(rows, cols, what)) != ZERO_OK) return rc;
    if (ld < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (rows == 0 || cols == 0) return ok();
    if (codes == nullptr || scales == nullptr || dst == nullptr) return fail(ZERO_EINVAL, "%s: null buffer", what);
    if (!aligned(codes, 16) || !aligned(scales, 16)) return fail(ZERO_EALIGN, "%s: operand not 16-byte aligned", what);
    if (!aligned(dst, elem_bytes(dtype))) return fail(ZERO_EALIGN, "%s: result not aligned to its elements", what);
    const Place to = values_at(dst, dtype, rows, cols, ld);
    if (overlap(to, codes8_at(codes, rows, cols)) || overlap(to, scales_at(scales, rows, cols)))
        return fail(ZERO_EINVAL, "%s: the result overlaps the operand", what);
    const Dequant8Args a{(const uint8_t*)codes, (const uint8_t*)scales, rows, cols, ld, dst};
    const int64_t wgs = ceil_div(rows, kValueRows8) * (padded(cols) / kMxPad);
    if (wgs > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    return with_dtype(dtype, [&](auto t) {
        return launch(mx8_values_kernel<decltype(t)::value>, dim3((unsigned)wgs), kThreads, (hipStream_t)stream, a, what);
    });
}

int zero_mx8_matmul(const void* a, const void* sa, const void* b, const void* sb, int64_t m, int64_t n, int64_t k, void* c,
                    int32_t c_dtype, int64_t ldc, int32_t accumulate, void* stream) {
    const char* what = "zero_mx8_matmul";
    const int rc = check_matmul(b, sb, m, n, k, c, c_dtype, ldc, accumulate, what);
    if (rc == 1) return ok();
    if (rc != ZERO_OK) return rc;
    if (k > 0 && (a == nullptr || sa == nullptr)) return fail(ZERO_EINVAL, "%s: null operand", what);
    if (!aligned(a, 16) || !aligned(sa, 16)) return fail(ZERO_EALIGN, "%s: operands not 16-byte aligned", what);
    const Place to = values_at(c, c_dtype, m, n, ldc);
    if (overlap(to, codes8_at(a, m, k)) || overlap(to, scales_at(sa, m, k)))
        return fail(ZERO_EINVAL, "%s: the result overlaps an operand", what);
    const Matmul8Args g{(const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b, (const uint8_t*)sb,
                        m, n, padded(k), c, ldc, 0, 0, accumulate, 0};
    return matmul(g, c_dtype, (hipStream_t)stream, what);
}

size_t zero_mx8_matmul_rows_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m <= 0 || n <= 0 || k <= 0 || m > kMaxSide || n > kMaxSide || k > kMaxSide || few_values(m, k)) return 0;
    return (size_t)(round_up(m * padded(k), 256) + round_up(m * (padded(k) / kMxBlock), 256));
}

int zero_mx8_matmul_rows(const void* a, int32_t a_dtype, int64_t lda, const void* b, const void* sb, int64_t m, int64_t n,
                         int64_t k, void* c, int32_t c_dtype, int64_t ldc, int32_t accumulate, void* ws, size_t ws_bytes,
                         void* stream) {
    const char* what = "zero_mx8_matmul_rows";
    if (!valid_dtype(a_dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    int rc = check_matmul(b, sb, m, n, k, c, c_dtype, ldc, accumulate, what);
    if (rc == 1) return ok();
    if (rc != ZERO_OK) return rc;
    if (k > 0 && a == nullptr) return fail(ZERO_EINVAL, "%s: null operand", what);
    if (!aligned(a, elem_bytes(a_dtype))) return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    if (lda < k) return fail(ZERO_ERANGE, "%s: row stride below k", what);
    const size_t need = zero_mx8_matmul_rows_workspace_bytes(m, n, k);
    if (need > 0) {
        if (ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
        if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
        if (ws_bytes < need) return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
    }
    const Place to = values_at(c, c_dtype, m, n, ldc);
    if (overlap(to, values_at(a, a_dtype, m, k, lda))) return fail(ZERO_EINVAL, "%s: the result overlaps an operand", what);
    if (need > 0 && meets(Place(ws, (int64_t)need), {to, values_at(a, a_dtype, m, k, lda), codes_at(b, n, k), scales_at(sb, n, k)}))
        return fail(ZERO_EINVAL, "%s: the workspace overlaps the result or an operand", what);
    const hipStream_t s = (hipStream_t)stream;
    Matmul8Args g{nullptr, nullptr, (const uint8_t*)b, (const uint8_t*)sb, m, n, padded(k), c, ldc, 0, 0, accumulate, 0};
    if (few_values(m, k)) return few_of_values(Few8Args{g, a, lda, k}, a_dtype, c_dtype, s, what);
    if (k > 0) {
        uint8_t *const codes = (uint8_t*)ws, *const scales = codes + round_up(m * padded(k), 256);
        if ((rc = quantize(Quant8Args{a, m, k, lda, codes, scales}, a_dtype, s, what)) != ZERO_OK) return rc;
        g.a = codes;
        g.sa = scales;
    }
    return matmul(g, c_dtype, s, what);
}

}  // extern "C"
