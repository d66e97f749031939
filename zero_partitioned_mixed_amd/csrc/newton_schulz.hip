// Orthogonalised updates of whole matrices (Newton-Schulz), for gfx950.
//
// One step is three products on the smaller side m of an m x n matrix X:
//   S = X X^T,   M = a I + b S + c S^2,   X <- M X.
// Rounding.  The products take fp16 operands and sum in fp32 (the iteration
// in bf16 operands is off by 1e-2 to 3e-2, in plain fp16 by 1e-3 to 4e-3).  X itself
// stays in fp32 between steps, and the diagonals of S and M, which hold most of
// their weight, are kept in fp32 outside the fp16 operands:
//   S = D + E,  S^2 = E E + (d_i + d_j) e_ij + D^2,  X <- diag(M) X + (M - diag(M)) X.
// D is the rows' squared norms of the fp32 X, summed where X is made: from the rounded
// X, rows whose elements round alike came out up to 6e-3 off (an identity of 482).
// Only the off-diagonal parts and the product's copy of X are rounded.
//
// How far.  A result in fp16 shows what 11-bit operands leave (3e-4 to 1e-3 beside its own
// 2e-4), so there each of them has two parts, high and rest, of 22 bits together, and
// each product three products: nothing but the result's rounding is left.  A result in bf16
// rounds by 1.7e-3, and an update meets the weights times lr: their operands have one
// part, in 0.4 of the time (11008 x 4096: 3.8 against 9.6 ms, 1500 x 4099 0.42 against 0.99).
// In one part, against 64 bits: 2e-4 to 1e-3 for spectra from flat to 1/k, up to 1.5e-3
// for a quarter of the rank and 1.8e-3 for matrices of one or two values (55 sizes from
// 130 x 200 to 4096 x 4096).  In two parts: 1e-6, a quarter of the rank 5e-6.  In both
// forms sums over equal terms round alike: constant matrices are off by 5e-7 times the
// smaller side more (8192 x 8192: 4e-3), other matrices of rank one by 4e-5 to 3e-4.
//
// fp16 holds powers of two times the values: X * 2^8, E * 2^12, M * a power that
// the coefficients choose (coeffs_of); entries down to 1 / (65536 * 256)
// stay normal or lose less than X's own rounding.
//
// Memory.  X and its transpose are both kept row-major along k, so every
// product reads both operands the same way; S and M are symmetric and need one
// copy.  S and S^2 are computed for tiles on and above the diagonal and
// mirrored.
#include "matrix_common.h"

#include <cmath>

namespace {

constexpr float kXScale = 256.0f, kSScale = 4096.0f;

// Row i of an fp16 operand of the large matrices is stored times spread(i), a number in
// [1, 2) that differs from row to row, and a product's results are divided by their row's
// and column's.  Elements that are equal then round differently in different rows, so that
// the roundings average out as those of other matrices do: with plain powers of two,
// constant matrices came out up to 1.2e-2 off in one part (1393 x 21020; now at most 1.8e-3 at 55 sizes).
__device__ __forceinline__ float spread(int i) {
    return __builtin_bit_cast(float, 0x3F800000u | ((uint32_t)i * 0x9E3779B1u) >> 9);
}
// a b + c in fp16, one instruction.
__device__ __forceinline__ _Float16 half_fma(float a, float b, float c = 0.0f) { return (_Float16)__builtin_fmaf(a, b, c); }

struct Coeffs {
    float a, b, c, eps;
    float mscale;  // power of two of the fp16 M: (|a| + |b| S + |c| S^2) * mscale is below 2^15
};

// A stack in the workspace, on the wide side: m <= n, mp and np the row lengths
// (multiples of 64, the padding zero).
struct Work {
    int m, n, mp, np;
    // Row lengths of M and X^T (mp, or 2 mp where X^T has two parts), of X and of S (np and
    // mp, or twice that where all operands have two).  Of two parts the rests come first.
    int kp, nx, ms;
    int64_t stride;  // bytes from one matrix's block to the next
    char* base;
    int64_t x16, xt0, xt1, s16, m16, ds, dm, sums;  // byte offsets; X in fp32 at 0
    int64_t rows;  // parts of X's squared row norms: a run of mp floats for every group of columns
    int parts;                                      // partial sums of squares per matrix
    const int32_t* skip;                            // != NULL and set: leave everything as it is
    __device__ char* of(int b) const { return base + (int64_t)b * stride; }
    __device__ bool skipped() const { return skip != nullptr && *skip != 0; }
};

// ---------------------------------------------------------------- where a stack comes from and goes to
// The matrices of zero_orthogonalize.
template <int DTI, int DTO>
struct PlainIo {
    static constexpr bool kExact = DTO == ZERO_F16;  // a result of 11 bits: the operands have 22
    static constexpr bool kNarrow = true;            // narrow matrices come with this type too
    const typename Elem<DTI>::type* src;
    typename Elem<DTO>::type* dst;
    int64_t src_ld, src_stride, dst_ld, dst_stride;
    int rows, cols;

    __device__ float clip() const { return 1.0f; }
    // first reading of an element, and any later one
    __device__ float first(int b, int r, int64_t c, float) const { return again(b, r, c, 1.0f); }
    __device__ float again(int b, int r, int64_t c, float) const {
        return to_float<DTI>(src[b * src_stride + r * src_ld + c]);
    }
    __device__ bool contiguous() const { return src_ld == cols; }
    __device__ void first4(int b, int r, int64_t c, float, float* v) const {  // vectors at any alignment
        typename Elem<DTI>::type x[4];
        __builtin_memcpy(x, src + b * src_stride + r * src_ld + c, sizeof(x));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = to_float<DTI>(x[e]);
    }
    __device__ void put(int b, int r, int c, float o) const {
        dst[b * dst_stride + r * dst_ld + c] = from_float<DTO>(o);
    }
};

// The matrices of zero_muon_step: the momentum is updated at the first reading.
template <int DTO, bool EXACT>
struct MuonIo {
    static constexpr bool kExact = EXACT;
    static constexpr bool kNarrow = !EXACT;  // their operands have two parts anyway
    float* master;
    float* mom;
    const float* g;
    const zero_ctrl* ctrl;
    uint16_t* slot;
    int64_t stride;
    int rows, cols;
    float mu, one_mu, decay, step;  // decay = lr wd, step = lr s
    int nesterov;

    __device__ float clip() const { return ctrl != nullptr ? ctrl->clip : 1.0f; }
    __device__ float direction(float gi, float m) const { return nesterov ? one_mu * gi + mu * m : m; }
    __device__ float first(int b, int r, int64_t c, float clip) const {
        const int64_t i = b * stride + (int64_t)r * cols + c;
        const float gi = g[i] * clip, m = mu * mom[i] + one_mu * gi;
        mom[i] = m;
        return direction(gi, m);
    }
    __device__ bool contiguous() const { return true; }
    __device__ void first4(int b, int, int64_t c, float clip, float* v) const {
        const int64_t i = b * stride + c;
        float gi[4], m[4];
        __builtin_memcpy(gi, g + i, sizeof(gi));
        __builtin_memcpy(m, mom + i, sizeof(m));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            gi[e] *= clip;
            m[e] = mu * m[e] + one_mu * gi[e];
            v[e] = direction(gi[e], m[e]);
        }
        __builtin_memcpy(mom + i, m, sizeof(m));
    }
    __device__ float again(int b, int r, int64_t c, float clip) const {
        const int64_t i = b * stride + (int64_t)r * cols + c;
        return direction(g[i] * clip, mom[i]);
    }
    __device__ void put(int b, int r, int c, float o) const {
        const int64_t i = b * stride + (int64_t)r * cols + c;
        const float p = master[i];
        const float q = (p - decay * p) - step * o;
        master[i] = q;
        if (slot != nullptr) slot[i] = from_float<DTO>(q);
    }
};

// What a matrix of this norm is multiplied by: fp64, so that no norm overflows
// it; a matrix holding inf or NaN becomes NaN throughout.
__device__ __forceinline__ double scale_of(double norm, float eps) {
    const double d = norm + (double)eps;
    if (!(d < __builtin_inf())) return __builtin_nan("");
    return d > 0.0 ? kXScale / d : 0.0;
}

// Sum over the workgroup, in every thread (fp64; `red`: one double per wave).
__device__ __forceinline__ double block_sum(double v, double* red, int waves) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < waves; ++w) t += red[w];
    return t;
}

// ---------------------------------------------------------------- narrow matrices
// The smaller side is at most T = 32, 64 or 128.  Then S and M fit LDS, and the
// products cost next to nothing against launches and barriers, so here every
// operand is kept in two fp16 parts (high and rest; three products in place of one),
// which makes the iteration as exact as fp32: 1e-5 against 64 bits.
//
// A workgroup of sixteen waves holds a strip of X in registers, in the layout of the
// matrix cores' results: blocks of T x T, each by a group of waves with RT x RT tiles
// of 16 x 16 per wave; G groups side by side and NB blocks after each other, so a
// strip is G * NB * T columns.  A matrix of one strip takes one launch for all its
// steps.  A longer one takes a launch a step, a workgroup a strip: it makes M from all
// the strips' parts of S, applies it to its own columns and writes its part of the
// next S.  Past kFused strips, reading all the parts in every strip costs more than
// one workgroup that makes M in a launch of its own.
//
// What bounds a step is its chain of barriers: of the waves' cycles (32 of 128 x 128) 58%
// wait, 23% for their turn to issue, 7% for LDS, and the matrix cores are busy for 7%.
// Hence many waves with small tiles (eight waves with 32 x 32 tiles took 4.3 us a step at
// 64 x 64 and 10 at 128 x 128; these 1.7 and 7).  Strip<128> spills 7 registers.
template <int T_, int RT_, int G_, int NB_>
struct Strip {
    static constexpr int T = T_, RT = RT_, G = G_, NB = NB_;
    static constexpr int SIDE = T / 16 / RT, GROUP = SIDE * SIDE, WAVES = G * GROUP, THREADS = WAVES * 64;
    static constexpr int COLS = G * NB * T;
    static constexpr int ARRAY = T * T * 2;  // bytes of a T x T fp16 array
    static constexpr int VALUES = RT * RT * 4;  // of a block, per lane
    static constexpr int SIZE = COLS * T;    // elements of a strip
    // S and M by the waves on and below the diagonal only, mirrored: where LDS reads
    // bound the products (128 x 128: 8 against 10 us a step when it was taken, 7 now)
    static constexpr bool MIRROR = RT == 2;
};
typedef Strip<32, 1, 4, 8> Strip32;
typedef Strip<64, 1, 1, 8> Strip64;
typedef Strip<128, 2, 1, 2> Strip128;
constexpr int kFused = 32;

struct Pair {  // high part, and the rest right behind it: arrays in LDS
    char* hi;
};

template <int T>
__device__ __forceinline__ int small_at(int row, int col) {  // byte of an element of a swizzled T x T fp16 array
    constexpr int kPieces = T / 8;
    return row * T * 2 + (((col >> 3) ^ ((row / (128 / T)) & (kPieces - 1))) << 4) + (col & 7) * 2;
}

// Four values as two dwords of fp16, and what that leaves.
__device__ __forceinline__ void split4(const float* x, u32x2& h, u32x2& l) {
    f16x4 a, b;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        a[r] = (_Float16)x[r];
        b[r] = (_Float16)(x[r] - (float)a[r]);
    }
    h = __builtin_bit_cast(u32x2, a);
    l = __builtin_bit_cast(u32x2, b);
}

// LDS of a strip's workgroup: a pair per group for X^T of its current block (or the
// groups' parts of S), one for S and then M, the diagonals.
template <class P>
struct StripLds {
    __attribute__((aligned(16))) char block[P::G * 2 * P::ARRAY];
    __attribute__((aligned(16))) char square[2 * P::ARRAY];
    float ds[P::T], dm[P::T];
    double red[P::WAVES];
};

template <class P>
struct StripWave {
    static constexpr int T = P::T, RT = P::RT;
    typedef float Tiles[RT][RT][4];
    int wave, lane, quarter, c;  // lane / 16, lane % 16
    int group, i0, j0;     // this wave's group, and its tiles' place in a block
    StripLds<P>& lds;
    Pair mine, square;
    int side;        // 32-column pieces of the smaller side
    bool live, both; // whether this wave's rows, and its columns too, meet the smaller side
    bool lower;      // whether it makes its tiles of S and M

    __device__ __forceinline__ StripWave(StripLds<P>& s, int m) : lds(s) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        quarter = lane >> 4;
        c = lane & 15;
        group = wave / P::GROUP;
        int ti = wave % P::GROUP / P::SIDE, tj = wave % P::SIDE;
        if constexpr (P::MIRROR) {
            // the ten tiles on and below the diagonal first, so that they spread over the SIMDs
            static_assert(P::SIDE == 4, "tables of a 4 x 4 grid");
            ti = (int)(0x2110003333222110ull >> 4 * wave & 15);
            tj = (int)(0x3323213210210100ull >> 4 * wave & 15);
        }
        i0 = ti * 16 * RT;
        j0 = tj * 16 * RT;
        mine = {s.block + group * 2 * P::ARRAY};
        square = {s.square};
        side = (m + 31) / 32;
        live = i0 < m;
        both = live && j0 < m;
        lower = !P::MIRROR || i0 >= j0;
    }
    __device__ __forceinline__ int row(int a, int r) const { return i0 + 16 * a + 4 * quarter + r; }
    __device__ __forceinline__ int at(int b) const { return j0 + 16 * b + c; }  // column within a block
    __device__ __forceinline__ int col(int n, int b) const { return (n * P::G + group) * T + at(b); }  // within the strip

    // Forgets what the compiler knows of the lane's place, so that it works addresses
    // and bounds out again rather than keep them in registers across the steps.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(c), "+v"(quarter)); }

    // acc += A B^T of two pairs over the first `pieces` 32 columns, the product of the two
    // rests left out.  Sixteen rows on, the swizzle repeats: a fragment's place is one
    // exclusive or with the k step and a constant.
    __device__ __forceinline__ void product(const Pair& A, const Pair& B, int pieces, f32x4 (&acc)[RT][RT]) const {
        const int pa = small_at<T>(i0 + c, quarter * 8), pb = small_at<T>(j0 + c, quarter * 8);
#pragma unroll 1
        for (int kk = 0; kk < pieces; ++kk) {
            const int xa = pa ^ kk * 64, xb = pb ^ kk * 64;
            f16x8 ah[RT], al[RT], bh[RT], bl[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                ah[t] = *(const f16x8*)(A.hi + xa + t * 16 * T * 2);
                bh[t] = *(const f16x8*)(B.hi + xb + t * 16 * T * 2);
                al[t] = *(const f16x8*)(A.hi + xa + t * 16 * T * 2 + P::ARRAY);
                bl[t] = *(const f16x8*)(B.hi + xb + t * 16 * T * 2 + P::ARRAY);
            }
            multiply(ah, al, bh, bl, acc);
        }
    }
    // Eight values along a column of a pair's array (rows first .. + 7 of this lane's
    // quarter): LDS reads that turn 4 rows x 16 columns among sixteen lanes.
    __device__ __forceinline__ f16x8 column8(const char* a, int to) const {
        typedef int16_t s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* Place;
        // four rows on, the swizzle differs in one bit
        const f16x4 lo = __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Place)(a + to)));
        const f16x4 hi = __builtin_bit_cast(
            f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Place)(a + ((to ^ (T / 32) * 16) + 4 * T * 2))));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // acc += X X^T over the first `pieces` 32 columns of X, from the pair of X^T.
    __device__ __forceinline__ void product_t(const Pair& X, int pieces, f32x4 (&acc)[RT][RT]) const {
        const int r = quarter * 8 + c / 4;
        const int pa = small_at<T>(r, i0 + 4 * (c & 3)), pb = small_at<T>(r, j0 + 4 * (c & 3));
#pragma unroll 1
        for (int kk = 0; kk < pieces; ++kk) {
            const char* rows = X.hi + kk * 32 * T * 2;
            f16x8 ah[RT], al[RT], bh[RT], bl[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                ah[t] = column8(rows, pa ^ t * 32);
                bh[t] = column8(rows, pb ^ t * 32);
                al[t] = column8(rows + P::ARRAY, pa ^ t * 32);
                bl[t] = column8(rows + P::ARRAY, pb ^ t * 32);
            }
            multiply(ah, al, bh, bl, acc);
        }
    }
    // The three products of two pairs' fragments.
    static __device__ __forceinline__ void multiply(const f16x8 (&ah)[RT], const f16x8 (&al)[RT], const f16x8 (&bh)[RT],
                                                    const f16x8 (&bl)[RT], f32x4 (&acc)[RT][RT]) {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah[a], bh[b], acc[a][b], 0, 0, 0);
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(al[a], bh[b], acc[a][b], 0, 0, 0);
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah[a], bl[b], acc[a][b], 0, 0, 0);
    }
    // This wave's tiles into a pair; TURNED: into its transpose.
    template <bool TURNED>
    __device__ __forceinline__ void store(const Pair& P_, const Tiles& v) const {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b) {
                u32x2 h, l;
                split4(v[a][b], h, l);
                int to;
                if constexpr (TURNED) {
                    to = small_at<T>(at(b), row(a, 0));
                } else {
                    h = quad_turn16(h);  // four columns of one row
                    l = quad_turn16(l);
                    to = small_at<T>(row(a, c & 3), j0 + 16 * b + (c & ~3));
                }
                *(u32x2*)(P_.hi + to) = h;
                *(u32x2*)(P_.hi + to + P::ARRAY) = l;
            }
    }
    static __device__ __forceinline__ void zero(f32x4 (&acc)[RT][RT]) {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b) acc[a][b] = f32x4{0, 0, 0, 0};
    }
    // f(a, b, r) for every value of a block
    template <class F>
    static __device__ __forceinline__ void values(F f) {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) f(a, b, r);
    }

    // This wave's tiles of S = X X^T (times kSScale) of the strip's first nb blocks of
    // every group.  cols: the strip's columns.
    __device__ __forceinline__ void gram(const Tiles (&x)[P::NB], int nb, int cols, Tiles& s) {
        f32x4 acc[RT][RT];
        zero(acc);
#pragma unroll
        for (int n = 0; n < P::NB; ++n) {
            if (n >= nb) break;
            __syncthreads();  // the block's last readers are done
            store<true>(mine, x[n]);
            __syncthreads();
            const int left = cols - (n * P::G + group) * T, k = left < T ? left : T;
            if (both && lower && k > 0) product_t(mine, (k + 31) / 32, acc);
        }
        values([&](int a, int b, int r) { s[a][b][r] = acc[a][b][r] * (kSScale / (kXScale * kXScale)); });
        if constexpr (P::G > 1) {
            float* parts = (float*)lds.block;
            __syncthreads();
            values([&](int a, int b, int r) { parts[group * T * T + row(a, r) * T + at(b)] = s[a][b][r]; });
            __syncthreads();
            values([&](int a, int b, int r) {
                float v = 0.0f;
#pragma unroll
                for (int g = 0; g < P::G; ++g) v += parts[g * T * T + row(a, r) * T + at(b)];
                s[a][b][r] = v;
            });
        }
    }

    // Symmetric tiles into the square pair.
    __device__ __forceinline__ void store_square(const Tiles& v) const {
        if (group != 0 || !lower) return;
        store<true>(square, v);
        if (P::MIRROR && i0 != j0) store<false>(square, v);
    }

    // M from S, which every group holds: into the square pair, the diagonal into lds.dm.
    // No barrier after the last writes.
    __device__ __forceinline__ void poly(const Coeffs& k, Tiles& s) {
        const bool diagonal = i0 == j0;  // of the whole wave
        if (diagonal) {
            values([&](int a, int b, int r) {
                if (row(a, r) != at(b)) return;
                if (group == 0) lds.ds[row(a, r)] = s[a][b][r];
                s[a][b][r] = 0.0f;
            });
        }
        store_square(s);
        __syncthreads();
        if (lower) {
            f32x4 acc[RT][RT];
            zero(acc);
            if (both) product(square, square, side, acc);
            float dj[RT];
#pragma unroll
            for (int b = 0; b < RT; ++b) dj[b] = lds.ds[at(b)];
            // all in powers of kSScale: M - diag(M) = b E + c (E E + (d_i + d_j) E)
            const float kb = k.b * k.mscale * (1.0f / kSScale), kc = k.c * k.mscale * (1.0f / (kSScale * kSScale));
            if (diagonal && group == 0) {
                values([&](int a, int b, int r) {
                    if (row(a, r) != at(b)) return;
                    const float d = dj[b] * (1.0f / kSScale), s2 = acc[a][b][r] * (1.0f / (kSScale * kSScale)) + d * d;
                    lds.dm[row(a, r)] = k.a + k.b * d + k.c * s2;
                });
            }
            values([&](int a, int b, int r) {
                const float di = lds.ds[row(a, r)];
                s[a][b][r] = __builtin_fmaf(kb, s[a][b][r], kc * __builtin_fmaf(s[a][b][r], di + dj[b], acc[a][b][r]));
            });
            if (diagonal)
                values([&](int a, int b, int r) {
                    if (row(a, r) == at(b)) s[a][b][r] = 0.0f;
                });
        }
        __syncthreads();  // the readers of S are done
        store_square(s);
    }

    // X <- M X; M's pair and diagonal are written just before, without a barrier.
    // there: the one block's X^T is in its pair (from gram).
    __device__ __forceinline__ void apply(const Coeffs& k, int nb, int cols, bool there, Tiles (&x)[P::NB]) {
        const float un = 1.0f / k.mscale;
#pragma unroll
        for (int n = 0; n < P::NB; ++n) {
            if (n >= nb) break;
            if (n > 0) __syncthreads();
            if (!there) store<true>(mine, x[n]);
            __syncthreads();
            f32x4 acc[RT][RT];
            zero(acc);
            if (live && (n * P::G + group) * T + j0 < cols) product(square, mine, side, acc);
            values([&](int a, int b, int r) { x[n][a][b][r] = __builtin_fmaf(lds.dm[row(a, r)], x[n][a][b][r], acc[a][b][r] * un); });
        }
    }

    // every value of a strip's first nb blocks: f(value, row, column in the strip)
    template <class F>
    __device__ __forceinline__ void each(Tiles (&x)[P::NB], int nb, F f) const {
#pragma unroll
        for (int n = 0; n < P::NB; ++n) {
            if (n >= nb) break;
            values([&](int a, int b, int r) { f(x[n][a][b][r], row(a, r), col(n, b)); });
        }
    }
    // A wave's tiles in memory, a vector of four values a lane at a time: RT * RT * 256 floats.
    __device__ __forceinline__ void save(float* to, const Tiles& v) const {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b)
                *(f32x4*)(to + (a * RT + b) * 256 + lane * 4) = f32x4{v[a][b][0], v[a][b][1], v[a][b][2], v[a][b][3]};
    }
    __device__ __forceinline__ void load(const float* from, Tiles& v) const {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b) {
                const f32x4 w = *(const f32x4*)(from + (a * RT + b) * 256 + lane * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[a][b][r] = w[r];
            }
    }
    // Where this wave's tiles of a T x T matrix, or of a strip's block n, are.
    __device__ __forceinline__ int place() const { return wave % P::GROUP * RT * RT * 256; }
    __device__ __forceinline__ int place(int n) const { return (n * P::WAVES + wave) * RT * RT * 256; }
};

struct StripPlan {
    Coeffs k;
    int m, steps;
    const int32_t* skip;
    // several strips a matrix:
    char* ws;
    int64_t stride;             // bytes from one matrix's workspace to the next
    int64_t parts, next, mat;   // byte offsets of the strips' parts of S, now and next, and of M; X at 0
    int64_t sums;
    int sum_parts, strips;
    int cols;                   // of a strip
    int step;                   // 0: normalise; k: apply the k-th M
    int fused;                  // M is made in every strip
};

template <class IO>
struct StripArgs : StripPlan {
    IO io;
};

// The whole iteration of a matrix of one strip.
template <class P, class IO>
__global__ void __launch_bounds__(P::THREADS) ns_strip_kernel(StripArgs<IO> a) {
    __shared__ StripLds<P> lds;
    if (a.skip != nullptr && *a.skip != 0) return;
    const IO& io = a.io;
    const int b = blockIdx.x;
    const bool tall = io.rows > io.cols;
    const int m = a.m, n = tall ? io.rows : io.cols;
    StripWave<P> w(lds, m);
    const int nb = (n + P::G * P::T - 1) / (P::G * P::T);
    const float clip = io.clip();
    typename StripWave<P>::Tiles x[P::NB], s;
    double ss = 0.0;
    w.each(x, nb, [&](float& v, int i, int j) {
        v = i < m && j < n ? io.first(b, tall ? j : i, tall ? i : j, clip) : 0.0f;
        ss += (double)v * (double)v;
    });
    const double scale = scale_of(sqrt(block_sum(ss, lds.red, P::WAVES)), a.k.eps);
    w.each(x, nb, [&](float& v, int, int) { v = (float)(v * scale); });
    w.forget();
#pragma unroll 1
    for (int step = 0; step < a.steps; ++step) {
        w.gram(x, nb, n, s);
        w.poly(a.k, s);
        w.apply(a.k, nb, n, P::G == 1 && nb == 1, x);
    }
    w.forget();
    w.each(x, nb, [&](float& v, int i, int j) {
        if (i < m && j < n) io.put(b, tall ? j : i, tall ? i : j, v * (1.0f / kXScale));
    });
}

// S of a matrix of several strips, this wave's tiles: the sum of the strips' parts,
// several of them on their way at once.
template <class P, class W>
__device__ __forceinline__ void sum_parts_of(const W& w, const StripPlan& a, const char* ws, typename W::Tiles& s) {
    constexpr int kAtOnce = P::RT == 1 ? 8 : 4;
    const float* parts = (const float*)(ws + a.parts) + w.place();
    W::values([&](int i, int j, int r) { s[i][j][r] = 0.0f; });
    if (!w.lower) return;
    for (int p = 0; p < a.strips; p += kAtOnce) {
        typename W::Tiles v[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            w.load(parts + (int64_t)(p + k < a.strips ? p + k : p) * P::T * P::T, v[k]);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float keep = p + k < a.strips ? 1.0f : 0.0f;
            W::values([&](int i, int j, int r) { s[i][j][r] += keep * v[k][i][j][r]; });
        }
    }
}

// M of a matrix of many strips: both parts of its pair, then the diagonal.
template <class P>
__global__ void __launch_bounds__(P::GROUP * 64) ns_poly_kernel(StripPlan a) {
    typedef Strip<P::T, P::RT, 1, 1> One;
    __shared__ StripLds<One> lds;
    if (a.skip != nullptr && *a.skip != 0) return;
    StripWave<One> w(lds, a.m);
    char* ws = a.ws + blockIdx.x * a.stride;
    typename StripWave<One>::Tiles s;
    sum_parts_of<P>(w, a, ws, s);
    w.poly(a.k, s);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * P::ARRAY / 16; i += One::THREADS)
        ((u32x4*)(ws + a.mat))[i] = ((const u32x4*)lds.square)[i];
    for (int i = threadIdx.x; i < P::T; i += One::THREADS) ((float*)(ws + a.mat + 2 * P::ARRAY))[i] = lds.dm[i];
}

// One strip: step 0 makes X; step k applies the k-th M; the last one writes the
// result, the others their X and part of S.
template <class P, class IO>
__global__ void __launch_bounds__(P::THREADS) ns_strips_kernel(StripArgs<IO> a) {
    __shared__ StripLds<P> lds;
    if (a.skip != nullptr && *a.skip != 0) return;
    const IO& io = a.io;
    const int b = blockIdx.y, strip = blockIdx.x, j0 = strip * a.cols;
    const bool tall = io.rows > io.cols;
    const int m = a.m, n = tall ? io.rows : io.cols;
    StripWave<P> w(lds, m);
    const int left = n - j0 < a.cols ? n - j0 : a.cols, nb = (left + P::G * P::T - 1) / (P::G * P::T);
    char* ws = a.ws + b * a.stride;
    float* mine = (float*)ws + (int64_t)strip * P::SIZE;
    typename StripWave<P>::Tiles x[P::NB], s;
    if (a.step == 0) {
        double ss = 0.0;
        for (int p = threadIdx.x; p < a.sum_parts; p += P::THREADS) ss += ((const double*)(ws + a.sums))[p];
        const double scale = scale_of(sqrt(block_sum(ss, lds.red, P::WAVES)), a.k.eps);
        const float clip = io.clip();
        w.each(x, nb, [&](float& v, int i, int jj) {
            const int j = j0 + jj;
            v = i < m && jj < left ? (float)(io.again(b, tall ? j : i, tall ? i : j, clip) * scale) : 0.0f;
        });
    } else {
#pragma unroll
        for (int k = 0; k < P::NB; ++k)
            if (k < nb) w.load(mine + w.place(k), x[k]);
        if (a.fused) {
            sum_parts_of<P>(w, a, ws, s);
            w.poly(a.k, s);
        } else {
            for (int i = threadIdx.x; i < 2 * P::ARRAY / 16; i += P::THREADS)
                ((u32x4*)lds.square)[i] = ((const u32x4*)(ws + a.mat))[i];
            for (int i = threadIdx.x; i < P::T; i += P::THREADS) lds.dm[i] = ((const float*)(ws + a.mat + 2 * P::ARRAY))[i];
        }
        w.apply(a.k, nb, left, false, x);
    }
    if (a.step == a.steps) {
        w.each(x, nb, [&](float& v, int i, int jj) {
            const int j = j0 + jj;
            if (i < m && jj < left) io.put(b, tall ? j : i, tall ? i : j, v * (1.0f / kXScale));
        });
        return;
    }
#pragma unroll
    for (int k = 0; k < P::NB; ++k)
        if (k < nb) w.save(mine + w.place(k), x[k]);
    w.gram(x, nb, left, s);
    if (w.group == 0 && w.lower) w.save((float*)(ws + a.next) + (int64_t)strip * P::T * P::T + w.place(), s);
}

// ---------------------------------------------------------------- large matrices
constexpr int kSumThreads = 256;
constexpr int64_t kSumElems = 8192;  // elements per partial sum of squares, at least
constexpr int kMaxParts = 1024;

template <class IO>
struct IoArgs {
    IO io;
    Work w;
    float eps;
};

// One partial of the squared norm per workgroup (and the momentum update): runs of
// kSumRun elements, four per thread; contiguous matrices as one long row.
constexpr int kSumRun = 4 * kSumThreads;
template <class IO>
__global__ void __launch_bounds__(kSumThreads) ns_sum_kernel(IoArgs<IO> a) {
    __shared__ double red[kSumThreads / 64];
    if (a.w.skipped()) return;
    const int b = blockIdx.y;
    const bool flat = a.io.contiguous();
    const int64_t cols = flat ? (int64_t)a.io.rows * a.io.cols : a.io.cols;
    const uint32_t across = (uint32_t)((cols + kSumRun - 1) / kSumRun), runs = across * (flat ? 1 : a.io.rows);
    const float clip = a.io.clip();
    double ss = 0.0;
    for (uint32_t run = blockIdx.x; run < runs; run += gridDim.x) {
        const int r = (int)(run / across);
        const int64_t c = (int64_t)(run % across) * kSumRun + threadIdx.x * 4;
        if (c >= cols) continue;
        float v[4] = {0, 0, 0, 0};
        if (c + 4 <= cols) {
            a.io.first4(b, r, c, clip, v);
        } else {
            for (int e = 0; c + e < cols; ++e) v[e] = a.io.first(b, r, c + e, clip);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) ss += (double)v[e] * (double)v[e];
    }
    const double t = block_sum(ss, red, kSumThreads / 64);
    if (threadIdx.x == 0) ((double*)(a.w.of(b) + a.w.sums))[blockIdx.x] = t;
}

constexpr int kPatch = 64;  // elements each way of the patches that change orientation

// X = u / (||u|| + eps) in fp32 and fp16, and its fp16 transpose, the padding
// zeroed.  A patch of the source per workgroup, turned through LDS.
template <class IO>
__global__ void __launch_bounds__(256) ns_begin_kernel(IoArgs<IO> a) {
    __shared__ float patch[kPatch][kPatch + 1];
    __shared__ double red[4];
    const Work& w = a.w;
    if (w.skipped()) return;
    const int b = blockIdx.z, tid = threadIdx.x;
    char* base = w.of(b);
    const bool tall = a.io.rows > a.io.cols;
    double ss = 0.0;
    for (int p = tid; p < w.parts; p += 256) ss += ((const double*)(base + w.sums))[p];
    const double norm = sqrt(block_sum(ss, red, 4));
    const double scale = scale_of(norm, a.eps);
    const float clip = a.io.clip();

    const int r0 = blockIdx.y * kPatch, c0 = blockIdx.x * kPatch, x = tid & 63, y = tid >> 6;
#pragma unroll 4
    for (int i = y; i < kPatch; i += 4) {
        const int r = r0 + i, c = c0 + x;
        patch[i][x] = r < a.io.rows && c < a.io.cols ? (float)(a.io.again(b, r, c, clip) * scale) : 0.0f;
    }
    __syncthreads();
    float* x32 = (float*)base;
    _Float16 *x16 = (_Float16*)(base + w.x16), *xt = (_Float16*)(base + w.xt0);
    // wide orientation: row i of the patch's rows (or columns, when tall)
    const int i0 = tall ? c0 : r0, j0 = tall ? r0 : c0;
    {  // the patch's part of the squared row norms, four lanes a row
        const int i = tid >> 2, from = (tid & 3) * (kPatch / 4);
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < kPatch / 4; ++e) {
            const float v = tall ? patch[from + e][i] : patch[i][from + e];
            t += v * v;
        }
        t += __shfl_xor(t, 1);
        t += __shfl_xor(t, 2);
        if ((tid & 3) == 0 && i0 + i < w.m) ((float*)(base + w.rows))[(int64_t)(j0 / kPatch) * w.mp + i0 + i] = t;
    }
    for (int i = y; i < kPatch; i += 4) {
        const float v = tall ? patch[x][i] : patch[i][x];   // element (i0 + i, j0 + x) of X
        const float vt = tall ? patch[i][x] : patch[x][i];  // element (i0 + x, j0 + i) of X
        if (i0 + i < w.m && j0 + x < w.np) {
            x32[(int64_t)(i0 + i) * w.np + j0 + x] = v;
            const int64_t at = (int64_t)(i0 + i) * w.nx + j0 + x;
            const _Float16 high = half_fma(v, spread(i0 + i));
            x16[at + (w.nx - w.np)] = high;
            if (w.nx > w.np) x16[at] = half_fma(v, spread(i0 + i), -(float)high);
        }
        if (j0 + i < w.n && i0 + x < w.mp) {
            const int64_t at = (int64_t)(j0 + i) * w.kp + i0 + x;
            const _Float16 high = half_fma(vt, spread(j0 + i));
            xt[at + (w.kp - w.mp)] = high;
            if (w.kp > w.mp) xt[at] = half_fma(vt, spread(j0 + i), -(float)high);
        }
    }
}

// The result in the source's orientation.
template <class IO>
__global__ void __launch_bounds__(256) ns_end_kernel(IoArgs<IO> a) {
    __shared__ float patch[kPatch][kPatch + 1];
    const Work& w = a.w;
    if (w.skipped()) return;
    const int b = blockIdx.z, tid = threadIdx.x, x = tid & 63, y = tid >> 6;
    const bool tall = a.io.rows > a.io.cols;
    const float* x32 = (const float*)w.of(b);
    const int r0 = blockIdx.y * kPatch, c0 = blockIdx.x * kPatch;
    const int i0 = tall ? c0 : r0, j0 = tall ? r0 : c0;
#pragma unroll 4
    for (int i = y; i < kPatch; i += 4)
        if (i0 + i < w.m && j0 + x < w.n) patch[i][x] = x32[(int64_t)(i0 + i) * w.np + j0 + x];
    __syncthreads();
    for (int i = y; i < kPatch; i += 4) {
        const int r = r0 + i, c = c0 + x;
        if (r < a.io.rows && c < a.io.cols) a.io.put(b, r, c, (tall ? patch[x][i] : patch[i][x]) * (1.0f / kXScale));
    }
}

struct StepArgs {
    Work w;
    Coeffs k;
    int tiles_m, tiles_n;  // tile grid of the product with M
    int tiles;             // tiles on and above the diagonal of S or M
    int odd;               // which copy of X^T is current
    int last;              // the last step: only the fp32 X is wanted
    int row_parts;         // parts of each squared row norm of X
};

// Upper triangle tile t -> (i <= j).
__device__ __forceinline__ void triangle_tile(int t, int& i, int& j) {
    j = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (j * (j + 1) / 2 > t) --j;
    while ((j + 1) * (j + 2) / 2 <= t) ++j;
    i = t - j * (j + 1) / 2;
}

// Results leave through two doors.  Four lanes turn their 4 x 4 values, so a
// lane then has four neighbouring columns of one row: row-major reads and writes
// are vectors.  The transposed copy goes through the wave's part of LDS.
template <class S>
constexpr int ns_lds() {
    const int a = product_lds<S, MmF16>(), b = 2 * S::WAVES * Turner<S>::kBytes;
    return a > b ? a : b;
}

// The diagonal of S for 64 rows, a lane each: the parts of the rows' squared norms,
// summed by the waves in turn and then over the waves (`sums`: 64 floats per wave).
constexpr int kNormRows = 64;
template <int WAVES>
__device__ __forceinline__ void row_norms(const Work& w, char* base, int row_parts, int first, float* sums) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = first + lane;
    const float* parts = (const float*)(base + w.rows) + (i < w.m ? i : w.m - 1);
    float t = 0.0f;
#pragma unroll 8
    for (int p = wave; p < row_parts; p += WAVES) t += parts[(int64_t)p * w.mp];
    sums[wave * 64 + lane] = t;
    __syncthreads();
    if (wave > 0 || i >= w.m) return;
#pragma unroll
    for (int v = 1; v < WAVES; ++v) t += sums[v * 64 + lane];
    ((float*)(base + w.ds))[i] = t * (1.0f / (kXScale * kXScale));
}

// S (POLY false) or M (POLY true): tiles on and above the diagonal, mirrored.  S: the
// workgroups after the tiles' make its diagonal, 64 rows each.  EXACT: operands of two parts.
template <class S, bool POLY, bool EXACT>
__global__ void __launch_bounds__(S::THREADS) ns_square_kernel(StepArgs a) {
    __shared__ __attribute__((aligned(16))) char lds[ns_lds<S>()];
    const Work& w = a.w;
    if (w.skipped()) return;
    char* base = w.of(blockIdx.y);
    if constexpr (!POLY) {
        if ((int)blockIdx.x >= a.tiles) {
            row_norms<S::THREADS / 64>(w, base, a.row_parts, ((int)blockIdx.x - a.tiles) * kNormRows, (float*)lds);
            return;
        }
    }
    int ti, tj;
    triangle_tile(xcd_tile(blockIdx.x, a.tiles), ti, tj);
    const int ld = POLY ? w.ms : w.nx;  // elements
    const char* from = base + (POLY ? w.s16 : w.x16);
    const int i0 = ti * S::TILE, j0 = tj * S::TILE;
    const Operand A{from + (int64_t)i0 * ld * 2, (uint32_t)ld * 2, w.m - i0};
    const Operand B{from + (int64_t)j0 * ld * 2, (uint32_t)ld * 2, w.m - j0};
    f32x16 acc[S::MT][S::NT];
    Product<S, MmF16, EXACT ? 2 : 1> product(lds, (POLY ? w.mp : w.np) / 64, false);
    product.tile(A, B, A, B);
    product.ahead();
    const bool holds = product.run(acc);
    __syncthreads();  // LDS is free
    if (!holds) return;

    const Lane L(S::WAVES);
    const int iw = i0 + L.wave / (S::TILE / S::WN) * S::WM, jw = j0 + L.wave % (S::TILE / S::WN) * S::WN;
    const Coeffs& k = a.k;
    float* dm = (float*)(base + w.dm);
    const float* ds = (const float*)(base + w.ds);
    const _Float16* s16 = (const _Float16*)(base + w.s16);
    _Float16* out = (_Float16*)(base + (POLY ? w.m16 : w.s16));
    const int ldo = POLY ? w.kp : w.ms;
    const bool twice = POLY && !EXACT && w.kp > w.mp;  // M meets both parts of X^T
    Turner<S> turner(lds, L), rest(lds + S::WAVES * Turner<S>::kBytes, L);
#pragma unroll
    for (int jj = 0; jj < S::NT; ++jj) {
        const int j = jw + jj * 32 + (L.c & ~3);  // and the three after it
        // worked out again for every column block: kept across them, the rows' addresses and
        // factors take registers that the tile of 256 has not left
        int mine = iw + 4 * L.h + (L.c & 3);
        asm volatile("" : "+v"(mine));
        float tj4[4], uj4[4];  // the columns' factors: their rows' of the mirrored tile
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            tj4[e] = spread(j + e);
            uj4[e] = __builtin_amdgcn_rcpf(tj4[e]);
        }
        // what the tile needs from memory, all of a column block before its first use
        float dj[4], di4[S::MT * 4];
        f16x4 old[S::MT * 4], old_rest[EXACT ? S::MT * 4 : 1];
        if constexpr (POLY) {
#pragma unroll
            for (int e = 0; e < 4; ++e) dj[e] = ds[j + e < w.m ? j + e : w.m - 1];
#pragma unroll
            for (int t = 0; t < S::MT * 4; ++t) {
                const int i = mine + 8 * t, ic = i < w.m ? i : w.m - 1;
                const _Float16* at = s16 + (int64_t)ic * w.ms + (j < w.mp ? j : w.mp - 4);
                old[t] = *(const f16x4*)(EXACT ? at + w.mp : at);
                if constexpr (EXACT) old_rest[t] = *(const f16x4*)at;
                di4[t] = ds[ic];
            }
        }
#pragma unroll
        for (int ii = 0; ii < S::MT; ++ii)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = ii * 32 + 8 * q + 4 * L.h, i = mine + ii * 32 + 8 * q;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[ii][jj][4 * q + r];
                quad_turn(v);
                const bool inside = i < w.m && j < w.mp;
                const float ti1 = spread(i), ui1 = __builtin_amdgcn_rcpf(ti1);
                // the value times its row's factor, and times its column's; what their rounding leaves
                f16x4 h, mirrored, h_rest, mirrored_rest;
                if constexpr (POLY) {
                    const float di = di4[ii * 4 + q];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = (float)old[ii * 4 + q][e];
                        if constexpr (EXACT) x += (float)old_rest[ii * 4 + q][e];
                        x *= (1.0f / kSScale) * ui1;
                        float s2 = v[e] * (1.0f / (kSScale * kSScale)) * (ui1 * uj4[e]) + x * (di + dj[e]);
                        if (i == j + e) {
                            s2 += di * di;
                            if (i < w.m) dm[i] = k.a + k.b * di + k.c * s2;
                        }
                        v[e] = i == j + e ? 0.0f : (k.b * x + k.c * s2) * k.mscale;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (i == j + e) v[e] = 0.0f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (i >= w.m || j + e >= w.m) v[e] = 0.0f;  // rows repeated past the end
                    // S: one of the two factors that the product carries is wanted
                    constexpr float kOne = kSScale / (kXScale * kXScale);
                    const float fi = POLY ? ti1 : uj4[e] * kOne, fj = POLY ? tj4[e] : ui1 * kOne;
                    h[e] = half_fma(v[e], fi);
                    mirrored[e] = half_fma(v[e], fj);
                    if constexpr (EXACT) {
                        h_rest[e] = half_fma(v[e], fi, -(float)h[e]);
                        mirrored_rest[e] = half_fma(v[e], fj, -(float)mirrored[e]);
                    }
                }
                if (inside) *(f16x4*)(out + (int64_t)i * ldo + j) = EXACT ? h_rest : h;
                if (inside && (EXACT || twice)) *(f16x4*)(out + (int64_t)i * ldo + w.mp + j) = h;
                if (ti != tj) {
                    turner.put(L, row, quad_turn16(mirrored));
                    if constexpr (EXACT) rest.put(L, row, quad_turn16(mirrored_rest));
                }
            }
        if (ti != tj) {
            turner.flush(L, EXACT ? out + w.mp : out, ldo, jw + jj * 32, iw, w.m, w.mp);
            if constexpr (EXACT) rest.flush(L, out, ldo, jw + jj * 32, iw, w.m, w.mp);
            if (twice) turner.flush(L, out + w.mp, ldo, jw + jj * 32, iw, w.m, w.mp);
        }
    }
}

// X <- diag(M) X + (M - diag(M)) X, with its fp16 copies for the next step.
template <class S, bool EXACT>
__global__ void __launch_bounds__(S::THREADS) ns_apply_kernel(StepArgs a) {
    __shared__ __attribute__((aligned(16))) char lds[ns_lds<S>()];
    const Work& w = a.w;
    if (w.skipped()) return;
    char* base = w.of(blockIdx.y);
    int ti, tj;
    band_tile(xcd_tile(blockIdx.x, gridDim.x), a.tiles_m, a.tiles_n, ti, tj);
    const int i0 = ti * S::TILE, j0 = tj * S::TILE;
    const char* xt = base + (a.odd ? w.xt1 : w.xt0);
    const Operand A{base + w.m16 + (int64_t)i0 * w.kp * 2, (uint32_t)w.kp * 2, w.m - i0};
    const Operand B{xt + (int64_t)j0 * w.kp * 2, (uint32_t)w.kp * 2, w.n - j0};
    f32x16 acc[S::MT][S::NT];
    Product<S, MmF16, EXACT ? 2 : 1> product(lds, (EXACT ? w.mp : w.kp) / 64, false);
    product.tile(A, B, A, B);
    product.ahead();
    const bool holds = product.run(acc);
    __syncthreads();  // LDS is free
    if (!holds) return;

    const Lane L(S::WAVES);
    const int iw = i0 + L.wave / (S::TILE / S::WN) * S::WM, jw = j0 + L.wave % (S::TILE / S::WN) * S::WN;
    const float un = 1.0f / a.k.mscale;
    const float* dm = (const float*)(base + w.dm);
    float* x32 = (float*)base;
    _Float16 *x16 = (_Float16*)(base + w.x16), *next = (_Float16*)(base + (a.odd ? w.xt0 : w.xt1));
    const bool two = EXACT || w.kp > w.mp;
    Turner<S> turner(lds, L), rest(lds + S::WAVES * Turner<S>::kBytes, L);
    float norms[S::MT * 4];  // of this lane's rows, its columns' part
#pragma unroll
    for (int t = 0; t < S::MT * 4; ++t) norms[t] = 0.0f;
#pragma unroll
    for (int jj = 0; jj < S::NT; ++jj) {
        const int j = jw + jj * 32 + (L.c & ~3);
        // worked out again, as in ns_square_kernel (47 registers spilled without)
        int mine = iw + 4 * L.h + (L.c & 3);
        asm volatile("" : "+v"(mine));
        float tj4[4], uj4[4];  // the columns' factors
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            tj4[e] = spread(j + e);
            uj4[e] = __builtin_amdgcn_rcpf(tj4[e]) * un;
        }
        // X of the column block, all of it before its first use
        f32x4 old[S::MT * 4];
        float dm4[S::MT * 4];
#pragma unroll
        for (int t = 0; t < S::MT * 4; ++t) {
            const int i = mine + 8 * t, ic = i < w.m ? i : w.m - 1;
            old[t] = *(const f32x4*)(x32 + (int64_t)ic * w.np + (j < w.np ? j : w.np - 4));
            dm4[t] = dm[ic];
        }
#pragma unroll
        for (int ii = 0; ii < S::MT; ++ii)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = ii * 32 + 8 * q + 4 * L.h, i = mine + ii * 32 + 8 * q;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[ii][jj][4 * q + r];
                quad_turn(v);
                const bool inside = i < w.m && j < w.np;
                const int64_t at = (int64_t)i * w.np + j;
                f32x4 x = old[ii * 4 + q];
                const float d = dm4[ii * 4 + q], ti1 = spread(i), ui1 = __builtin_amdgcn_rcpf(ti1);
                f16x4 h, turned, h_rest;  // for X and for X^T, whose rows are the columns here
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // past the ends of both sides: rows repeated
                    v[e] = inside && j + e < w.n ? __builtin_fmaf(d, x[e], v[e] * (ui1 * uj4[e])) : 0.0f;
                    x[e] = v[e];
                    norms[ii * 4 + q] = __builtin_fmaf(v[e], v[e], norms[ii * 4 + q]);
                    h[e] = half_fma(v[e], ti1);
                    if constexpr (EXACT) h_rest[e] = half_fma(v[e], ti1, -(float)h[e]);
                    turned[e] = half_fma(v[e], tj4[e]);
                }
                if (inside) {
                    *(f32x4*)(x32 + at) = x;
                    if (!a.last) {
                        _Float16* const to = x16 + (int64_t)i * w.nx + j;
                        *(f16x4*)(EXACT ? to + w.np : to) = h;
                        if constexpr (EXACT) *(f16x4*)to = h_rest;
                    }
                }
                if (!a.last) {
                    turner.put(L, row, quad_turn16(turned));
                    if (two) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) turned[e] = half_fma(v[e], tj4[e], -(float)turned[e]);
                        rest.put(L, row, quad_turn16(turned));
                    }
                }
            }
        if (!a.last) {
            turner.flush(L, next + (w.kp - w.mp), w.kp, jw + jj * 32, iw, w.n, w.mp);
            if (two) rest.flush(L, next, w.kp, jw + jj * 32, iw, w.n, w.mp);
        }
    }
    if (!a.last) {  // the eight lanes that share a row: a part of its squared norm for every wave's columns
        constexpr int kAcross = S::TILE / S::WN;
        float* part = (float*)(base + w.rows) + (int64_t)(tj * kAcross + L.wave % kAcross) * w.mp;
#pragma unroll
        for (int t = 0; t < S::MT * 4; ++t) {
            float v = norms[t];
            v += quad_swap<0x124>(v);  // of the lane four on among sixteen, then eight
            v += quad_swap<0x128>(v);
            v += __shfl_xor(v, 16);
            const int i = iw + t / 4 * 32 + 8 * (t % 4) + 4 * L.h + (L.c & 3);
            if (L.c < 4 && i < w.m) part[i] = v;
        }
    }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kMaxSide = 65536;
constexpr int32_t kMaxCount = 65535;
constexpr int kNarrow = 128;  // smaller sides up to this take the strip kernels
// Up to this smaller side the product with M takes X in two fp16 parts.  The rounding
// of X puts noise into directions that X lacks, which grows 140-fold over the
// steps after; it averages out over a long side only (a matrix of rank one was 4e-3
// off at 130 x 200 with one part, 2e-3 at 256 x 700).
constexpr int kTwoParts = 512;

bool narrow(int64_t rows, int64_t cols) { return rows <= kNarrow || cols <= kNarrow; }

int sum_parts(int64_t rows, int64_t cols) {
    const int64_t p = ceil_div(rows * cols, kSumElems);
    return (int)(p < kMaxParts ? p : kMaxParts);
}

// The workspace block of one matrix; exact: all operands in two parts.
Work work_of(int64_t rows, int64_t cols, bool exact) {
    Work w{};
    w.m = (int)(rows < cols ? rows : cols);
    w.n = (int)(rows < cols ? cols : rows);
    w.mp = (int)round_up(w.m, 64);
    w.np = (int)round_up(w.n, 64);
    w.kp = exact || w.m <= kTwoParts ? 2 * w.mp : w.mp;
    w.nx = exact ? 2 * w.np : w.np;
    w.ms = exact ? 2 * w.mp : w.mp;
    w.parts = sum_parts(rows, cols);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    take((int64_t)w.m * w.np * 4);
    w.x16 = take((int64_t)w.m * w.nx * 2);
    w.xt0 = take((int64_t)w.n * w.kp * 2);
    w.xt1 = take((int64_t)w.n * w.kp * 2);
    w.s16 = take((int64_t)w.m * w.ms * 2);
    w.m16 = take((int64_t)w.m * w.kp * 2);
    w.ds = take((int64_t)w.m * 4);
    w.dm = take((int64_t)w.m * 4);
    w.sums = take((int64_t)w.parts * 8);
    w.rows = take((int64_t)(w.np / 64) * 2 * w.mp * 4);  // tiles of 64 have the most: two waves each
    w.stride = at;
    return w;
}

// The strips of a narrow matrix of a stack: f(Strip32(), count of strips, columns of
// each) and so on.  One strip where the stack alone fills the CUs or the
// matrix has up to three rounds of blocks; else strips as short as kFused of them
// allow, since a strip takes its blocks one after another.
template <class P>
int strip_cols(int32_t count, int64_t n) {
    const int64_t round = P::G * P::T, rounds = ceil_div(n, round);
    if (rounds <= P::NB && (rounds <= 3 || count >= 128)) return (int)(rounds * round);
    int64_t per = ceil_div(rounds, kFused);
    const int64_t fill = ceil_div(rounds * count, 256);  // more strips than CUs gain nothing
    if (per < fill) per = fill;
    return (int)((per < P::NB ? per : P::NB) * round);
}

template <class F>
auto with_strip(int32_t count, int64_t rows, int64_t cols, F f) {
    const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    auto go = [&](auto shape) {
        const int each = strip_cols<decltype(shape)>(count, n);
        return f(shape, (int)ceil_div(n, each), each);
    };
    if (m <= 32) return go(Strip32());
    if (m <= 64) return go(Strip64());
    return go(Strip128());
}

// Workspace of one narrow matrix of several strips: X, the parts of S, M, the sums.
struct StripWork {
    int64_t parts[2], mat, sums, stride;
};

template <class P>
StripWork strip_work(int strips, int sum_parts) {
    StripWork w;
    w.parts[0] = round_up((int64_t)strips * P::SIZE * 4, 256);
    w.parts[1] = w.parts[0] + round_up((int64_t)strips * P::T * P::T * 4, 256);
    w.mat = w.parts[1] + round_up((int64_t)strips * P::T * P::T * 4, 256);
    w.sums = w.mat + round_up(2 * P::ARRAY + P::T * 4, 256);
    w.stride = w.sums + round_up((int64_t)sum_parts * 8, 256);
    return w;
}

// The largest singular value that an iterate which enters a product (all but the last)
// can have: those of the first are up to 1.
double reach(const zero_newton_schulz& ns) {
    const double a = ns.a, b = ns.b, c = ns.c;
    double top = 1.0, r = 1.0;
    for (int step = 1; step < ns.steps && top <= ZERO_NS_REACH; ++step) {
        auto at = [&](double t) { return std::fabs(std::sqrt(t) * (a + t * (b + t * c))); };  // t = s^2
        double next = at(r * r);
        auto turn = [&](double t) {
            if (t > 0.0 && t < r * r) next = std::fmax(next, at(t));
        };
        // a + 3 b t + 5 c t^2 = 0
        if (c == 0.0) {
            if (b != 0.0) turn(-a / (3.0 * b));
        } else {
            const double half = -3.0 * b / (10.0 * c), under = half * half - a / (5.0 * c);
            if (under >= 0.0) {
                turn(half - std::sqrt(under));
                turn(half + std::sqrt(under));
            }
        }
        r = next;
        top = std::fmax(top, r);
    }
    return top;
}

int check_ns(const zero_newton_schulz* ns, const char* what) {
    if (ns == nullptr) return fail(ZERO_EINVAL, "%s: null settings", what);
    if (!std::isfinite(ns->a) || !std::isfinite(ns->b) || !std::isfinite(ns->c))
        return fail(ZERO_EINVAL, "%s: coefficients must be finite", what);
    if (!std::isfinite(ns->eps) || ns->eps < 0.0f) return fail(ZERO_EINVAL, "%s: eps must be >= 0", what);
    if (ns->steps < 0 || ns->steps > 64) return fail(ZERO_EINVAL, "%s: steps must be 0..64", what);
    if (!(reach(*ns) <= ZERO_NS_REACH))
        return fail(ZERO_EINVAL, "%s: the coefficients let singular values between steps grow above %g", what, ZERO_NS_REACH);
    return ZERO_OK;
}

int check_stack(int32_t count, int64_t rows, int64_t cols, const char* what) {
    if (count < 0 || count > kMaxCount) return fail(ZERO_ERANGE, "%s: count %d out of range", what, count);
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return fail(ZERO_ERANGE, "%s: %lld x %lld out of range (at most %lld each way)", what, (long long)rows,
                    (long long)cols, (long long)kMaxSide);
    return ZERO_OK;
}

int check_space(const void* ws, size_t ws_bytes, size_t need, const char* what) {
    if (need == 0) return ZERO_OK;
    if (ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
    if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
    if (ws_bytes < need)
        return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
    return ZERO_OK;
}

Coeffs coeffs_of(const zero_newton_schulz& ns) {
    Coeffs k{ns.a, ns.b, ns.c, ns.eps, 0.0f};
    // M for S up to 1.5, which the usual coefficients keep to, or up to what these let it reach; S times
    // kSScale stays in fp16's range for a reach of ZERO_NS_REACH, its elements off the diagonal at most half of it
    const double far = reach(ns), s = far * far > 1.5 ? far * far : 1.5;
    const double top = std::fabs((double)ns.a) + s * std::fabs((double)ns.b) + s * s * std::fabs((double)ns.c);
    int e = 0;
    std::frexp(top, &e);  // top < 2^e
    e = 15 - e;
    k.mscale = (float)std::ldexp(1.0, e > 15 ? 15 : e < -100 ? -100 : e);
    return k;
}

// The steps of a large stack: three launches each.
template <bool EXACT>
int run_steps(const Work& w, const Coeffs& k, int32_t count, int steps, hipStream_t s, const char* what) {
    auto square_tiles = [&](int64_t t) { return count * (ceil_div(w.m, t) * (ceil_div(w.m, t) + 1) / 2); };
    auto whole_tiles = [&](int64_t t) { return count * ceil_div(w.m, t) * ceil_div(w.np, t); };
    const int square = pick_tile(square_tiles), whole = pick_tile(whole_tiles);
    StepArgs a{w, k, 0, 0, 0, 0, 0, w.np / kPatch};  // ns_begin's parts of the row norms
    auto squares = [&](auto poly) {
        return with_tile(square, [&](auto shape) {
            typedef decltype(shape) S;
            a.tiles = (int)(square_tiles(S::TILE) / count);
            const int64_t norms = decltype(poly)::value ? 0 : ceil_div(w.m, kNormRows);
            const dim3 grid((unsigned)(a.tiles + norms), (unsigned)count);
            return launch(ns_square_kernel<S, decltype(poly)::value, EXACT>, grid, S::THREADS, s, a, what);
        });
    };
    for (int i = 0; i < steps; ++i) {
        a.odd = i & 1;
        a.last = i + 1 == steps;
        int rc;
        if ((rc = squares(std::false_type())) != ZERO_OK || (rc = squares(std::true_type())) != ZERO_OK) return rc;
        rc = with_tile(whole, [&](auto shape) {
            typedef decltype(shape) S;
            a.tiles_m = (int)ceil_div(w.m, S::TILE);
            a.tiles_n = (int)ceil_div(w.np, S::TILE);
            const int launched = launch(ns_apply_kernel<S, EXACT>, dim3((unsigned)(a.tiles_m * a.tiles_n), (unsigned)count),
                                        S::THREADS, s, a, what);
            a.row_parts = a.tiles_n * (S::TILE / S::WN);
            return launched;
        });
        if (rc != ZERO_OK) return rc;
    }
    return ZERO_OK;
}

template <class IO>
int run_strips(const IO& io, int32_t count, const zero_newton_schulz& ns, const Coeffs& k, const int32_t* skip,
               void* ws, hipStream_t s, const char* what) {
    return with_strip(count, io.rows, io.cols, [&](auto shape, int strips, int each_cols) {
        typedef decltype(shape) P;
        const int m = io.rows < io.cols ? io.rows : io.cols;
        StripArgs<IO> a{{k, m, ns.steps, skip, (char*)ws, 0, 0, 0, 0, 0, 0, strips, each_cols, 0, strips <= kFused}, io};
        const dim3 each((unsigned)count);
        if (strips == 1) return launch(ns_strip_kernel<P, IO>, each, P::THREADS, s, a, what);
        a.sum_parts = sum_parts(io.rows, io.cols);
        const StripWork w = strip_work<P>(strips, a.sum_parts);
        a.mat = w.mat;
        a.sums = w.sums;
        a.stride = w.stride;
        Work sum{};
        sum.base = (char*)ws;
        sum.stride = w.stride;
        sum.sums = w.sums;
        sum.skip = skip;
        int rc = launch(ns_sum_kernel<IO>, dim3((unsigned)a.sum_parts, (unsigned)count), kSumThreads, s,
                        IoArgs<IO>{io, sum, ns.eps}, what);
        for (a.step = 0; rc == ZERO_OK && a.step <= ns.steps; ++a.step) {
            a.parts = w.parts[a.step & 1];  // a strip may still read them when another one writes the next
            a.next = w.parts[(a.step + 1) & 1];
            if (a.step > 0 && !a.fused) rc = launch(ns_poly_kernel<P>, each, P::GROUP * 64, s, (const StripPlan&)a, what);
            if (rc == ZERO_OK)
                rc = launch(ns_strips_kernel<P, IO>, dim3((unsigned)strips, (unsigned)count), P::THREADS, s, a, what);
        }
        return rc;
    });
}

template <class IO>
int run_stack(const IO& io, int32_t count, const zero_newton_schulz& ns, const int32_t* skip, void* ws,
              hipStream_t s, const char* what) {
    int rc = ZERO_OK;
    const Coeffs k = coeffs_of(ns);
    if constexpr (IO::kNarrow) {
        if (narrow(io.rows, io.cols)) return run_strips(io, count, ns, k, skip, ws, s, what);
    }
    Work w = work_of(io.rows, io.cols, IO::kExact);
    w.base = (char*)ws;
    w.skip = skip;
    const IoArgs<IO> a{io, w, ns.eps};
    if ((rc = launch(ns_sum_kernel<IO>, dim3((unsigned)w.parts, (unsigned)count), kSumThreads, s, a, what)) != ZERO_OK)
        return rc;
    // patches cover the padding of both orientations
    const dim3 patches((unsigned)ceil_div(io.cols, kPatch), (unsigned)ceil_div(io.rows, kPatch), (unsigned)count);
    if ((rc = launch(ns_begin_kernel<IO>, patches, 256, s, a, what)) != ZERO_OK) return rc;
    if ((rc = run_steps<IO::kExact>(w, k, count, ns.steps, s, what)) != ZERO_OK) return rc;
    return launch(ns_end_kernel<IO>, patches, 256, s, a, what);
}

}  // namespace

extern "C" {

static size_t workspace_bytes(int32_t count, int64_t rows, int64_t cols, bool exact) {
    if (count <= 0 || count > kMaxCount || rows <= 0 || cols <= 0 || rows > kMaxSide || cols > kMaxSide) return 0;
    if (narrow(rows, cols))
        return with_strip(count, rows, cols, [&](auto shape, int strips, int) -> size_t {
            if (strips == 1) return 0;
            return (size_t)strip_work<decltype(shape)>(strips, sum_parts(rows, cols)).stride * (size_t)count;
        });
    return (size_t)work_of(rows, cols, exact).stride * (size_t)count;
}

size_t zero_ns_workspace_bytes(int32_t count, int64_t rows, int64_t cols) {
    return workspace_bytes(count, rows, cols, true);
}

size_t zero_muon_workspace_bytes(int32_t count, int64_t rows, int64_t cols) {
    return workspace_bytes(count, rows, cols, false);
}

int zero_orthogonalize(const void* src, int32_t src_dtype, int32_t count, int64_t rows, int64_t cols,
                       int64_t src_ld, int64_t src_stride, void* dst, int32_t dst_dtype, int64_t dst_ld,
                       int64_t dst_stride, const zero_newton_schulz* ns, void* ws, size_t ws_bytes, void* stream) {
    const char* what = "zero_orthogonalize";
    int rc;
    if (!valid_dtype(src_dtype, true) || !valid_dtype(dst_dtype, false))
        return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_ns(ns, what)) != ZERO_OK) return rc;
    if ((rc = check_stack(count, rows, cols, what)) != ZERO_OK) return rc;
    if (count == 0 || rows == 0 || cols == 0) return ok();
    if (src == nullptr || dst == nullptr) return fail(ZERO_EINVAL, "%s: null matrices", what);
    if (!aligned(src, elem_bytes(src_dtype)) || !aligned(dst, 2))
        return fail(ZERO_EALIGN, "%s: matrices not aligned to their elements", what);
    if (src_ld < cols || dst_ld < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (count > 1 && (src_stride < (rows - 1) * src_ld + cols || dst_stride < (rows - 1) * dst_ld + cols))
        return fail(ZERO_ERANGE, "%s: matrices overlap", what);
    const size_t need = workspace_bytes(count, rows, cols, dst_dtype == ZERO_F16);
    if ((rc = check_space(ws, ws_bytes, need, what)) != ZERO_OK) return rc;
    const int64_t from = (int64_t)elem_bytes(src_dtype);
    const bool same = src == dst && from == 2 && src_ld == dst_ld && (count == 1 || src_stride == dst_stride);
    if (!same && overlap(Place(src, rows, cols * from, src_ld * from, count, src_stride * from),
                         Place(dst, rows, cols * 2, dst_ld * 2, count, dst_stride * 2)))
        return fail(ZERO_EINVAL, "%s: the result overlaps the source, in another layout", what);
    auto with = [&](auto si, auto so) {
        constexpr int DTI = decltype(si)::value, DTO = decltype(so)::value;
        PlainIo<DTI, DTO> io{(const typename Elem<DTI>::type*)src, (typename Elem<DTO>::type*)dst,
                             src_ld, src_stride, dst_ld, dst_stride, (int)rows, (int)cols};
        return run_stack(io, count, *ns, nullptr, ws, (hipStream_t)stream, what);
    };
    auto to = [&](auto si) {
        return dst_dtype == ZERO_F16 ? with(si, std::integral_constant<int, ZERO_F16>())
                                     : with(si, std::integral_constant<int, ZERO_BF16>());
    };
    switch (src_dtype) {
        case ZERO_F16: return to(std::integral_constant<int, ZERO_F16>());
        case ZERO_BF16: return to(std::integral_constant<int, ZERO_BF16>());
        default: return to(std::integral_constant<int, ZERO_F32>());
    }
}

static int muon_step(float* master, float* mom, const float* g, int32_t count, int64_t rows, int64_t cols,
                     int64_t stride, const zero_muon_hparams* hp, const zero_ctrl* ctrl, void* gather,
                     int32_t gather_dtype, int64_t offset, void* ws, size_t ws_bytes, void* stream, bool exact,
                     const char* what) {
    int rc;
    if (hp == nullptr) return fail(ZERO_EINVAL, "%s: null hyperparameters", what);
    if ((rc = check_ns(&hp->ns, what)) != ZERO_OK) return rc;
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay) || !(hp->momentum >= 0.0f && hp->momentum < 1.0f))
        return fail(ZERO_EINVAL, "%s: lr, weight_decay or momentum out of range", what);
    if (hp->scale != ZERO_MUON_SCALE_SHAPE && hp->scale != ZERO_MUON_SCALE_RMS)
        return fail(ZERO_EINVAL, "%s: unknown scale %d", what, hp->scale);
    if (gather != nullptr && !valid_dtype(gather_dtype, false)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_stack(count, rows, cols, what)) != ZERO_OK) return rc;
    if (count == 0 || rows == 0 || cols == 0) return ok();
    if (master == nullptr || mom == nullptr || g == nullptr) return fail(ZERO_EINVAL, "%s: null matrices", what);
    if (!aligned(master, 4) || !aligned(mom, 4) || !aligned(g, 4) || (gather != nullptr && !aligned(gather, 2)) ||
        (ctrl != nullptr && !aligned(ctrl, 8)))
        return fail(ZERO_EALIGN, "%s: buffers not aligned to their elements", what);
    if (offset < 0) return fail(ZERO_ERANGE, "%s: negative offset", what);
    if (count > 1 && stride < rows * cols) return fail(ZERO_ERANGE, "%s: matrices overlap", what);
    if ((rc = check_space(ws, ws_bytes, workspace_bytes(count, rows, cols, exact), what)) != ZERO_OK) return rc;
    const int64_t size = rows * cols * 4, apart = stride * 4;
    const Place place[4] = {Place(master, 1, size, size, count, apart), Place(mom, 1, size, size, count, apart),
                            Place(g, 1, size, size, count, apart),
                            Place(gather == nullptr ? nullptr : (uint16_t*)gather + offset, 1, size / 2, size / 2, count, apart / 2)};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(place[i], place[j])) return fail(ZERO_EINVAL, "%s: master, mom, g or slot overlap", what);
    const double wide = (double)(rows > cols ? rows : cols);
    const double s = hp->scale == ZERO_MUON_SCALE_RMS ? 0.2 * std::sqrt(wide)
                                                      : std::sqrt(rows > cols ? (double)rows / (double)cols : 1.0);
    auto with = [&](auto so, auto parts) {
        constexpr int DTO = decltype(so)::value;
        MuonIo<DTO, decltype(parts)::value> io{master, mom, g, ctrl, gather == nullptr ? nullptr : (uint16_t*)gather + offset, stride,
                       (int)rows, (int)cols, hp->momentum, 1.0f - hp->momentum,
                       (float)((double)hp->lr * (double)hp->weight_decay), (float)((double)hp->lr * s),
                       hp->nesterov != 0};
        return run_stack(io, count, hp->ns, ctrl == nullptr ? nullptr : &ctrl->skip, ws, (hipStream_t)stream, what);
    };
    const bool two = exact && !narrow(rows, cols);
    auto to = [&](auto so) { return two ? with(so, std::true_type()) : with(so, std::false_type()); };
    return gather_dtype == ZERO_F16 ? to(std::integral_constant<int, ZERO_F16>())
                                    : to(std::integral_constant<int, ZERO_BF16>());
}

int zero_muon_step(float* master, float* mom, const float* g, int32_t count, int64_t rows, int64_t cols,
                   int64_t stride, const zero_muon_hparams* hp, const zero_ctrl* ctrl, void* gather,
                   int32_t gather_dtype, int64_t offset, void* ws, size_t ws_bytes, void* stream) {
    return muon_step(master, mom, g, count, rows, cols, stride, hp, ctrl, gather, gather_dtype, offset, ws, ws_bytes,
                     stream, false, "zero_muon_step");
}

int zero_muon_step_exact(float* master, float* mom, const float* g, int32_t count, int64_t rows, int64_t cols,
                         int64_t stride, const zero_muon_hparams* hp, const zero_ctrl* ctrl, void* gather,
                         int32_t gather_dtype, int64_t offset, void* ws, size_t ws_bytes, void* stream) {
    return muon_step(master, mom, g, count, rows, cols, stride, hp, ctrl, gather, gather_dtype, offset, ws, ws_bytes,
                     stream, true, "zero_muon_step_exact");
}

}  // extern "C"
