// Orthogonalised updates of whole matrices (Newton-Schulz), for gfx950.
//
// One step is three products on the smaller side m of an m x n matrix X:
//   S = X X^T,   M = a I + b S + c S^2,   X <- M X.
// Rounding.  The products take fp16 operands and sum in fp32 (the iteration
// in bf16 operands is off by 1e-2 to 3e-2, in plain fp16 by 1e-3 to 4e-3).  X itself
// stays in fp32 between steps, and the diagonals of S and M, which hold most of
// their weight, are kept in fp32 outside the fp16 operands:
//   S = D + E,  S^2 = E E + (d_i + d_j) e_ij + D^2,  X <- diag(M) X + (M - diag(M)) X.
// Only the off-diagonal parts and the product's copy of X are rounded to 11
// bits: 3e-4 to 9e-4 against 64 bits for spectra from flat to 1/k, up to 4e-3
// where every element rounds alike (constant matrices).
// fp16 holds powers of two times the values: X * 2^8, E * 2^12, M * a power that
// keeps |a| + 1.5 |b| + 2.25 |c| below 2^15; entries down to 1 / (65536 * 256)
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

struct Coeffs {
    float a, b, c, eps;
    float mscale;  // power of two of the fp16 M
};

// A stack in the workspace, on the wide side: m <= n, mp and np the row lengths
// (multiples of 64, the padding zero).
struct Work {
    int m, n, mp, np;
    int64_t stride;  // bytes from one matrix's block to the next
    char* base;
    int64_t x16, xt0, xt1, s16, m16, ds, dm, sums;  // byte offsets; X in fp32 at 0
    int parts;                                      // partial sums of squares per matrix
    const int32_t* skip;                            // != NULL and set: leave everything as it is
    __device__ char* of(int b) const { return base + (int64_t)b * stride; }
    __device__ bool skipped() const { return skip != nullptr && *skip != 0; }
};

// ---------------------------------------------------------------- where a stack comes from and goes to
// The matrices of zero_orthogonalize.
template <int DTI, int DTO>
struct PlainIo {
    static constexpr bool kInPlace = false;
    const typename Elem<DTI>::type* src;
    typename Elem<DTO>::type* dst;
    int64_t src_ld, src_stride, dst_ld, dst_stride;
    int rows, cols;

    __device__ float clip() const { return 1.0f; }
    // first reading of an element, and any later one
    __device__ float first(int b, int r, int c, float) const { return again(b, r, c, 1.0f); }
    __device__ float again(int b, int r, int c, float) const {
        return to_float<DTI>(src[b * src_stride + r * src_ld + c]);
    }
    __device__ void put(int b, int r, int c, float o) const {
        dst[b * dst_stride + r * dst_ld + c] = from_float<DTO>(o);
    }
};

// The matrices of zero_muon_step: the momentum is updated at the first reading.
template <int DTO>
struct MuonIo {
    static constexpr bool kInPlace = true;
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
    __device__ float first(int b, int r, int c, float clip) const {
        const int64_t i = b * stride + (int64_t)r * cols + c;
        const float gi = g[i] * clip, m = mu * mom[i] + one_mu * gi;
        mom[i] = m;
        return direction(gi, m);
    }
    __device__ float again(int b, int r, int c, float clip) const {
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
// A workgroup holds a strip of X in registers, in the layout of the matrix
// cores' results: blocks of T x T, each by a group of (T / 32)^2 waves with
// 32 x 32 elements per wave; G groups side by side and NB blocks after each other,
// so a strip is G * NB * T columns.  A matrix of one strip takes one
// launch for all its steps; a longer one takes, per step, one workgroup that
// makes M from the strips' parts of S, and one workgroup per strip that
// applies M and makes its part of the next S.
template <int T_, int G_, int NB_>
struct Strip {
    static constexpr int T = T_, G = G_, NB = NB_;
    static constexpr int TILES = T / 32, GROUP = TILES * TILES, WAVES = G * GROUP, THREADS = WAVES * 64;
    static constexpr int COLS = G * NB * T;
    static constexpr int ARRAY = T * T * 2;  // bytes of a T x T fp16 array
    static constexpr int SIZE = COLS * T;    // elements of a strip
};
typedef Strip<32, 8, 4> Strip32;
typedef Strip<64, 4, 2> Strip64;
typedef Strip<128, 1, 2> Strip128;

struct Pair {  // high part and rest, arrays in LDS
    char *hi, *lo;
};

template <int T>
__device__ __forceinline__ int small_at(int row, int col) {  // byte of an element of a swizzled T x T fp16 array
    constexpr int kPieces = T / 8;
    return row * T * 2 + (((col >> 3) ^ (row & (kPieces - 1))) << 4) + (col & 7) * 2;
}

template <int T>
__device__ __forceinline__ f16x8 small_frag(const char* a, int row, int kk, int h) {
    return *(const f16x8*)(a + small_at<T>(row, kk * 16 + h * 8));
}

// acc += A B^T of two pairs, the product of the two rests left out.
template <int T>
__device__ __forceinline__ void small_product(const Pair& A, const Pair& B, int i0, int j0, const Lane& L, f32x16& acc) {
#pragma unroll
    for (int kk = 0; kk < T / 16; ++kk) {
        const f16x8 ah = small_frag<T>(A.hi, i0 + L.c, kk, L.h), al = small_frag<T>(A.lo, i0 + L.c, kk, L.h);
        const f16x8 bh = small_frag<T>(B.hi, j0 + L.c, kk, L.h), bl = small_frag<T>(B.lo, j0 + L.c, kk, L.h);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, bh, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bl, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bh, acc, 0, 0, 0);
    }
}

// A wave's 32 x 32 elements into a pair; TURNED: into its transpose.
template <int T, bool TURNED>
__device__ __forceinline__ void small_store(const Pair& P, int i0, int j0, const Lane& L, const float* v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int i = i0 + 8 * q + 4 * L.h, j = j0 + L.c;
        f16x4 h, l;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            h[r] = (_Float16)v[4 * q + r];
            l[r] = (_Float16)(v[4 * q + r] - (float)h[r]);
        }
        if constexpr (TURNED) {
            *(f16x4*)(P.hi + small_at<T>(j, i)) = h;
            *(f16x4*)(P.lo + small_at<T>(j, i)) = l;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                *(_Float16*)(P.hi + small_at<T>(i + r, j)) = h[r];
                *(_Float16*)(P.lo + small_at<T>(i + r, j)) = l[r];
            }
        }
    }
}

// LDS of a strip's workgroup: a pair per group for its current block of X (or the
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
    static constexpr int T = P::T;
    Lane L;
    int group, i0, j0;  // this wave's group, and its tile's place in a block
    StripLds<P>& lds;
    Pair mine, square;

    __device__ StripWave(StripLds<P>& s) : lds(s) {
        group = L.wave / P::GROUP;
        i0 = L.wave % P::GROUP / P::TILES * 32;
        j0 = L.wave % P::TILES * 32;
        mine = {s.block + group * 2 * P::ARRAY, s.block + (group * 2 + 1) * P::ARRAY};
        square = {s.square, s.square + P::ARRAY};
    }
    __device__ int row(int r) const { return i0 + 8 * (r / 4) + 4 * L.h + r % 4; }
    __device__ int col(int b) const { return (b * P::G + group) * T + j0 + L.c; }  // within the strip

    // This wave's tile of S = X X^T of the strip's first nb blocks of every group.
    __device__ void gram(const float (&x)[P::NB][16], int nb, float (&s)[16]) {
        f32x16 acc;
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll
        for (int b = 0; b < P::NB; ++b) {
            if (b >= nb) break;
            __syncthreads();  // the block's last readers are done
            small_store<T, false>(mine, i0, j0, L, x[b]);
            __syncthreads();
            small_product<T>(mine, mine, i0, j0, L, acc);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = acc[r] * (1.0f / (kXScale * kXScale));
        if constexpr (P::G > 1) {
            float* parts = (float*)lds.block;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 16; ++r) parts[group * T * T + row(r) * T + j0 + L.c] = s[r];
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float v = 0.0f;
                for (int g = 0; g < P::G; ++g) v += parts[g * T * T + row(r) * T + j0 + L.c];
                s[r] = v;
            }
        }
    }

    // M from S, which every group holds: m[] this wave's tile off the diagonal
    // (times mscale), lds.dm the diagonal.
    __device__ void poly(const Coeffs& k, float (&s)[16], float (&m)[16]) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const bool diag = row(r) == j0 + L.c;
            if (diag && group == 0) lds.ds[row(r)] = s[r];
            s[r] = diag ? 0.0f : s[r];
            m[r] = s[r] * kSScale;
        }
        if (group == 0) small_store<T, true>(square, i0, j0, L, m);  // symmetric
        __syncthreads();
        f32x16 acc;
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
        small_product<T>(square, square, i0, j0, L, acc);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int i = row(r), j = j0 + L.c;
            const float di = lds.ds[i];
            float s2 = acc[r] * (1.0f / (kSScale * kSScale)) + s[r] * (di + lds.ds[j]);
            if (i == j) {
                s2 += di * di;
                if (group == 0) lds.dm[i] = k.a + k.b * di + k.c * s2;
            }
            m[r] = i == j ? 0.0f : (k.b * s[r] + k.c * s2) * k.mscale;
        }
        __syncthreads();  // the readers of S are done
    }

    // X <- M X; M's pair is written by the caller before, without a barrier.
    __device__ void apply(const Coeffs& k, int nb, float (&x)[P::NB][16]) {
        const float un = 1.0f / k.mscale;
#pragma unroll
        for (int b = 0; b < P::NB; ++b) {
            if (b >= nb) break;
            if (b > 0) __syncthreads();
            small_store<T, true>(mine, i0, j0, L, x[b]);
            __syncthreads();
            f32x16 acc;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
            small_product<T>(square, mine, i0, j0, L, acc);
#pragma unroll
            for (int r = 0; r < 16; ++r) x[b][r] = lds.dm[row(r)] * x[b][r] + acc[r] * un;
        }
    }
};

template <class IO>
struct StripArgs {
    IO io;
    Coeffs k;
    int steps;
    const int32_t* skip;
    // several strips a matrix:
    char* ws;
    int64_t stride;     // bytes from one matrix's workspace to the next
    int64_t parts, mat; // byte offsets of the strips' parts of S and of M; X at 0
    int64_t sums;
    int sum_parts, strips;
    int step;           // 0: normalise; k: apply the k-th M
};

// The whole iteration of a matrix of one strip.
template <class P, class IO>
__global__ void __launch_bounds__(P::THREADS) ns_strip_kernel(StripArgs<IO> a) {
    __shared__ StripLds<P> lds;
    if (a.skip != nullptr && *a.skip != 0) return;
    const IO& io = a.io;
    StripWave<P> w(lds);
    const int b = blockIdx.x;
    const bool tall = io.rows > io.cols;
    const int m = tall ? io.cols : io.rows, n = tall ? io.rows : io.cols;
    const int nb = (n + P::G * P::T - 1) / (P::G * P::T);
    const float clip = io.clip();
    float x[P::NB][16];
    double ss = 0.0;
#pragma unroll
    for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int i = w.row(r), j = w.col(bl);
            const float v = i < m && j < n ? io.first(b, tall ? j : i, tall ? i : j, clip) : 0.0f;
            ss += (double)v * (double)v;
            x[bl][r] = v;
        }
    const double scale = scale_of(sqrt(block_sum(ss, lds.red, P::WAVES)), a.k.eps);
#pragma unroll
    for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[bl][r] = (float)(x[bl][r] * scale);
    for (int step = 0; step < a.steps; ++step) {
        float s[16], mv[16];
        w.gram(x, nb, s);
        w.poly(a.k, s, mv);
        if (w.group == 0) small_store<P::T, true>(w.square, w.i0, w.j0, w.L, mv);
        w.apply(a.k, nb, x);
    }
#pragma unroll
    for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int i = w.row(r), j = w.col(bl);
            if (i < m && j < n) io.put(b, tall ? j : i, tall ? i : j, x[bl][r] * (1.0f / kXScale));
        }
}

// M of a matrix of several strips: fp32 [T][T] off the diagonal, then the diagonal.
template <class P, class IO>
__global__ void __launch_bounds__(P::GROUP * 64) ns_poly_kernel(StripArgs<IO> a) {
    typedef Strip<P::T, 1, 1> One;
    __shared__ StripLds<One> lds;
    if (a.skip != nullptr && *a.skip != 0) return;
    StripWave<One> w(lds);
    char* ws = a.ws + blockIdx.x * a.stride;
    const float* parts = (const float*)(ws + a.parts);
    float s[16], mv[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
    for (int p = 0; p < a.strips; ++p)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] += parts[(int64_t)p * P::T * P::T + w.row(r) * P::T + w.j0 + w.L.c];
    w.poly(a.k, s, mv);
    float* mat = (float*)(ws + a.mat);
#pragma unroll
    for (int r = 0; r < 16; ++r) mat[w.row(r) * P::T + w.j0 + w.L.c] = mv[r];
    if ((int)threadIdx.x < P::T) mat[P::T * P::T + threadIdx.x] = lds.dm[threadIdx.x];
}

// One strip: step 0 makes X; step k applies the k-th M; the last one writes the
// result, the others their X and part of S.
template <class P, class IO>
__global__ void __launch_bounds__(P::THREADS) ns_strips_kernel(StripArgs<IO> a) {
    __shared__ StripLds<P> lds;
    if (a.skip != nullptr && *a.skip != 0) return;
    const IO& io = a.io;
    StripWave<P> w(lds);
    const int b = blockIdx.y, strip = blockIdx.x, j0 = strip * P::COLS;
    const bool tall = io.rows > io.cols;
    const int m = tall ? io.cols : io.rows, n = tall ? io.rows : io.cols;
    const int left = n - j0 < P::COLS ? n - j0 : P::COLS, nb = (left + P::G * P::T - 1) / (P::G * P::T);
    char* ws = a.ws + b * a.stride;
    float* mine = (float*)ws + (int64_t)strip * P::SIZE + w.L.wave * 1024 + w.L.lane;
    float x[P::NB][16];
    if (a.step == 0) {
        double ss = 0.0;
        for (int p = threadIdx.x; p < a.sum_parts; p += P::THREADS) ss += ((const double*)(ws + a.sums))[p];
        const double scale = scale_of(sqrt(block_sum(ss, lds.red, P::WAVES)), a.k.eps);
        const float clip = io.clip();
#pragma unroll
        for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = w.row(r), j = j0 + w.col(bl);
                x[bl][r] = i < m && j < n ? (float)(io.again(b, tall ? j : i, tall ? i : j, clip) * scale) : 0.0f;
            }
    } else {
#pragma unroll
        for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[bl][r] = mine[bl * P::WAVES * 1024 + r * 64];
        const float* mat = (const float*)(ws + a.mat);
        if (w.group == 0) {
            float mv[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) mv[r] = mat[w.row(r) * P::T + w.j0 + w.L.c];
            small_store<P::T, true>(w.square, w.i0, w.j0, w.L, mv);
        }
        if ((int)threadIdx.x < P::T) lds.dm[threadIdx.x] = mat[P::T * P::T + threadIdx.x];
        w.apply(a.k, nb, x);
    }
    if (a.step == a.steps) {
#pragma unroll
        for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = w.row(r), j = j0 + w.col(bl);
                if (i < m && j < n) io.put(b, tall ? j : i, tall ? i : j, x[bl][r] * (1.0f / kXScale));
            }
        return;
    }
#pragma unroll
    for (int bl = 0; bl < P::NB; ++bl)
#pragma unroll
        for (int r = 0; r < 16; ++r) mine[bl * P::WAVES * 1024 + r * 64] = x[bl][r];
    float s[16];
    w.gram(x, nb, s);
    float* part = (float*)(ws + a.parts) + (int64_t)strip * P::T * P::T;
    if (w.group == 0) {
#pragma unroll
        for (int r = 0; r < 16; ++r) part[w.row(r) * P::T + w.j0 + w.L.c] = s[r];
    }
}

// ---------------------------------------------------------------- large matrices
constexpr int kSumThreads = 256;
constexpr int64_t kSumElems = 16384;  // elements per partial sum of squares, at least
constexpr int kMaxParts = 1024;

template <class IO>
struct IoArgs {
    IO io;
    Work w;
    float eps;
};

// One partial of the squared norm per workgroup (and the momentum update):
// rows blockIdx.x, + gridDim.x, ...
template <class IO>
__global__ void __launch_bounds__(kSumThreads) ns_sum_kernel(IoArgs<IO> a) {
    __shared__ double red[kSumThreads / 64];
    if (a.w.skipped()) return;
    const int b = blockIdx.y, cols = a.io.cols;
    const int64_t elems = (int64_t)a.io.rows * cols;
    const float clip = a.io.clip();
    const int64_t per = (elems + gridDim.x - 1) / gridDim.x;
    const int64_t e0 = blockIdx.x * per, e1 = e0 + per < elems ? e0 + per : elems;
    double ss = 0.0;
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kSumThreads) {
        const int r = (int)(e / cols), c = (int)(e - (int64_t)r * cols);
        const float v = a.io.first(b, r, c, clip);
        ss += (double)v * (double)v;
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
    for (int i = y; i < kPatch; i += 4) {
        const float v = tall ? patch[x][i] : patch[i][x];   // element (i0 + i, j0 + x) of X
        const float vt = tall ? patch[i][x] : patch[x][i];  // element (i0 + x, j0 + i) of X
        if (i0 + i < w.m && j0 + x < w.np) {
            x32[(int64_t)(i0 + i) * w.np + j0 + x] = v;
            x16[(int64_t)(i0 + i) * w.np + j0 + x] = (_Float16)v;
        }
        if (j0 + i < w.n && i0 + x < w.mp) xt[(int64_t)(j0 + i) * w.mp + i0 + x] = (_Float16)vt;
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
    int tiles_m, tiles_n;  // tile grid of the product
    int odd;               // which copy of X^T is current
    int last;              // the last step: only the fp32 X is wanted
};

// Upper triangle tile t -> (i <= j).
__device__ __forceinline__ void triangle_tile(int t, int& i, int& j) {
    j = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (j * (j + 1) / 2 > t) --j;
    while ((j + 1) * (j + 2) / 2 <= t) ++j;
    i = t - j * (j + 1) / 2;
}

// S (POLY false) or M (POLY true): tiles on and above the diagonal, mirrored.
template <class S, bool POLY>
__global__ void __launch_bounds__(S::THREADS) ns_square_kernel(StepArgs a) {
    __shared__ __attribute__((aligned(16))) char lds[S::LDS];
    const Work& w = a.w;
    if (w.skipped()) return;
    char* base = w.of(blockIdx.y);
    int ti, tj;
    triangle_tile(xcd_tile(blockIdx.x, gridDim.x), ti, tj);
    const int ld = POLY ? w.mp : w.np;  // elements
    const char* from = base + (POLY ? w.s16 : w.x16);
    const int i0 = ti * S::TILE, j0 = tj * S::TILE;
    const Operand A{from + (int64_t)i0 * ld * 2, (uint32_t)ld * 2, w.m - i0};
    const Operand B{from + (int64_t)j0 * ld * 2, (uint32_t)ld * 2, w.m - j0};
    f32x16 acc[S::MT][S::NT];
    MmF16 mm;
    tile_product<S>(A, B, ld / 64, false, mm, lds, acc);

    const Lane L;
    const int wm = L.wave / (S::TILE / S::WN), wn = L.wave % (S::TILE / S::WN);
    const Coeffs& k = a.k;
    float* diag = (float*)(base + (POLY ? w.dm : w.ds));
    const float* ds = (const float*)(base + w.ds);
    const _Float16* s16 = (const _Float16*)(base + w.s16);
    _Float16* out = (_Float16*)(base + (POLY ? w.m16 : w.s16));
#pragma unroll
    for (int ii = 0; ii < S::MT; ++ii)
#pragma unroll
        for (int jj = 0; jj < S::NT; ++jj) {
            const int j = j0 + wn * S::WN + jj * 32 + L.c;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int ib = i0 + wm * S::WM + ii * 32 + 8 * q + 4 * L.h;
                f16x4 h;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = ib + r;
                    float v = 0.0f;
                    if (i < w.m && j < w.m) {
                        if constexpr (POLY) {
                            const float di = ds[i];
                            const float e = (float)s16[(int64_t)i * w.mp + j] * (1.0f / kSScale);
                            float s2 = acc[ii][jj][4 * q + r] * (1.0f / (kSScale * kSScale)) + e * (di + ds[j]);
                            if (i == j) {
                                s2 += di * di;
                                diag[i] = k.a + k.b * di + k.c * s2;
                            } else {
                                v = (k.b * e + k.c * s2) * k.mscale;
                            }
                        } else {
                            v = acc[ii][jj][4 * q + r] * (1.0f / (kXScale * kXScale));
                            if (i == j) {
                                diag[i] = v;
                                v = 0.0f;
                            }
                            v *= kSScale;
                        }
                    }
                    h[r] = (_Float16)v;
                    if (i < w.m && j < w.mp) out[(int64_t)i * w.mp + j] = h[r];
                }
                if (ti != tj && j < w.m && ib < w.mp) *(f16x4*)(out + (int64_t)j * w.mp + ib) = h;
            }
        }
}

// X <- diag(M) X + (M - diag(M)) X, with its fp16 copies for the next step.
template <class S>
__global__ void __launch_bounds__(S::THREADS) ns_apply_kernel(StepArgs a) {
    __shared__ __attribute__((aligned(16))) char lds[S::LDS];
    const Work& w = a.w;
    if (w.skipped()) return;
    char* base = w.of(blockIdx.y);
    int ti, tj;
    band_tile(xcd_tile(blockIdx.x, gridDim.x), a.tiles_m, a.tiles_n, ti, tj);
    const int i0 = ti * S::TILE, j0 = tj * S::TILE;
    const char* xt = base + (a.odd ? w.xt1 : w.xt0);
    const Operand A{base + w.m16 + (int64_t)i0 * w.mp * 2, (uint32_t)w.mp * 2, w.m - i0};
    const Operand B{xt + (int64_t)j0 * w.mp * 2, (uint32_t)w.mp * 2, w.n - j0};
    f32x16 acc[S::MT][S::NT];
    MmF16 mm;
    tile_product<S>(A, B, w.mp / 64, false, mm, lds, acc);

    const Lane L;
    const int wm = L.wave / (S::TILE / S::WN), wn = L.wave % (S::TILE / S::WN);
    const float un = 1.0f / a.k.mscale;
    const float* dm = (const float*)(base + w.dm);
    float* x32 = (float*)base;
    _Float16 *x16 = (_Float16*)(base + w.x16), *next = (_Float16*)(base + (a.odd ? w.xt0 : w.xt1));
#pragma unroll
    for (int ii = 0; ii < S::MT; ++ii)
#pragma unroll
        for (int jj = 0; jj < S::NT; ++jj) {
            const int j = j0 + wn * S::WN + jj * 32 + L.c;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int ib = i0 + wm * S::WM + ii * 32 + 8 * q + 4 * L.h;
                f16x4 h;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = ib + r;
                    float v = 0.0f;
                    if (i < w.m && j < w.np) {
                        const int64_t at = (int64_t)i * w.np + j;
                        // columns from n on are zero: their X^T row repeats row n - 1
                        if (j < w.n) v = dm[i] * x32[at] + acc[ii][jj][4 * q + r] * un;
                        x32[at] = v;
                        if (!a.last) x16[at] = (_Float16)v;
                    }
                    h[r] = (_Float16)v;
                }
                if (!a.last && j < w.n && ib < w.mp) *(f16x4*)(next + (int64_t)j * w.mp + ib) = h;
            }
        }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kMaxSide = 65536;
constexpr int32_t kMaxCount = 65535;
constexpr int kNarrow = 128;  // smaller sides up to this take the strip kernels

typedef Shape<256, 128, 64> Big;
typedef Shape<128, 64, 64> Mid;
typedef Shape<64, 32, 32> Low;

bool narrow(int64_t rows, int64_t cols) { return rows <= kNarrow || cols <= kNarrow; }

int sum_parts(int64_t rows, int64_t cols) {
    const int64_t p = ceil_div(rows * cols, kSumElems);
    return (int)(p < kMaxParts ? p : kMaxParts);
}

// The workspace block of one matrix.
Work work_of(int64_t rows, int64_t cols) {
    Work w{};
    w.m = (int)(rows < cols ? rows : cols);
    w.n = (int)(rows < cols ? cols : rows);
    w.mp = (int)round_up(w.m, 64);
    w.np = (int)round_up(w.n, 64);
    w.parts = sum_parts(rows, cols);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    take((int64_t)w.m * w.np * 4);
    w.x16 = take((int64_t)w.m * w.np * 2);
    w.xt0 = take((int64_t)w.n * w.mp * 2);
    w.xt1 = take((int64_t)w.n * w.mp * 2);
    w.s16 = take((int64_t)w.m * w.mp * 2);
    w.m16 = take((int64_t)w.m * w.mp * 2);
    w.ds = take((int64_t)w.m * 4);
    w.dm = take((int64_t)w.m * 4);
    w.sums = take((int64_t)w.parts * 8);
    w.stride = at;
    return w;
}

// Strips of a narrow matrix: f(Strip32(), count of strips) and so on.
template <class F>
auto with_strip(int64_t rows, int64_t cols, F f) {
    const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    if (m <= 32) return f(Strip32(), (int)ceil_div(n, Strip32::COLS));
    if (m <= 64) return f(Strip64(), (int)ceil_div(n, Strip64::COLS));
    return f(Strip128(), (int)ceil_div(n, Strip128::COLS));
}

// Workspace of one narrow matrix of several strips: X, the parts of S, M, the sums.
struct StripWork {
    int64_t parts, mat, sums, stride;
};

template <class P>
StripWork strip_work(int strips, int sum_parts) {
    StripWork w;
    w.parts = round_up((int64_t)strips * P::SIZE * 4, 256);
    w.mat = w.parts + round_up((int64_t)strips * P::T * P::T * 4, 256);
    w.sums = w.mat + round_up((P::T * P::T + P::T) * 4, 256);
    w.stride = w.sums + round_up((int64_t)sum_parts * 8, 256);
    return w;
}

int check_ns(const zero_newton_schulz* ns, const char* what) {
    if (ns == nullptr) return fail(ZERO_EINVAL, "%s: null settings", what);
    if (!std::isfinite(ns->a) || !std::isfinite(ns->b) || !std::isfinite(ns->c))
        return fail(ZERO_EINVAL, "%s: coefficients must be finite", what);
    if (!std::isfinite(ns->eps) || ns->eps < 0.0f) return fail(ZERO_EINVAL, "%s: eps must be >= 0", what);
    if (ns->steps < 0 || ns->steps > 64) return fail(ZERO_EINVAL, "%s: steps must be 0..64", what);
    return ZERO_OK;
}

int check_stack(int32_t count, int64_t rows, int64_t cols, const char* what) {
    if (count < 0 || count > kMaxCount) return fail(ZERO_ERANGE, "%s: count %d out of range", what, count);
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return fail(ZERO_ERANGE, "%s: %lld x %lld out of range (at most %lld each way)", what, (long long)rows,
                    (long long)cols, (long long)kMaxSide);
    return ZERO_OK;
}

int check_space(const void* ws, size_t ws_bytes, int32_t count, int64_t rows, int64_t cols, const char* what) {
    const size_t need = zero_ns_workspace_bytes(count, rows, cols);
    if (need == 0) return ZERO_OK;
    if (ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
    if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
    if (ws_bytes < need)
        return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
    return ZERO_OK;
}

Coeffs coeffs_of(const zero_newton_schulz& ns) {
    Coeffs k{ns.a, ns.b, ns.c, ns.eps, 0.0f};
    const double top = std::fabs((double)ns.a) + 1.5 * std::fabs((double)ns.b) + 2.25 * std::fabs((double)ns.c);
    int e = 0;
    std::frexp(top, &e);  // top < 2^e
    e = 15 - e;
    k.mscale = (float)std::ldexp(1.0, e > 15 ? 15 : e < -100 ? -100 : e);
    return k;
}

template <class S>
int steps_with(const Work& w, const Coeffs& k, int32_t count, int steps, hipStream_t s, const char* what) {
    int rc = ZERO_OK;
    const int tm = (int)ceil_div(w.m, S::TILE), tn = (int)ceil_div(w.np, S::TILE);
    StepArgs a{w, k, tm, tn, 0, 0};
    const dim3 square((unsigned)(tm * (tm + 1) / 2), (unsigned)count), whole((unsigned)(tm * tn), (unsigned)count);
    for (int i = 0; i < steps; ++i) {
        a.odd = i & 1;
        a.last = i + 1 == steps;
        if ((rc = launch(ns_square_kernel<S, false>, square, S::THREADS, s, a, what)) != ZERO_OK) return rc;
        if ((rc = launch(ns_square_kernel<S, true>, square, S::THREADS, s, a, what)) != ZERO_OK) return rc;
        if ((rc = launch(ns_apply_kernel<S>, whole, S::THREADS, s, a, what)) != ZERO_OK) return rc;
    }
    return rc;
}

// Tiles of a stack's symmetric products at a tile side.
int64_t square_tiles(const Work& w, int32_t count, int tile) {
    const int64_t t = ceil_div(w.m, tile);
    return count * (t * (t + 1) / 2);
}

template <class IO>
int run_strips(const IO& io, int32_t count, const zero_newton_schulz& ns, const Coeffs& k, const int32_t* skip,
               void* ws, hipStream_t s, const char* what) {
    return with_strip(io.rows, io.cols, [&](auto shape, int strips) {
        typedef decltype(shape) P;
        StripArgs<IO> a{io, k, ns.steps, skip, (char*)ws, 0, 0, 0, 0, 0, strips, 0};
        const dim3 each((unsigned)count);
        if (strips == 1) return launch(ns_strip_kernel<P, IO>, each, P::THREADS, s, a, what);
        a.sum_parts = sum_parts(io.rows, io.cols);
        const StripWork w = strip_work<P>(strips, a.sum_parts);
        a.parts = w.parts;
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
            if (a.step > 0) rc = launch(ns_poly_kernel<P, IO>, each, P::GROUP * 64, s, a, what);
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
    if (narrow(io.rows, io.cols)) return run_strips(io, count, ns, k, skip, ws, s, what);
    Work w = work_of(io.rows, io.cols);
    w.base = (char*)ws;
    w.skip = skip;
    const IoArgs<IO> a{io, w, ns.eps};
    if ((rc = launch(ns_sum_kernel<IO>, dim3((unsigned)w.parts, (unsigned)count), kSumThreads, s, a, what)) != ZERO_OK)
        return rc;
    // patches cover the padding of both orientations
    const dim3 patches((unsigned)ceil_div(io.cols, kPatch), (unsigned)ceil_div(io.rows, kPatch), (unsigned)count);
    if ((rc = launch(ns_begin_kernel<IO>, patches, 256, s, a, what)) != ZERO_OK) return rc;
    if (square_tiles(w, count, 256) >= 256)
        rc = steps_with<Big>(w, k, count, ns.steps, s, what);
    else if (square_tiles(w, count, 128) >= 256)
        rc = steps_with<Mid>(w, k, count, ns.steps, s, what);
    else
        rc = steps_with<Low>(w, k, count, ns.steps, s, what);
    if (rc != ZERO_OK) return rc;
    return launch(ns_end_kernel<IO>, patches, 256, s, a, what);
}

}  // namespace

extern "C" {

size_t zero_ns_workspace_bytes(int32_t count, int64_t rows, int64_t cols) {
    if (count <= 0 || count > kMaxCount || rows <= 0 || cols <= 0 || rows > kMaxSide || cols > kMaxSide) return 0;
    if (narrow(rows, cols))
        return with_strip(rows, cols, [&](auto shape, int strips) -> size_t {
            if (strips == 1) return 0;
            return (size_t)strip_work<decltype(shape)>(strips, sum_parts(rows, cols)).stride * (size_t)count;
        });
    return (size_t)work_of(rows, cols).stride * (size_t)count;
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
    if ((rc = check_space(ws, ws_bytes, count, rows, cols, what)) != ZERO_OK) return rc;
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

int zero_muon_step(float* master, float* mom, const float* g, int32_t count, int64_t rows, int64_t cols,
                   int64_t stride, const zero_muon_hparams* hp, const zero_ctrl* ctrl, void* gather,
                   int32_t gather_dtype, int64_t offset, void* ws, size_t ws_bytes, void* stream) {
    const char* what = "zero_muon_step";
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
    if ((rc = check_space(ws, ws_bytes, count, rows, cols, what)) != ZERO_OK) return rc;
    const double wide = (double)(rows > cols ? rows : cols);
    const double s = hp->scale == ZERO_MUON_SCALE_RMS ? 0.2 * std::sqrt(wide)
                                                      : std::sqrt(rows > cols ? (double)rows / (double)cols : 1.0);
    auto with = [&](auto so) {
        constexpr int DTO = decltype(so)::value;
        MuonIo<DTO> io{master, mom, g, ctrl, gather == nullptr ? nullptr : (uint16_t*)gather + offset, stride,
                       (int)rows, (int)cols, hp->momentum, 1.0f - hp->momentum,
                       (float)((double)hp->lr * (double)hp->weight_decay), (float)((double)hp->lr * s),
                       hp->nesterov != 0};
        return run_stack(io, count, hp->ns, ctrl == nullptr ? nullptr : &ctrl->skip, ws, (hipStream_t)stream, what);
    };
    return gather_dtype == ZERO_F16 ? with(std::integral_constant<int, ZERO_F16>())
                                    : with(std::integral_constant<int, ZERO_BF16>());
}

}  // extern "C"
