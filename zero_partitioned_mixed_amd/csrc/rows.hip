// Operators on rows of tokens: the root-mean-square norm with the residual's addition (its
// result in the inputs' type or as MXFP8) and its gradients, and dropout.
#include "mx_common.h"

namespace {

// ---------------------------------------------------------------- root-mean-square norm
//   h = x + residual, rounded to the residual's type;  y = h / sqrt(mean(h^2) + eps) * w
// A row's elements stay in registers between the sum of squares and their use, so that x and the
// residual are read and h and y written once.  Bound by memory: 8192 x 4096 bf16 with a residual 42 us for
// 268 MB (6.4 TB/s; a large copy reaches 5.1, writes alone 6.9), 4000 x 8192 to MXFP8 39 us for 230 MB.
// Up to two vectors of eight a lane, and as many lanes as the row needs: with four vectors the registers
// left four waves a SIMD, and 8192 columns took 66 us.  WHOLE: columns a multiple of eight, without the code for a
// row's last elements, whose registers cost the gradient 6 of 57 us.
constexpr int kMostThreads = 1024;
constexpr int64_t kWaveCols = 512;

// 1 / sqrt(mean + eps) = r * pre: squares that leave fp32's range, or that its smallest numbers
// would swallow, are summed again of elements times pre.  Up: a mean of squares below 2^-100 leaves sums below 2^124
// for up to 2^24 elements, and the square of the smallest number, 2^-149, becomes 2^-98.
constexpr float kPreDown = 0x1p-96f, kPreUp = 0x1p100f;
__device__ __forceinline__ float pre_of(float q) { return !(q <= 0x1p120f) ? kPreDown : q < 0x1p-100f ? kPreUp : 1.0f; }
// The results' elements take pre in two parts, h times the one and r times the other, so that those far below a
// large row's keep their bits: h 2^-96 would leave the normal numbers where h 2^-48 does not.
__device__ __forceinline__ float pre_of_h(float pre) { return pre == kPreDown ? 0x1p-48f : pre; }
__device__ __forceinline__ float pre_of_r(float pre) { return pre == kPreDown ? 0x1p-48f : 1.0f; }

// The lanes of a row: a wave (four rows a workgroup, for up to kWaveCols columns), or a workgroup
// of as many waves as the row needs with V vectors a lane.
template <bool WAVE>
struct RowOf {
    int64_t row;  // this row, or group of rows
    int t, lanes, wave = 0;  // wave: this row's in the workgroup
    __device__ __forceinline__ RowOf() {
        if constexpr (WAVE) {
            wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
            row = (int64_t)blockIdx.x * 4 + wave;
            t = threadIdx.x % 64;
            lanes = 64;
        } else {
            row = blockIdx.x;
            t = threadIdx.x;
            lanes = blockDim.x;
        }
    }
};

// The sums of N values over the lanes of a row, the same bits in every lane.  One barrier each:
// consecutive calls take turns with the places in LDS, of which there are sixteen, zeros where there
// is no wave: four vectors, where a loop over the waves waits for each place in turn.
constexpr int kMostWaves = kMostThreads / 64;
template <int N>
struct RowSums {
    f32x4 at[2][N][kMostWaves / 4];
    // before the first sums: the places without a wave
    __device__ __forceinline__ void clear() {
        if (threadIdx.x < kMostWaves && threadIdx.x >= blockDim.x / 64) {
            for (int i = 0; i < 2 * N; ++i) (&((float*)at)[i * kMostWaves])[threadIdx.x] = 0.0f;
        }
    }
};
template <bool WAVE, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], RowSums<N>& meet, int turn) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
    if constexpr (!WAVE) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) ((float*)meet.at[turn & 1][i])[threadIdx.x / 64] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f32x4 p[kMostWaves / 4];
#pragma unroll
            for (int w = 0; w < kMostWaves / 4; ++w) p[w] = meet.at[turn & 1][i][w];
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kMostWaves / 4; ++w) s += (p[w][0] + p[w][1]) + (p[w][2] + p[w][3]);
            v[i] = s;
        }
    }
}

// The sum of eight squares of h times pre, in pairs.
__device__ __forceinline__ float squares8(const float* h) {
    return ((h[0] * h[0] + h[1] * h[1]) + (h[2] * h[2] + h[3] * h[3])) +
           ((h[4] * h[4] + h[5] * h[5]) + (h[6] * h[6] + h[7] * h[7]));
}

// by / sqrt(q), by a power of two, as the sum of two fp32 numbers: results rounded to 8 bits next to a border, and the
// last bits of fp32 ones, show the rounding of one.
struct Root {
    float r, rest;
    __device__ __forceinline__ Root(float q, float by) {
        r = 1.0f / sqrtf(q);
        // one Newton step: r (1 - q r^2) / 2, q r^2 - 1 with its rounding undone by fused products
        const float p = q * r, e = fmaf(q, r, -p);
        const float one = fmaf(p, r, -1.0f) + e * r;
        rest = q > 0.0f && q < 3.0e38f ? -0.5f * r * one * by : 0.0f;
        r *= by;
    }
    // h by / sqrt(q) * w: h by / sqrt(q), which is of moderate size, in two parts too (h w alone may leave fp32's range).
    __device__ __forceinline__ float times(float h, float w) const {
        const float u = h * r, low = fmaf(h, r, -u) + h * rest;
        return fmaf(u, w, __builtin_isinf(w) ? 0.0f : low * w);
    }
};

struct NormArgs {
    const void *x, *residual, *w;
    int64_t ldx, ldr;
    int64_t tokens, cols;
    float eps;
    void *y, *h;
    int64_t ldy, ldh;
    uint8_t *codes, *scales;  // MX8
};

template <int DT>
__device__ __forceinline__ float rounded(float v) {
    return to_float<DT>(from_float<DT>(v));
}

// h of eight elements: from x, or from x and the residual, then also stored.
template <int DX, int DR, bool WHOLE>
__device__ __forceinline__ void sum8(const NormArgs& a, int64_t row, int64_t c, const Eight<DX>& ex, const Eight<DR>& er, float* h) {
    ex.floats(h);
    if (a.residual != nullptr) {
        float r[8];
        er.floats(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = rounded<DR>(h[i] + r[i]);
        put8<DR, WHOLE>((typename Elem<DR>::type*)a.h + row * a.ldh, c, a.cols, h);
    }
}

template <int DX, bool MX, bool WHOLE>
__device__ __forceinline__ void norm_out8(const NormArgs& a, int64_t row, int64_t c, const float* y) {
    if constexpr (MX) {
        const int64_t p = padded(a.cols);
        const uint32_t s = scale_byte8(block_top8(y));
        *(u32x2*)(a.codes + row * p + c) = codes8_e4m3(y, s);
        if ((threadIdx.x & 3) == 0) a.scales[row * (p / kMxBlock) + c / kMxBlock] = (uint8_t)s;
    } else {
        put8<DX, WHOLE>((typename Elem<DX>::type*)a.y + row * a.ldy, c, a.cols, y);
    }
}

template <int DX, int DR, bool WAVE, int V, bool MX, bool WHOLE>
__global__ void __launch_bounds__(WAVE ? 256 : kMostThreads) norm_kernel(NormArgs a) {
    typedef typename Elem<DX>::type X;
    typedef typename Elem<DR>::type R;
    __shared__ RowSums<1> meet;
    const RowOf<WAVE> of;
    if constexpr (!WAVE) meet.clear();
    const int64_t row = of.row;
    if (row >= a.tokens) return;  // whole waves; where a workgroup takes a row none
    const int t = of.t, T = of.lanes;
    const int64_t end = MX ? padded(a.cols) : a.cols;
    Eight<DX> ex[V], ew[V];
    Eight<DR> er[V];
    float h[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        if (c < a.cols) {
            ex[v].template fetch<WHOLE>((const X*)a.x + row * a.ldx, c, a.cols);
            if (a.residual != nullptr) er[v].template fetch<WHOLE>((const R*)a.residual + row * a.ldr, c, a.cols);
            ew[v].template fetch<WHOLE>((const X*)a.w, c, a.cols);
        }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        if (c < a.cols) {
            sum8<DX, DR, WHOLE>(a, row, c, ex[v], er[v], h[v]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = 0.0f;
        }
        ss[0] += squares8(h[v]);
    }
    const float n = (float)a.cols;
    row_sums<WAVE>(ss, meet, 0);
    float q = ss[0] / n + a.eps;
    const float pre = pre_of(q);
    if (pre != 1.0f) {
        ss[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = h[v][i] * pre;
                h[v][i] *= pre_of_h(pre);
            }
            ss[0] += squares8(p);
        }
        row_sums<WAVE>(ss, meet, 1);
        q = ss[0] / n + a.eps * pre * pre;
    }
    const Root root(q, pre_of_r(pre));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        if (c >= end) break;
        float w[8];
        if (MX && c >= a.cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0.0f;
        } else {
            ew[v].floats(w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[v][i] = root.times(h[v][i], w[i]);
            if (MX && c + i >= a.cols) h[v][i] = 0.0f;  // also where r is not finite
        }
        norm_out8<DX, MX, WHOLE>(a, row, c, h[v]);
    }
}

// Rows that registers do not hold: a workgroup reads each twice.
constexpr int kWide = 1024;
template <int DX, int DR, bool MX>
__global__ void __launch_bounds__(kWide) norm_wide_kernel(NormArgs a) {
    typedef typename Elem<DX>::type X;
    typedef typename Elem<DR>::type R;
    __shared__ RowSums<1> meet;
    const int64_t row = blockIdx.x, end = MX ? padded(a.cols) : a.cols;
    const int64_t c0 = (int64_t)threadIdx.x * 8;
    const X* const x = (const X*)a.x + row * a.ldx;
    const R* const hr = (const R*)a.h + row * a.ldh;  // what this lane wrote
    auto sum_of = [&](float pre, bool first) {
        float ss[1] = {0.0f};
        for (int64_t c = c0; c < a.cols; c += kWide * 8) {
            float h[8];
            if (first || a.residual == nullptr) {
                Eight<DX> ex;
                Eight<DR> er;
                ex.fetch(x, c, a.cols);
                if (a.residual != nullptr) er.fetch((const R*)a.residual + row * a.ldr, c, a.cols);
                sum8<DX, DR, false>(a, row, c, ex, er, h);
            } else {
                Eight<DR> eh;
                eh.fetch(hr, c, a.cols);
                eh.floats(h);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] *= pre;
            ss[0] += squares8(h);
        }
        row_sums<false>(ss, meet, first);
        return ss[0];
    };
    const float n = (float)a.cols;
    float q = sum_of(1.0f, true) / n + a.eps;
    const float pre = pre_of(q);
    if (pre != 1.0f) q = sum_of(pre, false) / n + a.eps * pre * pre;
    const Root root(q, pre_of_r(pre));
    const float of_h = pre_of_h(pre);
    for (int64_t c = c0; c < end; c += kWide * 8) {
        float h[8], w[8];
        if (c < a.cols) {
            if (a.residual == nullptr) {
                Eight<DX> ex;
                ex.fetch(x, c, a.cols);
                ex.floats(h);
            } else {
                Eight<DR> eh;
                eh.fetch(hr, c, a.cols);
                eh.floats(h);
            }
            Eight<DX> ew;
            ew.fetch((const X*)a.w, c, a.cols);
            ew.floats(w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = c + i < a.cols ? root.times(h[i] * of_h, w[i]) : 0.0f;
        norm_out8<DX, MX, false>(a, row, c, h);
    }
}

// The gradients.  With u = h / root, root = sqrt(mean(h^2) + eps), and g = dy w:
//   dh' = (g - u mean(g u)) / root + dh,  dw = sum over tokens of dy u
// dh' goes to the residual's gradient and, rounded to x's type, to x's.  root is computed again
// from h, which has to be read anyway: nothing but h is kept for the backward pass.
// A workgroup takes rows `groups` apart and holds its columns' part of dw in registers; the
// parts are summed in order by a second launch.  Bound by memory: 8192 x 4096 bf16 46 us for 276 MB
// and 4.5 us for dw.  The next row is read while this one's sums meet (without that, and two barriers a
// sum, 83 us).
constexpr int64_t kWaveGroups = 2048, kLeastGroups = 256;
struct NormGradArgs {
    const void *dy, *h, *w, *dh;
    int64_t lddy, ldh, lddh;
    int64_t tokens, cols;
    float eps;
    void *dx, *dr;
    int64_t lddx, lddr;
    float* parts;  // [groups][cols]
    void* dw;
    int groups;
};

// dh' and u of eight elements.
__device__ __forceinline__ void norm_grad8(const float* h, const float* y, const float* w, float r, float m, float* u, float* d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u[i] = h[i] * r;
        d[i] = (y[i] * w[i] - u[i] * m) * r + d[i];
    }
}

// The sums of squares and of g h over eight elements.
__device__ __forceinline__ void norm_sums8(const float* h, const float* y, const float* w, float (&s)[2]) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = y[i] * w[i] * h[i];
    s[0] += squares8(h);
    s[1] += ((g[0] + g[1]) + (g[2] + g[3])) + ((g[4] + g[5]) + (g[6] + g[7]));
}

// Whether fp32 holds a row's sums and what is made of them: its mean square q, and its sum of g h.
__device__ __forceinline__ bool norm_in_fp32(float q, float gh) {
    const float size = __builtin_fabsf(gh);
    return q >= 0x1p-60f && q <= 0x1p120f && size <= 0x1p90f && (size >= 0x1p-90f || size == 0.0f);
}

// The sum over a row's lanes in 64 bits, the same bits in every lane; consecutive calls take turns, as above.
typedef double RowSum64[2][kMostWaves];
template <bool WAVE>
__device__ __forceinline__ double row_sum64(double v, RowSum64& meet, int turn) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    if constexpr (!WAVE) {
        if ((threadIdx.x & 63) == 0) meet[turn][threadIdx.x / 64] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll 1
        for (uint32_t w = 0; w < blockDim.x / 64; ++w) v += meet[turn][w];
    }
    return v;
}

// Which of a group's rows are left for norm_grad_row64 when the others are done: a bit each, for the most rows in the
// fewest groups.  Among them it costs registers that every row pays for: 2048 x 16384 bf16 with an fp32 stream 148 us,
// behind them 128, without it 118.
template <bool WAVE>
struct LeftRows {
    static constexpr int kWords = (int)(kMaxSide / (WAVE ? kWaveGroups : kLeastGroups) / 32);
    uint32_t* bits;
    __device__ __forceinline__ LeftRows(uint32_t* all, int wave) : bits(all + (WAVE ? wave * kWords : 0)) {}
    __device__ __forceinline__ void meet() {
        if constexpr (WAVE) {
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            __builtin_amdgcn_wave_barrier();
        } else {
            __syncthreads();
        }
    }
    __device__ __forceinline__ void clear(int t, int T) {
        for (int i = t; i < kWords; i += T) bits[i] = 0;
        meet();
    }
    __device__ __forceinline__ void add(int t, int i) {
        if (t == 0) bits[i / 32] |= 1u << (i % 32);
    }
    __device__ __forceinline__ bool has(int i) const { return bits[i / 32] >> (i % 32) & 1; }
};

// The other rows (below 1e-9 or above 1e18, weights or gradients of such sizes, infinities and NaN): dr and dx
// in 64 bits, which hold every product and sum here, an element at a time, read again (8192 x 4096 bf16 of such rows
// alone 191 us, of others 44).  Leaves u = h by * r.
struct UnitOf {
    float by, r;
    __device__ __forceinline__ float operator()(float h) const { return h * by * r; }
};
template <int DX, int DR, bool WAVE>
__device__ __forceinline__ UnitOf norm_grad_row64(const NormGradArgs& a, int64_t row, int t, int T, RowSum64& meet) {
    typedef typename Elem<DX>::type X;
    typedef typename Elem<DR>::type R;
    const X *const dy = (const X*)a.dy + row * a.lddy, *const w = (const X*)a.w;
    const R *const h = (const R*)a.h + row * a.ldh, *const dh = (const R*)a.dh + row * a.lddh;
    const double n = (double)a.cols;
    double ss = 0.0, gu = 0.0;
#pragma unroll 1
    for (int64_t c = t; c < a.cols; c += T) {
        const double v = to_float<DR>(h[c]);
        ss += v * v;
    }
    const double q = row_sum64<WAVE>(ss, meet, 0) / n + a.eps, r = 1.0 / sqrt(q);
#pragma unroll 1
    for (int64_t c = t; c < a.cols; c += T) gu += (double)to_float<DX>(dy[c]) * to_float<DX>(w[c]) * (to_float<DR>(h[c]) * r);
    const double m = row_sum64<WAVE>(gu, meet, 1) / n;
#pragma unroll 1
    for (int64_t c = t; c < a.cols; c += T) {
        const double g = (double)to_float<DX>(dy[c]) * to_float<DX>(w[c]), u = to_float<DR>(h[c]) * r;
        const float d = (float)((g - u * m) * r + (a.dh != nullptr ? to_float<DR>(dh[c]) : 0.0f));
        if (a.dr != nullptr) ((R*)a.dr)[row * a.lddr + c] = from_float<DR>(d);
        if (a.dx != nullptr) ((X*)a.dx)[row * a.lddx + c] = from_float<DX>(d);
    }
    const float by = q > 0x1p120 ? 0x1p-48f : q < 0x1p-100 ? 0x1p100f : 1.0f;
    return UnitOf{by, (float)(r / by)};
}

template <int DX, int DR, bool WAVE, int V, bool WHOLE>
__global__ void __launch_bounds__(WAVE ? 256 : kMostThreads) norm_grad_kernel(NormGradArgs a) {
    typedef typename Elem<DX>::type X;
    typedef typename Elem<DR>::type R;
    __shared__ RowSums<2> meet;
    __shared__ RowSum64 meet64;
    __shared__ uint32_t left[WAVE ? 4 * LeftRows<WAVE>::kWords : LeftRows<WAVE>::kWords];
    const RowOf<WAVE> of;
    if constexpr (!WAVE) meet.clear();
    const int64_t group = of.row;
    const int t = of.t, T = of.lanes;
    const float n = (float)a.cols;
    struct Row {
        Eight<DX> y[V];
        Eight<DR> h[V], d[V];
        __device__ __forceinline__ void load(const NormGradArgs& a, int64_t row, int t, int T) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = (int64_t)(v * T + t) * 8;
                if (c >= a.cols) break;
                h[v].template fetch<WHOLE>((const R*)a.h + row * a.ldh, c, a.cols);
                y[v].template fetch<WHOLE>((const X*)a.dy + row * a.lddy, c, a.cols);
                if (a.dh != nullptr) d[v].template fetch<WHOLE>((const R*)a.dh + row * a.lddh, c, a.cols);
            }
        }
    };
    constexpr bool kAhead = V == 1;  // the next row is on its way while this one's sums meet; with V = 2 registers run out,
                                     // and the weights too are read again for each row
    Eight<DX> ew[V];
    auto weights = [&](int v, float* w) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        if (!kAhead) ew[v].template fetch<WHOLE>((const X*)a.w, c, a.cols);
        ew[v].floats(w);
    };
    float dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        if (kAhead && c < a.cols) ew[v].template fetch<WHOLE>((const X*)a.w, c, a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    Row next;
    if (kAhead && group < a.tokens) next.load(a, group, t, T);
    int turn = 0;
    bool any = false;  // the same in all lanes of a row
    LeftRows<WAVE> rest(left, of.wave);
    for (int64_t row = group; row < a.tokens; row += a.groups) {
        if (!kAhead) next.load(a, row, t, T);
        const Row e = next;
        if (kAhead && row + a.groups < a.tokens) next.load(a, row + a.groups, t, T);
        // f(v, c, h, y, w) for this lane's vectors
        auto each = [&](auto f) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = (int64_t)(v * T + t) * 8;
                if (c >= a.cols) break;
                float h[8], y[8], w[8];
                e.h[v].floats(h);
                e.y[v].floats(y);
                weights(v, w);
                f(v, c, h, y, w);
            }
        };
        float s[2] = {0.0f, 0.0f};
        each([&](int, int64_t, const float* h, const float* y, const float* w) { norm_sums8(h, y, w, s); });
        row_sums<WAVE>(s, meet, turn++);
        const float q = s[0] / n + a.eps;
        if (!norm_in_fp32(q, s[1])) {
            if (!any) rest.clear(t, T);
            any = true;
            rest.add(t, turn - 1);
            continue;
        }
        const float r = 1.0f / sqrtf(q), m = s[1] * r / n;
        each([&](int v, int64_t c, const float* h, const float* y, const float* w) {
            float u[8], d[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (a.dh != nullptr) e.d[v].floats(d);
            norm_grad8(h, y, w, r, m, u, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[v][i] += y[i] * u[i];
            if (a.dr != nullptr) put8<DR, WHOLE>((R*)a.dr + row * a.lddr, c, a.cols, d);
            if (a.dx != nullptr) put8<DX, WHOLE>((X*)a.dx + row * a.lddx, c, a.cols, d);
        });
    }
    if (any) {
        rest.meet();
        int64_t row = group;
        for (int k = 0; row < a.tokens; ++k, row += a.groups) {
            if (!rest.has(k)) continue;
            const UnitOf u = norm_grad_row64<DX, DR, WAVE>(a, row, t, T, meet64);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = (int64_t)(v * T + t) * 8;
                if (c >= a.cols) break;
                Eight<DX> ey;
                Eight<DR> eh;
                ey.template fetch<WHOLE>((const X*)a.dy + row * a.lddy, c, a.cols);
                eh.template fetch<WHOLE>((const R*)a.h + row * a.ldh, c, a.cols);
                float y[8], h[8];
                ey.floats(y);
                eh.floats(h);
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[v][i] += y[i] * u(h[i]);
            }
        }
    }
    if (a.parts == nullptr || group >= a.groups) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = (int64_t)(v * T + t) * 8;
        if (c < a.cols) put8<ZERO_F32, WHOLE>(a.parts + group * a.cols, c, a.cols, dw[v]);
    }
}

// Rows that registers do not hold: each read twice, the parts of dw kept in memory.
template <int DX, int DR>
__global__ void __launch_bounds__(kWide) norm_grad_wide_kernel(NormGradArgs a) {
    typedef typename Elem<DX>::type X;
    typedef typename Elem<DR>::type R;
    __shared__ RowSums<2> meet;
    __shared__ RowSum64 meet64;
    const int64_t c0 = (int64_t)threadIdx.x * 8;
    const float n = (float)a.cols;
    bool first = true;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.tokens; row += a.groups) {
        const X* const dy = (const X*)a.dy + row * a.lddy;
        const R* const hr = (const R*)a.h + row * a.ldh;
        // f(c, h, y, w) for this lane's vectors
        auto each = [&](auto f) {
            for (int64_t c = c0; c < a.cols; c += kWide * 8) {
                Eight<DX> ey, ew;
                Eight<DR> eh;
                eh.fetch(hr, c, a.cols);
                ey.fetch(dy, c, a.cols);
                ew.fetch((const X*)a.w, c, a.cols);
                float h[8], y[8], w[8];
                eh.floats(h);
                ey.floats(y);
                ew.floats(w);
                f(c, h, y, w);
            }
        };
        float* const part = a.parts == nullptr ? nullptr : a.parts + (int64_t)blockIdx.x * a.cols;
        auto add_part = [&](int64_t c, const float* y, const float* u) {
            if (part == nullptr) return;
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = (first || c + i >= a.cols ? 0.0f : part[c + i]) + y[i] * u[i];
            put8<ZERO_F32>(part, c, a.cols, p);
        };
        float s[2] = {0.0f, 0.0f};
        each([&](int64_t, const float* h, const float* y, const float* w) { norm_sums8(h, y, w, s); });
        row_sums<false>(s, meet, turn++);
        const float q = s[0] / n + a.eps;
        if (norm_in_fp32(q, s[1])) {
            const float r = 1.0f / sqrtf(q), m = s[1] * r / n;
            each([&](int64_t c, const float* h, const float* y, const float* w) {
                Eight<DR> ed;
                if (a.dh != nullptr)
                    ed.fetch((const R*)a.dh + row * a.lddh, c, a.cols);
                else
                    ed.zero();
                float u[8], d[8];
                ed.floats(d);
                norm_grad8(h, y, w, r, m, u, d);
                add_part(c, y, u);
                if (a.dr != nullptr) put8<DR>((R*)a.dr + row * a.lddr, c, a.cols, d);
                if (a.dx != nullptr) put8<DX>((X*)a.dx + row * a.lddx, c, a.cols, d);
            });
        } else {
            const UnitOf of = norm_grad_row64<DX, DR, false>(a, row, (int)threadIdx.x, kWide, meet64);
            each([&](int64_t c, const float* h, const float* y, const float*) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = of(h[i]);
                add_part(c, y, u);
            });
        }
        first = false;
    }
}

// dw: the groups' parts added in order, 16 columns a workgroup, 64 runs of groups.
template <int DX>
__global__ void __launch_bounds__(256) norm_dw_kernel(NormGradArgs a) {
    __shared__ float sums[64][17];
    const int lane = threadIdx.x % 4, run = threadIdx.x / 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + lane * 4;
    const int each = (a.groups + 63) / 64, to = (run + 1) * each < a.groups ? (run + 1) * each : a.groups;
    const bool whole = c + 4 <= a.cols && a.cols % 4 == 0;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int g = run * each; g < to; ++g) {
        const float* from = a.parts + g * a.cols + c;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        if (whole) {
            v = *(const f32x4*)from;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < a.cols) v[i] = from[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[run][lane * 4 + i] = s[i];
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x < 16 && col < a.cols) {
        float v = sums[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 64; ++k) v += sums[k][threadIdx.x];
        ((typename Elem<DX>::type*)a.dw)[col] = from_float<DX>(v);
    }
}

// ---------------------------------------------------------------- dropout
// y = x / (1 - p) or 0 (+ residual).  Which elements stay is computed, not stored: element c of
// row r takes sixteen bits of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011) at the counter (c / 8, r, offset), whose four words serve
// eight elements; it is dropped where they are below p 2^16.  The gradient is the same pass over dy.
// Sixteen bits an element keep the generator (20 wide products for eight elements) below what memory
// takes: 16384 x 8192 bf16 95 us for 537 MB, 140 with a residual for 805 MB.
struct DropArgs {
    const void *x, *residual;
    int64_t ldx, ldr, ldy;
    int64_t rows, cols;
    void* y;
    uint32_t key[2];
    uint64_t offset;
    const uint64_t* offset_dev;  // added to offset
    uint32_t limit;              // p 2^16
    float scale;
    uint32_t groups;             // of eight in a row
};

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)c[0] * 0xD2511F53u, q = (uint64_t)c[2] * 0xCD9E8D57u;
        c[0] = (uint32_t)(q >> 32) ^ c[1] ^ k0;
        c[1] = (uint32_t)q;
        c[2] = (uint32_t)(p >> 32) ^ c[3] ^ k1;
        c[3] = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

template <int DT>
__global__ void __launch_bounds__(256) dropout_kernel(DropArgs a) {
    typedef typename Elem<DT>::type T;
    const uint64_t offset = a.offset + (a.offset_dev != nullptr ? *a.offset_dev : 0);
    const uint64_t all = (uint64_t)a.rows * a.groups, step = (uint64_t)gridDim.x * 256;
    for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += step) {
        const uint64_t row = at >> 32 ? at / a.groups : (uint32_t)at / a.groups;
        const uint32_t group = (uint32_t)(at - row * a.groups);
        const int64_t c = (int64_t)group * 8;
        Eight<DT> ex, er;
        ex.fetch((const T*)a.x + row * a.ldx, c, a.cols);
        if (a.residual != nullptr) er.fetch((const T*)a.residual + row * a.ldr, c, a.cols);
        uint32_t w[4] = {group, (uint32_t)row, (uint32_t)offset, (uint32_t)(offset >> 32)};
        philox(w, a.key[0], a.key[1]);
        float x[8], r[8];
        ex.floats(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFF;
            x[i] = bits >= a.limit ? x[i] * a.scale : 0.0f;
        }
        if (a.residual != nullptr) {
            er.floats(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += r[i];
        }
        put8<DT>((T*)a.y + row * a.ldy, c, a.cols, x);
    }
}

// ---------------------------------------------------------------- host side
// f(x's type, residual's type) for the pairs in use.
template <class F>
int with_types(int32_t dx, int32_t dr, F f) {
    typedef std::integral_constant<int, ZERO_F16> H;
    typedef std::integral_constant<int, ZERO_BF16> B;
    typedef std::integral_constant<int, ZERO_F32> S;
    if (dx == ZERO_F16) return dr == ZERO_F32 ? f(H(), S()) : f(H(), H());
    if (dx == ZERO_BF16) return dr == ZERO_F32 ? f(B(), S()) : f(B(), B());
    return f(S(), S());
}

template <class F>
int with_type(int32_t dt, F f) {
    return with_types(dt, dt, [&](auto x, auto) { return f(x); });
}

// Threads for a row of n columns, v vectors each.
int threads_for(int64_t n, int v) { return (int)round_up(ceil_div(n, 8 * v), 64); }

template <int DX, int DR, bool MX, bool WHOLE>
int norm_with(const NormArgs& a, hipStream_t s, const char* what) {
    const int64_t n = MX ? padded(a.cols) : a.cols;
    const dim3 one((unsigned)a.tokens);
    if (n <= kWaveCols)
        return launch(norm_kernel<DX, DR, true, 1, MX, WHOLE>, dim3((unsigned)ceil_div(a.tokens, 4)), 256, s, a, what);
    if (n <= 2048) return launch(norm_kernel<DX, DR, false, 1, MX, WHOLE>, one, threads_for(n, 1), s, a, what);
    if (n <= 16 * kMostThreads) return launch(norm_kernel<DX, DR, false, 2, MX, WHOLE>, one, threads_for(n, 2), s, a, what);
    return launch(norm_wide_kernel<DX, DR, MX>, one, kWide, s, a, what);
}
template <bool MX>
int norm_any(const NormArgs& a, int32_t dx, int32_t dr, hipStream_t s, const char* what) {
    return with_types(dx, dr, [&](auto x, auto r) {
        if (a.cols % 8 == 0) return norm_with<decltype(x)::value, decltype(r)::value, MX, true>(a, s, what);
        return norm_with<decltype(x)::value, decltype(r)::value, MX, false>(a, s, what);
    });
}

// The checks shared by the norm's two forms.
int check_norm(const NormArgs& a, int32_t dx, int32_t dr, const char* what) {
    int rc;
    if (!valid_dtype(dx, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if (a.residual != nullptr && dr != dx && dr != ZERO_F32)
        return fail(ZERO_EINVAL, "%s: the residual has x's type or is fp32", what);
    if (!(a.eps >= 0.0f && a.eps <= 3.4028235e38f)) return fail(ZERO_EINVAL, "%s: eps is finite and not negative", what);
    if ((rc = check_sides(a.tokens, a.cols, what)) != ZERO_OK) return rc;
    if (a.ldx < a.cols || (a.residual != nullptr && (a.ldr < a.cols || a.ldh < a.cols)))
        return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (a.tokens == 0 || a.cols == 0) return ZERO_OK;
    if (a.x == nullptr || a.w == nullptr) return fail(ZERO_EINVAL, "%s: null input", what);
    if ((a.residual == nullptr) != (a.h == nullptr)) return fail(ZERO_EINVAL, "%s: a residual and its sum come together", what);
    if (!aligned(a.x, elem_bytes(dx)) || !aligned(a.w, elem_bytes(dx)) || !aligned(a.residual, elem_bytes(dr)) ||
        !aligned(a.h, elem_bytes(dr)))
        return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    if (a.residual != nullptr) {
        const Place h = values_at(a.h, dr, a.tokens, a.cols, a.ldh);
        const bool same = a.h == a.residual && a.ldh == a.ldr;  // the sum in the residual's place
        if (overlap(h, values_at(a.x, dx, a.tokens, a.cols, a.ldx)) || overlap(h, values_at(a.w, dx, 1, a.cols, a.cols)) ||
            (!same && overlap(h, values_at(a.residual, dr, a.tokens, a.cols, a.ldr))))
            return fail(ZERO_EINVAL, "%s: the sum overlaps an input", what);
    }
    return ZERO_OK;
}

// Groups of rows that a gradient call sums dw over: waves where a wave takes a row, else workgroups, as many
// as are at work at once.
int64_t grad_groups(int64_t tokens, int64_t cols) {
    const int64_t most = cols <= kWaveCols ? kWaveGroups : cols <= 2048 ? 1024 : cols <= 4096 ? 512 : kLeastGroups;
    return tokens < most ? tokens : most;
}

template <int DX, int DR, bool WHOLE>
int norm_grad_with(const NormGradArgs& a, hipStream_t s, const char* what) {
    const dim3 one((unsigned)a.groups);
    if (a.cols <= kWaveCols)
        return launch(norm_grad_kernel<DX, DR, true, 1, WHOLE>, dim3((unsigned)ceil_div(a.groups, 4)), 256, s, a, what);
    if (a.cols <= 8 * kMostThreads)
        return launch(norm_grad_kernel<DX, DR, false, 1, WHOLE>, one, threads_for(a.cols, 1), s, a, what);
    if (a.cols <= 16 * kMostThreads)
        return launch(norm_grad_kernel<DX, DR, false, 2, WHOLE>, one, threads_for(a.cols, 2), s, a, what);
    return launch(norm_grad_wide_kernel<DX, DR>, one, kWide, s, a, what);
}

}  // namespace

extern "C" {

int zero_rms_norm(const void* x, int32_t dtype, int64_t ldx, const void* residual, int32_t residual_dtype, int64_t ldr,
                  const void* w, int64_t tokens, int64_t cols, float eps, void* y, int64_t ldy, void* h, int64_t ldh,
                  void* stream) {
    const char* what = "zero_rms_norm";
    const int32_t dr = residual == nullptr ? dtype : residual_dtype;
    const NormArgs a{x, residual, w, ldx, ldr, tokens, cols, eps, y, h, ldy, ldh, nullptr, nullptr};
    int rc;
    if ((rc = check_norm(a, dtype, dr, what)) != ZERO_OK) return rc;
    if (ldy < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (tokens == 0 || cols == 0) return ok();
    if (y == nullptr) return fail(ZERO_EINVAL, "%s: null result", what);
    if (!aligned(y, elem_bytes(dtype))) return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    const Place to = values_at(y, dtype, tokens, cols, ldy);
    const bool same = y == x && ldy == ldx;  // the result in x's place
    if ((!same && overlap(to, values_at(x, dtype, tokens, cols, ldx))) || overlap(to, values_at(w, dtype, 1, cols, cols)) ||
        (residual != nullptr && overlap(to, values_at(residual, dr, tokens, cols, ldr))) ||
        (h != nullptr && overlap(to, values_at(h, dr, tokens, cols, ldh))))
        return fail(ZERO_EINVAL, "%s: the result overlaps an input or the sum", what);
    return norm_any<false>(a, dtype, dr, (hipStream_t)stream, what);
}

int zero_rms_norm_mx8(const void* x, int32_t dtype, int64_t ldx, const void* residual, int32_t residual_dtype, int64_t ldr,
                      const void* w, int64_t tokens, int64_t cols, float eps, void* codes, void* scales, void* h,
                      int64_t ldh, void* stream) {
    const char* what = "zero_rms_norm_mx8";
    const int32_t dr = residual == nullptr ? dtype : residual_dtype;
    const NormArgs a{x, residual, w, ldx, ldr, tokens, cols, eps, nullptr, h, 0, ldh, (uint8_t*)codes, (uint8_t*)scales};
    int rc;
    if ((rc = check_norm(a, dtype, dr, what)) != ZERO_OK) return rc;
    if (tokens == 0 || cols == 0) return ok();
    if (codes == nullptr || scales == nullptr) return fail(ZERO_EINVAL, "%s: null result", what);
    if (!aligned(codes, 16) || !aligned(scales, 16)) return fail(ZERO_EALIGN, "%s: codes or scales not 16-byte aligned", what);
    const Place to[2] = {codes8_at(codes, tokens, cols), scales_at(scales, tokens, cols)};
    for (const Place& p : to)
        if (overlap(p, values_at(x, dtype, tokens, cols, ldx)) || overlap(p, values_at(w, dtype, 1, cols, cols)) ||
            (residual != nullptr && (overlap(p, values_at(residual, dr, tokens, cols, ldr)) ||
                                     overlap(p, values_at(h, dr, tokens, cols, ldh)))))
            return fail(ZERO_EINVAL, "%s: codes or scales overlap an input or the sum", what);
    if (overlap(to[0], to[1])) return fail(ZERO_EINVAL, "%s: codes and scales overlap", what);
    return norm_any<true>(a, dtype, dr, (hipStream_t)stream, what);
}

size_t zero_rms_norm_grad_workspace_bytes(int64_t tokens, int64_t cols) {
    if (tokens <= 0 || cols <= 0 || tokens > kMaxSide || cols > kMaxSide) return 0;
    return (size_t)(grad_groups(tokens, cols) * cols * 4);
}

int zero_rms_norm_grad(const void* dy, int64_t lddy, const void* h, int32_t h_dtype, int64_t ldh, const void* w,
                       int32_t dtype, const void* dh, int64_t lddh, int64_t tokens, int64_t cols, float eps, void* dx,
                       int64_t lddx, void* dr, int64_t lddr, void* dw, void* ws, size_t ws_bytes, void* stream) {
    const char* what = "zero_rms_norm_grad";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if (h_dtype != dtype && h_dtype != ZERO_F32) return fail(ZERO_EINVAL, "%s: the sum has x's type or is fp32", what);
    if (!(eps >= 0.0f && eps <= 3.4028235e38f)) return fail(ZERO_EINVAL, "%s: eps is finite and not negative", what);
    if ((rc = check_sides(tokens, cols, what)) != ZERO_OK) return rc;
    if (lddy < cols || ldh < cols || (dh != nullptr && lddh < cols) || (dx != nullptr && lddx < cols) ||
        (dr != nullptr && lddr < cols))
        return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (cols == 0 || (dx == nullptr && dr == nullptr && dw == nullptr)) return ok();
    if (tokens > 0 && (dy == nullptr || h == nullptr || w == nullptr)) return fail(ZERO_EINVAL, "%s: null input", what);
    const size_t size = elem_bytes(dtype), size_h = elem_bytes(h_dtype);
    if (!aligned(dy, size) || !aligned(h, size_h) || !aligned(w, size) || !aligned(dh, size_h) || !aligned(dx, size) ||
        !aligned(dr, size_h) || !aligned(dw, size))
        return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    const Place from[4] = {values_at(dy, dtype, tokens, cols, lddy), values_at(h, h_dtype, tokens, cols, ldh),
                           values_at(dh, h_dtype, tokens, cols, lddh), values_at(w, dtype, 1, cols, cols)};
    const Place to[3] = {values_at(dx, dtype, tokens, cols, lddx), values_at(dr, h_dtype, tokens, cols, lddr),
                         values_at(dw, dtype, 1, cols, cols)};
    for (const Place& p : to)
        for (const Place& f : from)
            if (overlap(p, f)) return fail(ZERO_EINVAL, "%s: a gradient overlaps an input", what);
    if (meets(to[0], {to[1], to[2]}) || overlap(to[1], to[2])) return fail(ZERO_EINVAL, "%s: gradients overlap", what);
    NormGradArgs a{dy, h, w, dh, lddy, ldh, lddh, tokens, cols, eps, dx, dr, lddx, lddr, (float*)ws, dw,
                   (int)grad_groups(tokens, cols)};
    const hipStream_t s = (hipStream_t)stream;
    if (dw != nullptr) {
        const size_t need = zero_rms_norm_grad_workspace_bytes(tokens, cols);
        if (need > 0 && ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
        if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
        if (ws_bytes < need) return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
        if (need > 0 && meets(Place(ws, (int64_t)need), {from[0], from[1], from[2], from[3], to[0], to[1], to[2]}))
            return fail(ZERO_EINVAL, "%s: the workspace overlaps an input or a gradient", what);
    } else {
        a.parts = nullptr;
    }
    if (tokens > 0) {
        rc = with_types(dtype, h_dtype, [&](auto x, auto r) {
            if (cols % 8 == 0) return norm_grad_with<decltype(x)::value, decltype(r)::value, true>(a, s, what);
            return norm_grad_with<decltype(x)::value, decltype(r)::value, false>(a, s, what);
        });
        if (rc != ZERO_OK) return rc;
    }
    if (dw == nullptr) return ok();
    return with_type(dtype, [&](auto x) {
        return launch(norm_dw_kernel<decltype(x)::value>, dim3((unsigned)ceil_div(cols, 16)), 256, s, a, what);
    });
}

int zero_dropout(const void* x, int32_t dtype, int64_t ldx, const void* residual, int64_t ldr, int64_t rows, int64_t cols,
                 double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev, void* y, int64_t ldy, void* stream) {
    const char* what = "zero_dropout";
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if (!(p >= 0.0 && p <= 1.0)) return fail(ZERO_EINVAL, "%s: p is not in [0, 1]", what);
    // a counter has 32 bits for a row and 32 for a group of eight in it
    if (rows < 0 || cols < 0 || rows > (int64_t(1) << 32) || cols > (int64_t(1) << 34) ||
        (cols > 0 && rows > (int64_t(1) << 40) / cols))
        return fail(ZERO_ERANGE, "%s: %lld x %lld out of range", what, (long long)rows, (long long)cols);
    if (ldx < cols || ldy < cols || (residual != nullptr && ldr < cols))
        return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (rows == 0 || cols == 0) return ok();
    if (x == nullptr || y == nullptr) return fail(ZERO_EINVAL, "%s: null rows", what);
    if (!aligned(x, elem_bytes(dtype)) || !aligned(y, elem_bytes(dtype)) || !aligned(residual, elem_bytes(dtype)) ||
        !aligned(offset_dev, 8))
        return fail(ZERO_EALIGN, "%s: rows not aligned to their elements, or the offset not to 8 bytes", what);
    const Place to = values_at(y, dtype, rows, cols, ldy);
    if ((!(y == x && ldy == ldx) && overlap(to, values_at(x, dtype, rows, cols, ldx))) ||
        (residual != nullptr && !(y == residual && ldy == ldr) && overlap(to, values_at(residual, dtype, rows, cols, ldr))) ||
        overlap(to, Place(offset_dev, 8)))
        return fail(ZERO_EINVAL, "%s: the result overlaps an input", what);
    const uint32_t limit = (uint32_t)__builtin_rint(p * 65536.0);
    const DropArgs a{x, residual, ldx, ldr, ldy, rows, cols, y, {(uint32_t)seed, (uint32_t)(seed >> 32)}, offset, offset_dev,
                     limit, limit < 65536 ? (float)(65536.0 / (65536.0 - limit)) : 0.0f, (uint32_t)ceil_div(cols, 8)};
    const int64_t wgs = ceil_div(rows * ceil_div(cols, 8), 256);
    const dim3 grid((unsigned)(wgs < 65536 ? wgs : 65536));
    return with_type(dtype, [&](auto t) {
        return launch(dropout_kernel<decltype(t)::value>, grid, 256, (hipStream_t)stream, a, what);
    });
}

}  // extern "C"
