// Shared by the matrix kernels (newton_schulz.hip, mx4.hip): 16-bit formats,
// the tiled product on the matrix cores, launches and argument checks.
//
// The product.  A workgroup computes a TILE x TILE tile of A B^T, both
// operands stored row-major along k, from "slabs" of 128 bytes of every row
// (64 fp16 or 256 4-bit elements).  A slab of both operands is copied to LDS by
// direct global-to-LDS loads of 16 bytes per lane, one to three slabs ahead of the
// one that feeds the matrix cores: one barrier per slab.  Within a slab a k step's
// fragments are read while the one before multiplies, and a quarter of the next
// loads goes out with each k step: issued together they hold up their wave for as
// long as the memory pipeline takes them (4096^3, fp16: 900 TFLOP/s with neither,
// 1050 with both, 1110 with the shapes below; the library's product 1220 at 8192^3).  A fragment of
// the 32x32 matrix instructions is 16 bytes per lane, so fp16 (k = 16) and
// 4-bit (k = 64) operands move alike and share this code; which 16-byte
// pieces of a slab meet in one instruction does not matter as long as both
// operands agree, and lane group h takes pieces 4h..4h+3 (for the 4-bit
// operands its four block scales are then one dword).  Direct loads write LDS
// in lane order, so the bank swizzle is put into the addresses they read:
// piece q of row r sits in slot q ^ (r / 2 mod 8) (16 lanes then read all 64 banks;
// q ^ (r mod 8) measured 1-3% slower).
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

// A tile of TILE x TILE outputs by waves of WM x WN outputs each, with STAGES slabs
// in LDS: STAGES - 1 on their way while one is used.  KS such groups of waves take
// the slabs in turn, each with its own slabs in LDS, and add their sums at the
// end: for tiles that have a CU to themselves (1024 x 1024 x 4096, fp16: 16 us, with
// one group 21).
template <int TILE_, int WM_, int WN_, int STAGES_, int KS_ = 1>
struct Shape {
    static constexpr int TILE = TILE_, WM = WM_, WN = WN_, STAGES = STAGES_, KS = KS_;
    static constexpr int WAVES = (TILE / WM) * (TILE / WN);  // of a group
    static constexpr int THREADS = KS * WAVES * 64;
    static constexpr int MT = WM / 32, NT = WN / 32;
    static constexpr int LOADS = 2 * TILE / 8 / WAVES;    // direct loads (8 rows each) per wave and slab
    static constexpr int SCALES = 4 * TILE / 64 / WAVES;  // direct loads of block scales, 4-bit operands
    static constexpr int ROWS = 2 * TILE * kSlab;         // bytes of a slab of both operands
    static_assert((TILE / 8) % LOADS == 0 && (4 * TILE / 64) % WAVES == 0, "whole loads per wave");
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
    __device__ explicit Lane(int of) : Lane() { wave %= of; }  // wave within a group of `of`
};

// Bytes straight to LDS: lane l's 16 (or 4) go to `to` + 16 l (or 4 l).
typedef const __attribute__((address_space(1))) void* GlobalPtr;
typedef __attribute__((address_space(3))) void* LdsPtr;
__device__ __forceinline__ void load_to_lds16(const char* from, char* to) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 16, 0, 0);
}
__device__ __forceinline__ void load_to_lds4(const char* from, char* to) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)to, 4, 0, 0);
}

// Until at most N of this wave's loads are on their way and its LDS reads are
// done; then all waves of the workgroup.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// fp16 operands: four k = 16 instructions a slab.
struct MmF16 {
    static constexpr bool kScaled = false;
    template <int KK>
    static __device__ __forceinline__ f32x16 mma(const i32x4& a, const i32x4& b, f32x16 c, uint32_t, uint32_t) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                      c, 0, 0, 0);
    }
};

// 4-bit operands under block scales: four k = 64 instructions a slab.  The scales
// of a row's eight blocks go to LDS as two dwords, one per lane group.
struct MmFp4 {
    static constexpr bool kScaled = true;
    template <int KK>
    static __device__ __forceinline__ f32x16 mma(const i32x4& a, const i32x4& b, f32x16 c, uint32_t sa, uint32_t sb) {
        const i32x8 u = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8 v = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(u, v, c, 4, 4, KK, (int)sa, KK, (int)sb);
    }
};

// Bytes of LDS of a product.
template <class S, class MM>
constexpr int product_lds() {
    return S::KS * S::STAGES * (S::ROWS + (MM::kScaled ? 4 * S::TILE * 4 : 0));
}

// One k step's fragments of a wave's rows and columns.
template <class S>
struct Frags {
    i32x4 a[S::MT], b[S::NT];
    __device__ __forceinline__ void load(const char* ra, const char* rb, int at) {
#pragma unroll
        for (int i = 0; i < S::MT; ++i) a[i] = *(const i32x4*)(ra + i * 32 * kSlab + at);
#pragma unroll
        for (int j = 0; j < S::NT; ++j) b[j] = *(const i32x4*)(rb + j * 32 * kSlab + at);
    }
};

template <class S, class MM, int KK>
__device__ __forceinline__ void multiply(f32x16 (&acc)[S::MT][S::NT], const Frags<S>& f,
                                         const uint32_t (&sa)[S::MT], const uint32_t (&sb)[S::NT]) {
#pragma unroll
    for (int i = 0; i < S::MT; ++i)
#pragma unroll
        for (int j = 0; j < S::NT; ++j) acc[i][j] = MM::template mma<KK>(f.a[i], f.b[j], acc[i][j], sa[i], sb[j]);
}

// The product of one tile after another.  A tile is `slabs` whole slabs and then
// (4-bit operands) half a slab if `half`.  PARTS = 2: rows hold `slabs` slabs of rests
// and right behind them the high parts that left them; the product is rest x high +
// high x rest + high x high, three times the slabs, the small terms first: a matrix
// instruction cuts each term to the sum's last bits.
//   Product<S, MM> p(lds, slabs, half);
//   p.tile(A, B, SA, SB);  its operands, SA and SB their scales' rows (4-bit)
//   p.ahead();             its first loads: LDS has no readers any more
//   p.run(acc);            acc = the wave's part of the tile
// Element r of acc[i][j] is output row wm * WM + 32 i + 8 (r / 4) + 4 h + r % 4, column
// wn * WN + 32 j + c.  run() is true for the waves that hold the result (the first
// group); LDS (product_lds bytes) is free once all waves have met after it.
template <class S, class MM, int PARTS = 1>
struct Product {
    static_assert(PARTS == 1 || (PARTS == 2 && !MM::kScaled), "two parts of fp16 operands");
    static constexpr int kScaleLoads = MM::kScaled ? S::SCALES : 0;
    static constexpr int kStage = S::ROWS + (MM::kScaled ? 4 * S::TILE * 4 : 0);
    const Lane L;
    const int group, slabs, total;
    const int part, first_part, edge;  // PARTS = 2: slabs of a part; where this wave's operand starts, up to which slab
    const bool half;
    char *const all, *const lds;  // the workgroup's LDS, the group's part of it
    const char* base;             // this wave's operand
    uint32_t off[S::LOADS];
    const char* scale_base[kScaleLoads + 1];
    uint32_t scale_off[kScaleLoads + 1];

    __device__ __forceinline__ Product(char* shared, int slabs_, bool half_)
        : L(S::WAVES),
          group(S::KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (S::WAVES * 64))),
          slabs(PARTS == 2 ? 3 * slabs_ : slabs_),
          total(slabs + (MM::kScaled && half_ ? 1 : 0)),
          part(slabs_),
          first_part(first_load() < S::TILE / 8 ? 0 : slabs_),
          edge(2 * slabs_ - first_part),
          half(half_),
          all(shared),
          lds(shared + group * S::STAGES * kStage) {}

    // This wave's direct loads: groups of 8 rows, all of one operand.
    __device__ __forceinline__ int first_load() const { return L.wave * S::LOADS; }
    __device__ __forceinline__ int row_of(int i) const {
        const int g0 = first_load();
        return (g0 < S::TILE / 8 ? g0 : g0 - S::TILE / 8) * 8 + (L.lane >> 3) + i * 8;
    }
    __device__ __forceinline__ uint32_t piece_of(int i) const { return (L.lane & 7) ^ ((row_of(i) >> 1) & 7); }
    // And of scales: dword h * 2 TILE + row of the two operands' rows.
    __device__ __forceinline__ int scale_first(int i) const { return (L.wave * S::SCALES + i) * 64; }

    __device__ __forceinline__ void tile(const Operand& A, const Operand& B, const Operand& SA, const Operand& SB) {
        const Operand& O = first_load() < S::TILE / 8 ? A : B;
        base = O.base;
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i) {
            const int row = row_of(i);
            off[i] = (uint32_t)(row < O.rows - 1 ? row : O.rows - 1) * O.ld + piece_of(i) * 16;
        }
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) {
            const int r = scale_first(i) % (2 * S::TILE);
            const Operand& C = r < S::TILE ? SA : SB;
            const int row = (r < S::TILE ? r : r - S::TILE) + L.lane;
            scale_base[i] = C.base;
            scale_off[i] = (uint32_t)(row < C.rows - 1 ? row : C.rows - 1) * C.ld;
        }
    }

    // quarter q of the loads of a slab (q = 4: all)
    __device__ __forceinline__ void stage(int slab, char* buf, int q) const {
        const bool cut = MM::kScaled && slab >= slabs;  // past a half slab lies the next row
        // A's parts in the order rest, high, high; B's high, rest, high
        const char* from = base + (int64_t)(PARTS == 1 ? slab : slab < edge ? slab + first_part : slab - part) * kSlab;
        char* to = buf + first_load() * 1024;
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i)
            if (q == 4 || i * 4 / S::LOADS == q)
                load_to_lds16(from + (off[i] - (cut && piece_of(i) >= 4 ? 64u : 0u)), to + i * 1024);
        if (q >= 3) {
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i)
                load_to_lds4(scale_base[i] + (int64_t)slab * 8 +
                                 (scale_off[i] + (cut ? 0 : scale_first(i) / (2 * S::TILE) * 4)),
                             buf + S::ROWS + (L.wave * S::SCALES + i) * 256);
        }
    }

    __device__ __forceinline__ int slab_of(int t) const { return t * S::KS + group; }  // round t of this group

    __device__ __forceinline__ void ahead() const {
#pragma unroll
        for (int t = 0; t < S::STAGES - 1; ++t)
            if (slab_of(t) < total) stage(slab_of(t), lds + t * kStage, 4);
    }

    __device__ __forceinline__ void scales(const char* buf, int shift, uint32_t (&sa)[S::MT], uint32_t (&sb)[S::NT]) const {
        if constexpr (MM::kScaled) {
            const int wm = L.wave / (S::TILE / S::WN), wn = L.wave % (S::TILE / S::WN);
            const uint32_t* at = (const uint32_t*)(buf + S::ROWS) + L.h * 2 * S::TILE + L.c;
#pragma unroll
            for (int i = 0; i < S::MT; ++i) sa[i] = at[wm * S::WM + 32 * i] >> shift;
#pragma unroll
            for (int j = 0; j < S::NT; ++j) sb[j] = at[S::TILE + wn * S::WN + 32 * j] >> shift;
        }
    }

    __device__ __forceinline__ bool run(f32x16 (&acc)[S::MT][S::NT]) const {
        const int wm = L.wave / (S::TILE / S::WN), wn = L.wave % (S::TILE / S::WN);
#pragma unroll
        for (int i = 0; i < S::MT; ++i)
#pragma unroll
            for (int j = 0; j < S::NT; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        const int fa = (wm * S::WM + L.c) * kSlab, fb = (S::TILE + wn * S::WN + L.c) * kSlab;
        const int turn = (L.c >> 1) & 7;
        const int rounds = (slabs + S::KS - 1) / S::KS;
        char* const end = lds + S::STAGES * kStage;
        char *buf = lds, *fill = lds + (S::STAGES - 1) * kStage;
        auto after = [&](char* b) { return b + kStage == end ? lds : b + kStage; };
        for (int t = 0; t < rounds; ++t) {
            // this round's slab has landed in every wave's part, and the buffer used before it is free
            if (slab_of(t + S::STAGES - 2) < total)
                wait_and_meet<(S::STAGES - 2) * (S::LOADS + kScaleLoads)>();
            else
                wait_and_meet<0>();
            const int slab = slab_of(t), next = slab_of(t + S::STAGES - 1);
            const bool more = next < total;
            if (S::KS == 1 || slab < slabs) {
                uint32_t sa[S::MT], sb[S::NT];
                scales(buf, 0, sa, sb);
                const char *ra = buf + fa, *rb = buf + fb;
                const int slot = (4 * L.h) ^ turn;
                Frags<S> f[2];
                f[0].load(ra, rb, (slot ^ 0) << 4);
                if (more) stage(next, fill, 0);
                f[1].load(ra, rb, (slot ^ 1) << 4);
                multiply<S, MM, 0>(acc, f[0], sa, sb);
                if (more) stage(next, fill, 1);
                f[0].load(ra, rb, (slot ^ 2) << 4);
                multiply<S, MM, 1>(acc, f[1], sa, sb);
                if (more) stage(next, fill, 2);
                f[1].load(ra, rb, (slot ^ 3) << 4);
                multiply<S, MM, 2>(acc, f[0], sa, sb);
                if (more) stage(next, fill, 3);
                multiply<S, MM, 3>(acc, f[1], sa, sb);
            }
            buf = after(buf);
            fill = after(fill);
        }
        if constexpr (MM::kScaled) {
            if (half) {
                wait_and_meet<0>();
                if (S::KS == 1 || group == slabs % S::KS) {
                    buf = lds + slabs / S::KS % S::STAGES * kStage;
                    uint32_t sa[S::MT], sb[S::NT];
                    scales(buf, 16 * L.h, sa, sb);  // group h takes blocks 2h and 2h + 1 of four
                    const char *ra = buf + fa, *rb = buf + fb;
                    const int slot = (2 * L.h) ^ turn;
                    Frags<S> f[2];
                    f[0].load(ra, rb, (slot ^ 0) << 4);
                    f[1].load(ra, rb, (slot ^ 1) << 4);
                    multiply<S, MM, 0>(acc, f[0], sa, sb);
                    multiply<S, MM, 1>(acc, f[1], sa, sb);
                }
            }
        }
        if constexpr (S::KS > 1) {
            static_assert((S::KS - 1) * S::TILE * S::TILE * 4 <= product_lds<S, MM>(), "the groups' sums fit");
            __syncthreads();
            float* mine = (float*)all + (group - 1) * S::TILE * S::TILE + L.wave * S::MT * S::NT * 1024 + L.lane * 4;
            if (group > 0) {
#pragma unroll
                for (int i = 0; i < S::MT; ++i)
#pragma unroll
                    for (int j = 0; j < S::NT; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            f32x4 v;
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] = acc[i][j][4 * q + r];
                            *(f32x4*)(mine + ((i * S::NT + j) * 4 + q) * 256) = v;
                        }
            }
            __syncthreads();
            if (group > 0) return false;
#pragma unroll
            for (int g = 1; g < S::KS; ++g)
#pragma unroll
                for (int i = 0; i < S::MT; ++i)
#pragma unroll
                    for (int j = 0; j < S::NT; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f32x4 v =
                                *(const f32x4*)(mine + g * S::TILE * S::TILE + ((i * S::NT + j) * 4 + q) * 256);
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[i][j][4 * q + r] += v[r];
                        }
        }
        return true;
    }
};

// Turns the 4 x 4 values of four neighbouring lanes: v[r] of lane t <-> v[t] of lane r.
template <int CTRL>
__device__ __forceinline__ float quad_swap(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ void quad_turn(float (&v)[4]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
    for (int p = 0; p < 4; p += 2) {
        const float o = quad_swap<0xB1>(odd ? v[p] : v[p + 1]);  // with lane ^ 1
        v[p] = odd ? o : v[p];
        v[p + 1] = odd ? v[p + 1] : o;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const float o = quad_swap<0x4E>(high ? v[p] : v[p + 2]);  // with lane ^ 2
        v[p] = high ? o : v[p];
        v[p + 2] = high ? v[p + 2] : o;
    }
}

// Two dwords of four 16-bit values each: those of four neighbouring lanes turned, as
// quad_turn does.
__device__ __forceinline__ uint32_t lane_xor1(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t lane_xor2(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
}
__device__ __forceinline__ u32x2 quad_turn16(u32x2 d) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
    // even lanes: the low halves of (own, other); odd lanes: the high halves of (other, own)
    const uint32_t pick = odd ? 0x07060302u : 0x01000504u;
    const uint32_t a = __builtin_amdgcn_perm(d[0], lane_xor1(d[0]), pick);
    const uint32_t b = __builtin_amdgcn_perm(d[1], lane_xor1(d[1]), pick);
    const uint32_t o = lane_xor2(high ? a : b);
    return u32x2{high ? o : a, high ? b : o};
}
__device__ __forceinline__ f16x4 quad_turn16(f16x4 v) {
    return __builtin_bit_cast(f16x4, quad_turn16(__builtin_bit_cast(u32x2, v)));
}

// A wave's fp16 results on their way to the transposed place: 32 columns by WM rows
// at a time, through this wave's own part of LDS, so that a column's WM values
// leave as one run.
template <class S>
struct Turner {
    static constexpr int kLd = S::WM * 2 + 16;  // bytes a column
    static constexpr int kBytes = 32 * kLd;     // per wave
    char* lds;
    __device__ Turner(char* all, const Lane& L) : lds(all + L.wave * kBytes) {}
    // rows i..i+3 (i within WM) of this lane's column
    __device__ __forceinline__ void put(const Lane& L, int i, f16x4 v) { *(f16x4*)(lds + L.c * kLd + i * 2) = v; }
    // out[(j0 + c) * ld + i0 ..], columns below cols, rows below rows (a multiple of 8)
    __device__ __forceinline__ void flush(const Lane& L, _Float16* out, int64_t ld, int j0, int i0, int cols, int rows) {
        constexpr int kRun = S::WM / 8;  // 16-byte pieces a column
#pragma unroll
        for (int t = 0; t < 32 * kRun / 64; ++t) {
            const int p = t * 64 + L.lane, c = p / kRun, i = p % kRun * 8;
            const f16x8 v = *(const f16x8*)(lds + c * kLd + i * 2);
            if (j0 + c < cols && i0 + i < rows) *(f16x8*)(out + (int64_t)(j0 + c) * ld + i0 + i) = v;
        }
    }
};

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
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

template <class Args>
int launch(void (*kernel)(Args), dim3 grid, int block, hipStream_t s, const Args& args, const char* what) {
    // the threads of a launch are counted in 32 bits
    if ((uint64_t)grid.x * (uint64_t)block > 0xFFFFFFFFu) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    void* params[] = {const_cast<Args*>(&args)};
    const hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(block), params, 0, s);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(ZERO_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    }
    return ok();
}

// The shapes in use: (tile, wave rows, wave columns, slabs in LDS).
typedef Shape<256, 128, 128, 2> Tile256;
typedef Shape<192, 96, 96, 3> Tile192;
typedef Shape<128, 64, 64, 2> Tile128;      // two workgroups on a CU
typedef Shape<128, 64, 64, 3> Tile128Few;   // at most one workgroup for a CU
typedef Shape<64, 32, 32, 2> Tile64;        // four
typedef Shape<64, 32, 32, 4> Tile64Two;     // two
typedef Shape<64, 32, 32, 3, 2> Tile64Few;  // at most one: 16 against 21 us with one group (1024 x 1024 x 4096)

// The shape that a product takes, by the tiles it has at each: microseconds a slab
// as measured (fp16, 256 CUs, tiles of 4096 long rows) times the rounds that the
// tiles need.  4-bit operands move the same bytes a slab and take the same table; what
// a round costs beside its slabs (11 us for tiles of 256) is not in it.  Which of 192 and 256 wins at large sizes is mostly a matter of how
// whole the last round is: 136 tiles of 256 leave half of the CUs idle
// where 253 of 192 fill them.
template <class F>
int pick_tile(F tiles) {
    const int64_t t256 = tiles(256), t192 = tiles(192), t128 = tiles(128), t64 = tiles(64);
    const double cost[7] = {1.93 * (double)ceil_div(t256, 256),
                            1.17 * (double)ceil_div(t192, 256),
                            1.14 * (double)ceil_div(t128, 512),
                            0.61 * (double)ceil_div(t128, 256),
                            0.81 * (double)ceil_div(t64, 1024),
                            0.46 * (double)ceil_div(t64, 512),
                            0.25 * (double)ceil_div(t64, 256)};
    int k = 0;
    for (int i = 1; i < 7; ++i)
        if (cost[i] < cost[k]) k = i;
    return k;
}

template <class F>
int with_tile(int pick, F f) {
    switch (pick) {
        case 0: return f(Tile256());
        case 1: return f(Tile192());
        case 2: return f(Tile128());
        case 3: return f(Tile128Few());
        case 4: return f(Tile64());
        case 5: return f(Tile64Two());
        default: return f(Tile64Few());
    }
}

}  // namespace
