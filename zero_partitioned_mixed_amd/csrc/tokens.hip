// Operators that move rows of tokens by a number that each token has: the embedding lookup and
// its gradient, and tokens sorted by expert and back.  Both rest on one stable sort of small
// numbers; every sum is formed in a fixed order.
#include "mx_common.h"

namespace {

// ---------------------------------------------------------------- numbers of tokens
// A token's number as a key 0 .. limit: what lies outside [0, limit) is `limit`.
struct Ids {
    const void* at;
    int wide;  // int64, else int32
    uint32_t limit;
    __device__ __forceinline__ uint32_t operator()(int64_t i) const {
        if (wide) {
            const int64_t v = ((const int64_t*)at)[i];
            return v < 0 || v >= (int64_t)limit ? limit : (uint32_t)v;
        }
        const int32_t v = ((const int32_t*)at)[i];
        return v < 0 || (uint32_t)v >= limit ? limit : (uint32_t)v;
    }
};

// n / d of 32-bit numbers by a product and shifts (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
struct Divider {
    uint32_t d, m, s1, s2;
    Divider(uint32_t by = 1) : d(by) {
        uint32_t l = 0;
        while (l < 32 && (uint64_t(1) << l) < by) ++l;
        m = (uint32_t)(((((uint64_t)1 << l) - by) << 32) / by + 1);
        s1 = l < 1 ? l : 1;
        s2 = l < 1 ? 0 : l - 1;
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        const uint32_t t = __umulhi(m, n);
        return (t + ((n - t) >> s1)) >> s2;
    }
};

// Rows of `cols` elements as vectors of eight, one vector after the other over all rows; a
// workgroup takes kSpan of them, a thread kEach that are 256 apart.
constexpr int kEach = 4, kSpan = 256 * kEach;
struct Vectors {
    uint64_t all;
    uint32_t across;
    Divider by;
    Vectors(int64_t rows, int64_t cols)
        : all((uint64_t)rows * (uint64_t)ceil_div(cols, 8)), across((uint32_t)ceil_div(cols, 8)), by(across) {}
    int64_t workgroups() const { return (int64_t)((all + kSpan - 1) / kSpan); }
};
struct Place8 {
    int64_t row, c;
    bool there;
};
__device__ __forceinline__ void places8(const Vectors& v, Place8 (&p)[kEach]) {
    const uint64_t base = (uint64_t)blockIdx.x * kSpan;
    const uint64_t row0 = base >> 32 ? base / v.across : (uint64_t)((uint32_t)base / v.across);
    const uint32_t rem = (uint32_t)(base - row0 * v.across);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t o = rem + i * 256 + threadIdx.x, q = v.by(o);
        p[i].row = (int64_t)(row0 + q);
        p[i].c = (int64_t)(o - q * v.across) * 8;
        p[i].there = base + i * 256 + threadIdx.x < v.all;
    }
}

// ---------------------------------------------------------------- the sort
// Stable, by at most 9 bits of the key a pass (least significant first).  A workgroup takes a
// contiguous tile, each of its waves a contiguous part: counts per wave and digit give every
// wave its first place for every digit, and within 64 keys the lanes with the same digit find
// each other by one ballot per bit.  Integer counts alone are added atomically, in LDS.  A single tile
// (up to 4096 numbers) takes all its passes in one launch.  Bound by latency: 131072 numbers below 64
// 15 us in two launches, 1024 below 50258 11 us in one.  One tile against several, two passes within the embedding's
// gradient (us, and the host's): 4096 numbers 25.7 (9) and 26.0 (19), 6000 31.6 and 28.4, 16384 64 and 31.
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits, kSortWaves = 8, kSortThreads = 64 * kSortWaves;
constexpr int64_t kOneTile = 4096, kMinTile = 2048, kMostTiles = 256;  // three passes at most: 24 bits of key

struct SortArgs {
    Ids ids;                  // first pass
    const uint32_t *keys, *from;  // later ones: keys, and where they came from
    uint32_t *keys_out, *from_out;
    int32_t* place;           // last pass: from_out's inverse
    int32_t* offsets;         // single pass: the first places of keys 0 .. ids.limit
    uint32_t* counts;         // [tiles][kBins]
    uint32_t n, tile, tiles;
    int shift, bits;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) {
    return a.keys == nullptr ? a.ids(i) : a.keys[i];
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
    __shared__ uint32_t bins[kBins];
    bins[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t first = blockIdx.x * a.tile, end = a.n - first < a.tile ? a.n : first + a.tile, mask = (1u << a.bits) - 1;
    for (uint32_t i = first + threadIdx.x; i < end; i += kSortThreads) atomicAdd(&bins[sort_key(a, i) >> a.shift & mask], 1u);
    __syncthreads();
    a.counts[blockIdx.x * kBins + threadIdx.x] = bins[threadIdx.x];
}

// A batch of a wave's part: kAtOnce keys a lane, 64 apart, loaded together.
constexpr int kAtOnce = 4, kBatch = 64 * kAtOnce;
struct Batch {
    uint32_t key[kAtOnce], from[kAtOnce];
    __device__ __forceinline__ void load(const SortArgs& a, uint32_t i0, uint32_t end, bool origins) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const uint32_t i = i0 + u * 64 + (threadIdx.x & 63);
            key[u] = i < end ? sort_key(a, i) : 0;
            from[u] = origins && a.from != nullptr && i < end ? a.from[i] : i;
        }
    }
};

__device__ __forceinline__ void sort_pass(const SortArgs& a, uint32_t (&next)[kSortWaves][kBins], uint32_t (&meet)[kSortWaves]) {
    static_assert(kBins == kSortThreads, "a thread a digit");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t mask = (1u << a.bits) - 1, part = a.tile / kSortWaves;
    const uint64_t start = (uint64_t)blockIdx.x * a.tile + (uint64_t)wave * part;
    const uint32_t first = start < a.n ? (uint32_t)start : a.n, end = a.n - first < part ? a.n : first + part;
    const bool once = part <= kBatch;  // the keys stay in registers
    Batch k;
    if (once) k.load(a, first, end, true);
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) next[w][tid] = 0;
    __syncthreads();
    for (uint32_t i0 = first; i0 < end; i0 += kBatch) {
        if (!once) k.load(a, i0, end, false);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (i0 + u * 64 + lane < end) atomicAdd(&next[wave][k.key[u] >> a.shift & mask], 1u);
    }
    __syncthreads();
    uint32_t all = 0, before = 0;  // this thread's digit: everywhere, in tiles before this one
    if (a.tiles == 1) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) all += next[w][tid];
    } else {
#pragma unroll 8
        for (uint32_t t = 0; t < a.tiles; ++t) {
            const uint32_t c = a.counts[t * kBins + tid];
            all += c;
            before += t < blockIdx.x ? c : 0;
        }
    }
    uint32_t sum = all;  // of this digit and the lower ones
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t v = __shfl_up(sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 63) meet[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += meet[w];
    if (a.offsets != nullptr && blockIdx.x == 0 && (uint32_t)tid <= a.ids.limit) a.offsets[tid] = (int32_t)(sum - all);
    uint32_t at = sum - all + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = next[w][tid];
        next[w][tid] = at;
        at += c;
    }
    __syncthreads();
    for (uint32_t i0 = first; i0 < end; i0 += kBatch) {
        if (!once) k.load(a, i0, end, true);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const bool there = i0 + u * 64 + lane < end;
            const uint32_t digit = k.key[u] >> a.shift & mask;
            uint64_t same = __ballot(there);
            for (int b = 0; b < a.bits; ++b) {
                const uint64_t set = __ballot(digit >> b & 1);
                same &= digit >> b & 1 ? set : ~set;
            }
            const uint32_t rank = (uint32_t)__popcll(same & ((uint64_t(1) << lane) - 1)), many = (uint32_t)__popcll(same);
            const uint32_t base = next[wave][digit];
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // all lanes have read
            __builtin_amdgcn_wave_barrier();
            if (there && rank == 0) next[wave][digit] = base + many;
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (!there) continue;
            const uint32_t to = base + rank;
            if (a.keys_out != nullptr) a.keys_out[to] = k.key[u];
            a.from_out[to] = k.from[u];
            if (a.place != nullptr) a.place[k.from[u]] = (int32_t)to;
        }
    }
}

// One pass over all tiles, or (passes) all passes of a single tile.
struct SortPasses {
    SortArgs pass[3];
    int passes;
};
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortPasses a) {
    __shared__ uint32_t next[kSortWaves][kBins];  // of a wave and digit: how many, then the next one's place
    __shared__ uint32_t meet[kSortWaves];
    for (int p = 0; p < a.passes; ++p) {
        if (p > 0) __syncthreads();  // the pass before is in memory
        sort_pass(a.pass[p], next, meet);
    }
}

// Tile and number of tiles of a sort: enough tiles for the CUs, few enough for the sums over them.
int64_t sort_tile(int64_t n) {
    if (n <= kOneTile) return round_up(n, kSortThreads);
    const int64_t t = round_up(ceil_div(n, kMostTiles), kSortThreads);
    return t > kMinTile ? t : kMinTile;
}
int sort_passes(uint32_t limit) {
    int bits = 1;
    while (bits < 32 && limit >> bits) ++bits;
    return (bits + kDigitBits - 1) / kDigitBits;
}

// Words of scratch memory: counts, and the keys and origins between passes.
int64_t sort_words(int64_t n, uint32_t limit) {
    const int64_t tiles = ceil_div(n, sort_tile(n)), passes = sort_passes(limit);
    return round_up(tiles > 1 ? tiles * kBins : 0, 64) + round_up(passes > 1 ? 2 * n : 0, 64) + round_up(passes > 2 ? 2 * n : 0, 64);
}

// Sorts the numbers of n tokens: keys (may be null) and from (their origins, in order of key,
// then of origin), and, where asked for, place and offsets (one pass only).
int sort_ids(const Ids& ids, int64_t n, uint32_t* keys, uint32_t* from, int32_t* place, int32_t* offsets, uint32_t* scratch,
             hipStream_t s, const char* what) {
    const int passes = sort_passes(ids.limit);
    int bits = 1, rc;
    while (bits < 32 && ids.limit >> bits) ++bits;
    const int each = (bits + passes - 1) / passes;
    SortArgs a{};
    a.ids = ids;
    a.n = (uint32_t)n;
    a.tile = (uint32_t)sort_tile(n);
    a.tiles = (uint32_t)ceil_div(n, a.tile);
    a.counts = scratch;
    uint32_t* const one = scratch + round_up(a.tiles > 1 ? (int64_t)a.tiles * kBins : 0, 64);
    uint32_t* const two = one + round_up(2 * n, 64);
    SortPasses one_tile{};
    for (int p = 0; p < passes; ++p) {
        const bool last = p == passes - 1;
        uint32_t* const mid = p % 2 == 0 ? one : two;
        a.keys_out = last ? keys : mid;
        a.from_out = last ? from : mid + n;
        a.place = last ? place : nullptr;
        a.offsets = last && passes == 1 ? offsets : nullptr;
        a.shift = p * each;
        a.bits = each < bits - a.shift ? each : bits - a.shift;
        if (a.tiles > 1) {
            if ((rc = launch(sort_count_kernel, dim3(a.tiles), kSortThreads, s, a, what)) != ZERO_OK) return rc;
            SortPasses one_pass{};
            one_pass.pass[0] = a;
            one_pass.passes = 1;
            if ((rc = launch(sort_kernel, dim3(a.tiles), kSortThreads, s, one_pass, what)) != ZERO_OK) return rc;
        } else {
            one_tile.pass[p] = a;
        }
        a.keys = a.keys_out;
        a.from = a.from_out;
    }
    one_tile.passes = passes;
    return a.tiles > 1 ? ok() : launch(sort_kernel, dim3(1), kSortThreads, s, one_tile, what);
}

// The first place in keys[0 .. n) (sorted) whose key is `key` or more: a wave narrows the range
// to a 64th with each round of loads.
__device__ __forceinline__ uint32_t first_place(const uint32_t* keys, uint32_t n, uint32_t key) {
    uint32_t lo = 0, hi = n;  // the answer is in [lo, hi]
    const uint32_t lane = threadIdx.x & 63;
    while (hi > lo) {
        const uint32_t step = (hi - lo + 63) / 64, at = lo + lane * step;
        const bool below = at < hi && keys[at] < key;
        const uint32_t many = (uint32_t)__popcll(__ballot(below));  // the first `many` probes
        if (many == 0) return lo;
        const uint32_t from = lo + (many - 1) * step + 1, to = lo + many * step;
        lo = from;
        hi = to < hi ? to : hi;
    }
    return lo;
}

// ---------------------------------------------------------------- embedding
//   out[t] = table[id[t]] * scale, rounded once; zeros for an id outside [0, vocab)
// Bound by memory: 32768 rows of 4096 bf16 85 us for 451 MB.  Short rows share workgroups; those of 2048
// columns or more have one each, whose id is read once (85 against 102 us).
struct LookupArgs {
    Ids ids;
    Vectors v;
    const void* table;
    int64_t ldt, cols;
    float scale;
    void* out;
    int64_t ldo;
};

template <int DT>
__global__ void __launch_bounds__(256) embedding_kernel(LookupArgs a) {
    typedef typename Elem<DT>::type T;
    Place8 p[kEach];
    places8(a.v, p);
    uint32_t key[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) key[i] = p[i].there ? a.ids(p[i].row) : a.ids.limit;
    Eight<DT> e[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        e[i].zero();
        if (key[i] < a.ids.limit) e[i].fetch((const T*)a.table + (int64_t)key[i] * a.ldt, p[i].c, a.cols);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (!p[i].there) break;
        float x[8];
        e[i].floats(x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = key[i] < a.ids.limit ? x[k] * a.scale : 0.0f;
        put8<DT>((T*)a.out + p[i].row * a.ldo, p[i].c, a.cols, x);
    }
}

// Long rows: a workgroup takes a token, its vectors kEach at a time.
template <int DT>
__global__ void __launch_bounds__(256) embedding_long_kernel(LookupArgs a) {
    typedef typename Elem<DT>::type T;
    const int64_t token = (int64_t)blockIdx.x;
    const uint32_t key = a.ids(token);
    for (int64_t c0 = threadIdx.x * 8; c0 < a.cols; c0 += 256 * 8 * kEach) {
        Eight<DT> e[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int64_t c = c0 + i * 256 * 8;
            if (c < a.cols && key < a.ids.limit) e[i].fetch((const T*)a.table + (int64_t)key * a.ldt, c, a.cols);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int64_t c = c0 + i * 256 * 8;
            if (c >= a.cols) break;
            float x[8];
            e[i].floats(x);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = key < a.ids.limit ? x[k] * a.scale : 0.0f;
            put8<DT>((T*)a.out + token * a.ldo, c, a.cols, x);
        }
    }
}

// The gradient: row v is scale times the sum of dy over the tokens whose id is v, in their order,
// in fp32, rounded once; zeros where there is none.  With the tokens sorted by id a row's tokens
// are a run.  The sorted order is cut into pieces of 8 tokens or more, so that a frequent word's
// long run is as much work for a piece as many short ones: a piece sums each of its runs, writes
// those that lie in it to their rows, and of the two that may leave it the sums so far; a second
// launch adds what belongs together, in order.  Further workgroups of the first launch write
// the zeros, which are nearly all of a large table's gradient.  Bound by memory: 131072 x 4096 bf16 from
// 32768 tokens 247 us for 1.35 GB, 16 us for the join (1371 us with a row's tokens summed by the workgroup of
// its row: a few frequent words kept a few workgroups busy).
constexpr int kZeroVectors = 16384, kZeroRows = 256, kZeroGroups = 1024;

struct GradArgs {
    const uint32_t *keys, *from;  // sorted
    uint32_t n, vocab;
    const void* dy;
    int64_t lddy, cols;
    float scale;
    void* out;
    int64_t ldo;
    float* parts;             // [pieces][2][cols]: a run's sum in the piece where it goes on (0), starts and goes on (1)
    uint32_t piece, pieces;   // tokens in a piece
    uint32_t jobs, tiles;     // workgroups with pieces: for each 256 >> lanes pieces, of 256 vectors in a row
    int lanes;                // log2 of the threads that share a piece
    uint32_t rows;            // table rows of a workgroup that writes zeros
    uint32_t across;          // vectors in a row
    Divider by;               // across
};

template <int DT>
__device__ __forceinline__ void grad_piece(const GradArgs& a) {
    typedef typename Elem<DT>::type T;
    constexpr int kAhead = 8;
    const uint32_t set = blockIdx.x / a.tiles, tile = blockIdx.x - set * a.tiles, lane = threadIdx.x & ((1u << a.lanes) - 1);
    const uint32_t piece = set * (256u >> a.lanes) + (threadIdx.x >> a.lanes);
    const int64_t c = ((int64_t)tile * 256 + lane) * 8;
    if (piece >= a.pieces || c >= a.cols) return;
    const uint32_t p0 = piece * a.piece, p1 = a.n - p0 < a.piece ? a.n : p0 + a.piece;
    const uint32_t left = p0 > 0 ? a.keys[p0 - 1] : a.vocab, right = p1 < a.n ? a.keys[p1] : a.vocab;
    uint32_t run = a.vocab;  // the id whose run is being summed, at first none
    bool entered = false;    // it started before the piece
    float sum[8];
    auto done = [&](bool leaves) {
        if (run >= a.vocab) return;
        if (entered || leaves) {
            put8<ZERO_F32>(a.parts + (int64_t)(2 * piece + !entered) * a.cols, c, a.cols, sum);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] *= a.scale;
            put8<DT>((T*)a.out + (int64_t)run * a.ldo, c, a.cols, sum);
        }
    };
    for (uint32_t i0 = p0; i0 < p1; i0 += kAhead) {
        uint32_t key[kAhead], from[kAhead];
        Eight<DT> v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            key[u] = i0 + u < p1 ? a.keys[i0 + u] : a.vocab;
            from[u] = i0 + u < p1 ? a.from[i0 + u] : 0;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (key[u] < a.vocab) v[u].fetch((const T*)a.dy + (int64_t)from[u] * a.lddy, c, a.cols);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (key[u] >= a.vocab) continue;  // sorted: nothing follows
            if (key[u] != run) {
                done(false);
                run = key[u];
                entered = i0 + u == p0 && left == run;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
            }
            float x[8];
            v[u].floats(x);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += x[k];
        }
    }
    done(right == run);
}

template <int DT>
__global__ void __launch_bounds__(256) embedding_grad_kernel(GradArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ uint8_t used[kZeroRows];
    __shared__ uint32_t ends[2];
    if (blockIdx.x < a.jobs) return grad_piece<DT>(a);
    const int tid = threadIdx.x, wave = tid >> 6;
    const uint32_t v0 = (blockIdx.x - a.jobs) * a.rows, v1 = a.vocab - v0 < a.rows ? a.vocab : v0 + a.rows;
    if (wave < 2) {
        const uint32_t at = first_place(a.keys, a.n, wave == 0 ? v0 : v1);
        if ((tid & 63) == 0) ends[wave] = at;
    }
    used[tid] = 0;
    __syncthreads();
    for (uint32_t i = ends[0] + tid; i < ends[1]; i += 256) used[a.keys[i] - v0] = 1;
    __syncthreads();
    const uint32_t all = (v1 - v0) * a.across;
    const float none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t f = tid; f < all; f += 256) {
        const uint32_t r = a.by(f);
        if (!used[r]) put8<DT>((T*)a.out + (int64_t)(v0 + r) * a.ldo, (int64_t)(f - r * a.across) * 8, a.cols, none);
    }
}

// The runs that start in a piece and leave it (each piece's last key's, at most one).  A workgroup
// looks at kJoin pieces for 256 columns.  Most such runs end in the next piece: a thread a column
// adds the two parts.  Of longer ones eight groups of 32 threads add an eighth of the parts each, in order.
constexpr int kJoin = 8;
template <int DT>
__global__ void __launch_bounds__(256) embedding_join_kernel(GradArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float sums[8][256];
    const uint32_t across = (uint32_t)((a.cols + 255) / 256), set = blockIdx.x / across, tile = blockIdx.x - set * across;
    const int group = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t c = (int64_t)tile * 256 + lane * 8, col = (int64_t)tile * 256 + threadIdx.x;
    // every wave finds out for itself which of the pieces have such a run, and which of them a long one
    const uint32_t mine = set * kJoin + (threadIdx.x & (kJoin - 1));
    const uint64_t m0 = (uint64_t)mine * a.piece, m1 = m0 + a.piece, m2 = m1 + a.piece;
    bool starts = m1 < a.n, goes_on = m2 < a.n;
    if (starts) {
        const uint32_t key = a.keys[m1], before = a.keys[m1 - 1], first = a.keys[m0], left = m0 > 0 ? a.keys[m0 - 1] : a.vocab;
        goes_on = goes_on && a.keys[goes_on ? m2 : m1] == key;
        starts = key < a.vocab && before == key && !(first == key && left == key);
    }
    const uint32_t all = (uint32_t)__ballot(starts) & ((1u << kJoin) - 1), longs = all & (uint32_t)__ballot(goes_on);
    const int64_t at = col < a.cols ? col : a.cols - 1;
    float one[kJoin], two[kJoin];
    uint32_t key[kJoin];
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
        if (!((all & ~longs) >> i & 1)) continue;
        const uint32_t piece = set * kJoin + i;
        one[i] = a.parts[(int64_t)(2 * piece + 1) * a.cols + at];
        two[i] = a.parts[(int64_t)(2 * piece + 2) * a.cols + at];
        key[i] = a.keys[(piece + 1) * a.piece];
    }
#pragma unroll
    for (int i = 0; i < kJoin; ++i)
        if (((all & ~longs) >> i & 1) && col < a.cols)
            ((T*)a.out)[(int64_t)key[i] * a.ldo + col] = from_float<DT>((one[i] + two[i]) * a.scale);
    for (uint32_t left = longs; left != 0; left &= left - 1) {
        const uint32_t piece = set * kJoin + (uint32_t)__builtin_ctz(left), run = a.keys[(piece + 1) * a.piece];
        const uint32_t many = (first_place(a.keys, a.n, run + 1) - 1) / a.piece - piece + 1;
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (c < a.cols) {
            const uint32_t each = (many + 7) / 8, to = (group + 1) * each < many ? (group + 1) * each : many;
#pragma unroll 4
            for (uint32_t q = group * each; q < to; ++q) {
                Eight<ZERO_F32> v;
                v.fetch(a.parts + (int64_t)(2 * (piece + q) + (q == 0)) * a.cols, c, a.cols);
                float x[8];
                v.floats(x);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += x[k];
            }
        }
        __syncthreads();  // the run's before have been read
#pragma unroll
        for (int k = 0; k < 8; ++k) sums[group][lane * 8 + k] = sum[k];
        __syncthreads();
        if (col < a.cols) {
            float v = sums[0][threadIdx.x];
#pragma unroll
            for (int g = 1; g < 8; ++g) v += sums[g][threadIdx.x];
            ((T*)a.out)[(int64_t)run * a.ldo + col] = from_float<DT>(v * a.scale);
        }
    }
}

// ---------------------------------------------------------------- tokens by expert
// A slot is one of a token's k assignments; place[slot] is where it went in the order of experts,
// used how many have an expert (the others' places follow behind).
struct ExpertArgs {
    Vectors v;
    const void *x, *dy;  // what is read: tokens' rows, or sorted rows; for the gradient also dy
    int64_t ldx, lddy;
    const int32_t *place, *used;
    const void* weights;  // [tokens][k]; null: ones
    int weights_f32;
    uint32_t tokens, k;
    int64_t cols;
    void *out, *dw;
    int64_t ldo;
    uint32_t first;  // token of the launch
};

// Slots with an expert; places beyond are left out, whatever the plan's memory holds.
__device__ __forceinline__ uint32_t used_of(const ExpertArgs& a) {
    const uint32_t used = (uint32_t)*a.used, slots = a.tokens * a.k;
    return used < slots ? used : slots;
}

// Sorted rows from tokens' rows: a token's row is read once and written k times; zeros behind the last.
// Bound by memory: 16384 tokens of 4096 bf16, eight each, 204 us for 1.21 GB.
template <int DT>
__global__ void __launch_bounds__(256) expert_rows_kernel(ExpertArgs a) {
    typedef typename Elem<DT>::type T;
    Place8 p[kEach];
    places8(a.v, p);
    Eight<DT> e[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (p[i].there) e[i].fetch((const T*)a.x + p[i].row * a.ldx, p[i].c, a.cols);
    const uint32_t used = used_of(a), slots = a.tokens * a.k;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (!p[i].there) break;
        float x[8];
        e[i].floats(x);
        for (uint32_t j = 0; j < a.k; ++j) {
            const uint32_t to = (uint32_t)a.place[p[i].row * a.k + j];
            if (to >= slots) continue;
            if (to < used) {
                put8<DT>((T*)a.out + (int64_t)to * a.ldo, p[i].c, a.cols, x);
            } else {
                const float none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                put8<DT>((T*)a.out + (int64_t)to * a.ldo, p[i].c, a.cols, none);
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ float weight_of(const ExpertArgs& a, int64_t slot) {
    if (a.weights == nullptr) return 1.0f;
    if (a.weights_f32) return ((const float*)a.weights)[slot];
    return to_float<DT>(((const typename Elem<DT>::type*)a.weights)[slot]);
}

// LANES lanes take a token, 64 or more, so that its places and weights are the same for a wave.
template <int LANES>
struct TokenOf {
    static constexpr int kThreads = LANES < 256 ? 256 : LANES, kTokens = kThreads / LANES;
    int64_t token;
    int lane;
    __device__ __forceinline__ explicit TokenOf(uint32_t first)
        : token((int64_t)first + blockIdx.x * kTokens + __builtin_amdgcn_readfirstlane(threadIdx.x / LANES)),
          lane(threadIdx.x % LANES) {}
};

// Tokens' rows from sorted rows: the weighted sum of a token's k rows, in fp32, in the slots' order.
// Bound by memory: the same size 280 us for 1.21 GB, 246 with ones for weights.  A token's eight rows are on
// their way at once; with the places read by each lane, and four tokens' vectors a lane, 512 us.
template <int DT, int LANES>
__global__ void __launch_bounds__(TokenOf<LANES>::kThreads) expert_combine_kernel(ExpertArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t kSlots = 8;
    const TokenOf<LANES> t(a.first);
    if (t.token >= a.tokens) return;
    const uint32_t used = used_of(a);
    for (int64_t c = t.lane * 8; c < a.cols; c += LANES * 8) {
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (uint32_t j0 = 0; j0 < a.k; j0 += kSlots) {
            Eight<DT> e[kSlots];
            uint32_t from[kSlots];
            float w[kSlots];
#pragma unroll
            for (uint32_t u = 0; u < kSlots; ++u) {
                from[u] = j0 + u < a.k ? (uint32_t)a.place[t.token * a.k + j0 + u] : 0xFFFFFFFFu;
                w[u] = j0 + u < a.k ? weight_of<DT>(a, t.token * a.k + j0 + u) : 0.0f;
            }
#pragma unroll
            for (uint32_t u = 0; u < kSlots; ++u) {
                if (from[u] < used) e[u].fetch((const T*)a.x + (int64_t)from[u] * a.ldx, c, a.cols);
            }
#pragma unroll
            for (uint32_t u = 0; u < kSlots; ++u) {
                if (from[u] >= used) continue;
                float x[8];
                e[u].floats(x);
#pragma unroll
                for (int q = 0; q < 8; ++q) sum[q] += w[u] * x[q];
            }
        }
        put8<DT>((T*)a.out + t.token * a.ldo, c, a.cols, sum);
    }
}

// The gradients of that sum: of a sorted row its weight times dy of its token (zeros behind the
// last), of a weight the product of its row with dy.  Bound by memory: the same size 428 us for 2.29 GB.
template <int DT, int LANES>
__global__ void __launch_bounds__(TokenOf<LANES>::kThreads) expert_combine_grad_kernel(ExpertArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t kSlots = 8;
    constexpr int kWaves = LANES / 64;
    __shared__ float meet[kWaves][kSlots];
    const TokenOf<LANES> t(a.first);
    if (t.token >= a.tokens) return;  // whole waves; with more than 64 lanes none
    const uint32_t used = used_of(a), slots = a.tokens * a.k;
    const T* const dy = (const T*)a.dy + t.token * a.lddy;
    for (uint32_t j0 = 0; j0 < a.k; j0 += kSlots) {
        uint32_t at[kSlots];
        float w[kSlots], dot[kSlots];
#pragma unroll
        for (uint32_t u = 0; u < kSlots; ++u) {
            at[u] = j0 + u < a.k ? (uint32_t)a.place[t.token * a.k + j0 + u] : 0xFFFFFFFFu;
            w[u] = at[u] < used ? weight_of<DT>(a, t.token * a.k + j0 + u) : 0.0f;
            dot[u] = 0.0f;
        }
#pragma unroll 1
        for (int64_t c = t.lane * 8; c < a.cols; c += LANES * 8) {
            Eight<DT> ey, e[kSlots];
            ey.fetch(dy, c, a.cols);
            if (a.dw != nullptr) {
#pragma unroll
                for (uint32_t u = 0; u < kSlots; ++u)
                    if (at[u] < used) e[u].fetch((const T*)a.x + (int64_t)at[u] * a.ldx, c, a.cols);
            }
            float y[8];
            ey.floats(y);
            if (a.out != nullptr) {
#pragma unroll
                for (uint32_t u = 0; u < kSlots; ++u) {
                    if (at[u] >= slots) continue;
                    float g[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) g[q] = at[u] < used ? w[u] * y[q] : 0.0f;
                    put8<DT>((T*)a.out + (int64_t)at[u] * a.ldo, c, a.cols, g);
                }
            }
            if (a.dw != nullptr) {
#pragma unroll
                for (uint32_t u = 0; u < kSlots; ++u) {
                    if (at[u] >= used) continue;
                    float x[8];
                    e[u].floats(x);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dot[u] += x[q] * y[q];
                }
            }
        }
        if (a.dw == nullptr) continue;
#pragma unroll
        for (uint32_t u = 0; u < kSlots; ++u)
#pragma unroll
            for (int d = 1; d < 64; d *= 2) dot[u] += __shfl_xor(dot[u], d);
        if constexpr (kWaves > 1) {
            __syncthreads();  // the sums before have been read
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (uint32_t u = 0; u < kSlots; ++u) meet[threadIdx.x / 64][u] = dot[u];
            }
            __syncthreads();
        }
        if (t.lane < (int)kSlots && j0 + t.lane < a.k) {
            float v = 0.0f;
            if constexpr (kWaves > 1) {
                v = meet[0][t.lane];
                for (int i = 1; i < kWaves; ++i) v += meet[i][t.lane];
            } else {
#pragma unroll
                for (uint32_t u = 0; u < kSlots; ++u) v = t.lane == (int)u ? dot[u] : v;
            }
            const int64_t slot = t.token * a.k + j0 + t.lane;
            if (a.weights_f32)
                ((float*)a.dw)[slot] = v;
            else
                ((T*)a.dw)[slot] = from_float<DT>(v);
        }
    }
}

// Where each key's run starts, for the offsets of more experts than one pass sorts.
struct OffsetArgs {
    const uint32_t* keys;
    uint32_t n, limit;
    int32_t* offsets;
};
__global__ void __launch_bounds__(256) offsets_kernel(OffsetArgs a) {
    const uint32_t key = (uint32_t)(((uint64_t)blockIdx.x * 256 + threadIdx.x) / 64);
    if (key > a.limit) return;
    const uint32_t at = first_place(a.keys, a.n, key);
    if ((threadIdx.x & 63) == 0) a.offsets[key] = (int32_t)at;
}

// ---------------------------------------------------------------- host side
template <class F>
int with_type(int32_t dt, F f) {
    switch (dt) {
        case ZERO_F16: return f(std::integral_constant<int, ZERO_F16>());
        case ZERO_BF16: return f(std::integral_constant<int, ZERO_BF16>());
        default: return f(std::integral_constant<int, ZERO_F32>());
    }
}

// Lanes that share a token's row: one to three vectors a lane, whole waves.
template <class F>
int with_lanes(int64_t cols, F f) {
    if (cols <= 1024) return f(std::integral_constant<int, 64>());
    if (cols <= 2048) return f(std::integral_constant<int, 256>());
    return f(std::integral_constant<int, 512>());
}

// launch_of(arguments, tokens) for 2^22 tokens at a time: with up to 512 threads each, 2^31 in a launch.
constexpr int64_t kTokensAtOnce = int64_t(1) << 22;
template <class F>
int in_launches(ExpertArgs a, F launch_of) {
    int rc = ZERO_OK;
    for (int64_t first = 0; first < a.tokens && rc == ZERO_OK; first += kTokensAtOnce) {
        a.first = (uint32_t)first;
        rc = launch_of(a, a.tokens - first < kTokensAtOnce ? a.tokens - first : kTokensAtOnce);
    }
    return rc;
}

int check_ids(const void* ids, int32_t bytes, int64_t n, int64_t limit, const char* what) {
    if (bytes != 4 && bytes != 8) return fail(ZERO_EINVAL, "%s: numbers of 4 or 8 bytes", what);
    if (n < 0 || n > kMaxSide || limit < 1 || limit > kMaxSide)
        return fail(ZERO_ERANGE, "%s: %lld numbers below %lld out of range", what, (long long)n, (long long)limit);
    if (n > 0 && ids == nullptr) return fail(ZERO_EINVAL, "%s: null numbers", what);
    if (!aligned(ids, bytes)) return fail(ZERO_EALIGN, "%s: numbers not aligned", what);
    return ZERO_OK;
}

int check_space(const void* ws, size_t ws_bytes, size_t need, const char* what) {
    if (need == 0) return ZERO_OK;
    if (ws == nullptr) return fail(ZERO_EINVAL, "%s: null workspace", what);
    if (!aligned(ws, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", what);
    if (ws_bytes < need) return fail(ZERO_ESPACE, "%s: workspace %zu bytes, needs %zu", what, ws_bytes, need);
    return ZERO_OK;
}

// Tokens in a piece: few where there are few tokens, for their latency; 32 where the parts that pieces
// leave would cost (32768 tokens of 4096 columns: 16 write and read 134 MB of them); no more than 4096 pieces.
int64_t grad_piece_of(int64_t n) {
    int64_t p = n / 1024 < 8 ? 8 : n / 1024 < 32 ? n / 1024 : 32;
    if (p < ceil_div(n, 4096)) p = ceil_div(n, 4096);
    return round_up(p, 8);
}
int64_t grad_parts(int64_t n, int64_t cols) { return n > grad_piece_of(n) ? 2 * ceil_div(n, grad_piece_of(n)) * cols : 0; }

// The checks shared by the calls on experts' rows; 1: nothing to do.
int check_experts(const void* a, int64_t lda, const void* b, int64_t ldb, const void* place, const void* used, int32_t dtype,
                  int64_t tokens, int64_t k, int64_t cols, const char* what) {
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    int rc;
    if ((rc = check_sides(tokens, cols, what)) != ZERO_OK) return rc;
    if (k < 1 || k > kMaxSide || tokens * k > kMaxSide) return fail(ZERO_ERANGE, "%s: too many slots", what);
    if (lda < cols || ldb < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (tokens == 0 || cols == 0) return 1;
    if (a == nullptr || b == nullptr || place == nullptr || used == nullptr) return fail(ZERO_EINVAL, "%s: null rows or places", what);
    if (!aligned(a, elem_bytes(dtype)) || !aligned(b, elem_bytes(dtype)) || !aligned(place, 4) || !aligned(used, 4))
        return fail(ZERO_EALIGN, "%s: rows or places not aligned to their elements", what);
    return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_embedding(const void* ids, int32_t id_bytes, int64_t tokens, const void* table, int32_t dtype, int64_t ldt,
                   int64_t vocab, int64_t cols, float scale, void* out, int64_t ldo, void* stream) {
    const char* what = "zero_embedding";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_ids(ids, id_bytes, tokens, vocab, what)) != ZERO_OK || (rc = check_sides(vocab, cols, what)) != ZERO_OK) return rc;
    if (ldt < cols || ldo < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (tokens == 0 || cols == 0) return ok();
    if (table == nullptr || out == nullptr) return fail(ZERO_EINVAL, "%s: null table or result", what);
    if (!aligned(table, elem_bytes(dtype)) || !aligned(out, elem_bytes(dtype)))
        return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    const Place to = values_at(out, dtype, tokens, cols, ldo);
    if (overlap(to, values_at(table, dtype, vocab, cols, ldt)) || overlap(to, Place(ids, tokens * id_bytes)))
        return fail(ZERO_EINVAL, "%s: the result overlaps an input", what);
    const LookupArgs a{{ids, id_bytes == 8, (uint32_t)vocab}, Vectors(tokens, cols), table, ldt, cols, scale, out, ldo};
    if (a.v.workgroups() > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    return with_type(dtype, [&](auto t) {
        if (cols >= 2048)
            return launch(embedding_long_kernel<decltype(t)::value>, dim3((unsigned)tokens), 256, (hipStream_t)stream, a, what);
        return launch(embedding_kernel<decltype(t)::value>, dim3((unsigned)a.v.workgroups()), 256, (hipStream_t)stream, a, what);
    });
}

size_t zero_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols) {
    if (tokens <= 0 || cols <= 0 || vocab <= 0 || tokens > kMaxSide || cols > kMaxSide || vocab > kMaxSide) return 0;
    return (size_t)(4 * (round_up(2 * tokens, 64) + sort_words(tokens, (uint32_t)vocab) + grad_parts(tokens, cols)));
}

int zero_embedding_grad(const void* ids, int32_t id_bytes, int64_t tokens, const void* dy, int32_t dtype, int64_t lddy,
                        int64_t vocab, int64_t cols, float scale, void* out, int64_t ldo, void* ws, size_t ws_bytes,
                        void* stream) {
    const char* what = "zero_embedding_grad";
    int rc;
    if (!valid_dtype(dtype, true)) return fail(ZERO_EINVAL, "%s: unknown dtype", what);
    if ((rc = check_ids(ids, id_bytes, tokens, vocab, what)) != ZERO_OK || (rc = check_sides(vocab, cols, what)) != ZERO_OK) return rc;
    if (lddy < cols || ldo < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (cols == 0) return ok();
    if (out == nullptr || (tokens > 0 && dy == nullptr)) return fail(ZERO_EINVAL, "%s: null gradient", what);
    if (!aligned(dy, elem_bytes(dtype)) || !aligned(out, elem_bytes(dtype)))
        return fail(ZERO_EALIGN, "%s: rows not aligned to their elements", what);
    if ((rc = check_space(ws, ws_bytes, zero_embedding_grad_workspace_bytes(tokens, vocab, cols), what)) != ZERO_OK) return rc;
    const Place to = values_at(out, dtype, vocab, cols, ldo);
    if (overlap(to, values_at(dy, dtype, tokens, cols, lddy)) || overlap(to, Place(ids, tokens * id_bytes)))
        return fail(ZERO_EINVAL, "%s: the gradient overlaps an input", what);
    if (meets(Place(ws, (int64_t)zero_embedding_grad_workspace_bytes(tokens, vocab, cols)),
              {to, values_at(dy, dtype, tokens, cols, lddy), Place(ids, tokens * id_bytes)}))
        return fail(ZERO_EINVAL, "%s: the workspace overlaps an input or the gradient", what);
    const hipStream_t s = (hipStream_t)stream;
    uint32_t *const keys = (uint32_t*)ws, *const from = keys + tokens;
    uint32_t* const scratch = keys + round_up(2 * tokens, 64);
    const uint32_t across = (uint32_t)ceil_div(cols, 8);
    GradArgs a{};
    a.keys = keys;
    a.from = from;
    a.n = (uint32_t)tokens;
    a.vocab = (uint32_t)vocab;
    a.dy = dy;
    a.lddy = lddy;
    a.cols = cols;
    a.scale = scale;
    a.out = out;
    a.ldo = ldo;
    a.parts = (float*)(scratch + (tokens > 0 ? sort_words(tokens, (uint32_t)vocab) : 0));
    a.piece = (uint32_t)grad_piece_of(tokens);
    a.pieces = (uint32_t)ceil_div(tokens, a.piece);
    a.across = across;
    a.by = Divider(across);
    a.tiles = (uint32_t)ceil_div(across, 256);
    while ((1u << a.lanes) < across && a.lanes < 8) ++a.lanes;
    a.jobs = (uint32_t)ceil_div(a.pieces, 256 >> a.lanes) * a.tiles;
    // rows of zeros: a few writes a thread, but no fewer workgroups than fill the CUs
    int64_t rows = kZeroVectors / across;
    if (rows > ceil_div(vocab, kZeroGroups)) rows = ceil_div(vocab, kZeroGroups);
    a.rows = (uint32_t)(rows < 1 ? 1 : rows < kZeroRows ? rows : kZeroRows);
    const int64_t groups = ceil_div(vocab, a.rows), joins = a.pieces > 1 ? ceil_div(a.pieces, kJoin) * ceil_div(cols, 256) : 0;
    if (a.jobs + groups > 0x7FFFFFFF || joins > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    if (tokens > 0 && (rc = sort_ids(Ids{ids, id_bytes == 8, (uint32_t)vocab}, tokens, keys, from, nullptr, nullptr, scratch, s,
                                     what)) != ZERO_OK)
        return rc;
    return with_type(dtype, [&](auto t) {
        const int e = launch(embedding_grad_kernel<decltype(t)::value>, dim3((unsigned)(a.jobs + groups)), 256, s, a, what);
        if (e != ZERO_OK || joins == 0) return e;
        return launch(embedding_join_kernel<decltype(t)::value>, dim3((unsigned)joins), 256, s, a, what);
    });
}

size_t zero_expert_sort_workspace_bytes(int64_t slots, int64_t experts) {
    if (slots <= 0 || experts <= 0 || slots > kMaxSide || experts > kMaxSide) return 0;
    return (size_t)(4 * (sort_words(slots, (uint32_t)experts) + (sort_passes((uint32_t)experts) > 1 ? round_up(slots, 64) : 0)));
}

int zero_expert_sort(const void* ids, int32_t id_bytes, int64_t slots, int64_t experts, int32_t* order, int32_t* place,
                     int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
    const char* what = "zero_expert_sort";
    int rc;
    if ((rc = check_ids(ids, id_bytes, slots, experts, what)) != ZERO_OK) return rc;
    if (offsets == nullptr || (slots > 0 && (order == nullptr || place == nullptr))) return fail(ZERO_EINVAL, "%s: null result", what);
    if (!aligned(order, 4) || !aligned(place, 4) || !aligned(offsets, 4)) return fail(ZERO_EALIGN, "%s: results not aligned", what);
    if ((rc = check_space(ws, ws_bytes, zero_expert_sort_workspace_bytes(slots, experts), what)) != ZERO_OK) return rc;
    const Place from(ids, slots * id_bytes), to[3] = {Place(order, slots * 4), Place(place, slots * 4), Place(offsets, (experts + 1) * 4)};
    if (meets(from, {to[0], to[1], to[2]})) return fail(ZERO_EINVAL, "%s: a result overlaps the numbers", what);
    if (meets(to[0], {to[1], to[2]}) || overlap(to[1], to[2])) return fail(ZERO_EINVAL, "%s: results overlap", what);
    if (meets(Place(ws, (int64_t)zero_expert_sort_workspace_bytes(slots, experts)), {from, to[0], to[1], to[2]}))
        return fail(ZERO_EINVAL, "%s: the workspace overlaps the numbers or a result", what);
    const hipStream_t s = (hipStream_t)stream;
    const Ids numbers{ids, id_bytes == 8, (uint32_t)experts};
    const bool one = sort_passes((uint32_t)experts) == 1;
    uint32_t* const keys = one ? nullptr : (uint32_t*)ws;
    uint32_t* const scratch = (uint32_t*)ws + (one ? 0 : round_up(slots, 64));
    if (slots > 0 && (rc = sort_ids(numbers, slots, keys, (uint32_t*)order, place, offsets, scratch, s, what)) != ZERO_OK) return rc;
    if (slots > 0 && one) return ok();
    return launch(offsets_kernel, dim3((unsigned)ceil_div((experts + 1) * 64, 256)), 256, s,
                  OffsetArgs{keys, (uint32_t)slots, (uint32_t)experts, offsets}, what);
}

int zero_expert_rows(const void* x, int32_t dtype, int64_t ldx, const int32_t* place, const int32_t* used, int64_t tokens,
                     int64_t k, int64_t cols, void* rows, int64_t ldr, void* stream) {
    const char* what = "zero_expert_rows";
    const int rc = check_experts(x, ldx, rows, ldr, place, used, dtype, tokens, k, cols, what);
    if (rc == 1) return ok();
    if (rc != ZERO_OK) return rc;
    const Place to = values_at(rows, dtype, tokens * k, cols, ldr);
    if (overlap(to, values_at(x, dtype, tokens, cols, ldx)) || overlap(to, Place(place, tokens * k * 4)) || overlap(to, Place(used, 4)))
        return fail(ZERO_EINVAL, "%s: the rows overlap an input", what);
    const ExpertArgs a{Vectors(tokens, cols), x, nullptr, ldx, 0, place, used, nullptr, 0, (uint32_t)tokens, (uint32_t)k, cols,
                       rows, nullptr, ldr, 0};
    if (a.v.workgroups() > 0x7FFFFFFF) return fail(ZERO_ERANGE, "%s: too many elements for one launch", what);
    return with_type(dtype, [&](auto t) {
        return launch(expert_rows_kernel<decltype(t)::value>, dim3((unsigned)a.v.workgroups()), 256, (hipStream_t)stream, a, what);
    });
}

int zero_expert_combine(const void* rows, int32_t dtype, int64_t ldr, const int32_t* place, const int32_t* used,
                        const void* weights, int32_t weights_dtype, int64_t tokens, int64_t k, int64_t cols, void* y,
                        int64_t ldy, void* stream) {
    const char* what = "zero_expert_combine";
    const int rc = check_experts(rows, ldr, y, ldy, place, used, dtype, tokens, k, cols, what);
    if (rc < 0) return rc;
    if (weights != nullptr && weights_dtype != dtype && weights_dtype != ZERO_F32)
        return fail(ZERO_EINVAL, "%s: weights have the rows' type or are fp32", what);
    if (!aligned(weights, elem_bytes(weights_dtype))) return fail(ZERO_EALIGN, "%s: weights not aligned to their elements", what);
    if (rc == 1) return ok();
    const Place to = values_at(y, dtype, tokens, cols, ldy);
    if (overlap(to, values_at(rows, dtype, tokens * k, cols, ldr)) || overlap(to, Place(place, tokens * k * 4)) ||
        overlap(to, Place(used, 4)) || overlap(to, Place(weights, tokens * k * (int64_t)elem_bytes(weights_dtype))))
        return fail(ZERO_EINVAL, "%s: the result overlaps an input", what);
    const ExpertArgs a{Vectors(1, 8), rows, nullptr, ldr, 0, place, used, weights, weights_dtype == ZERO_F32,
                       (uint32_t)tokens, (uint32_t)k, cols, y, nullptr, ldy, 0};
    return with_type(dtype, [&](auto t) {
        return with_lanes(cols, [&](auto l) {
            typedef TokenOf<decltype(l)::value> Token;
            return in_launches(a, [&](const ExpertArgs& part, int64_t many) {
                return launch(expert_combine_kernel<decltype(t)::value, decltype(l)::value>,
                              dim3((unsigned)ceil_div(many, Token::kTokens)), Token::kThreads, (hipStream_t)stream, part, what);
            });
        });
    });
}

int zero_expert_combine_grad(const void* dy, int64_t lddy, const void* rows, int32_t dtype, int64_t ldr, const int32_t* place,
                             const int32_t* used, const void* weights, int32_t weights_dtype, int64_t tokens, int64_t k,
                             int64_t cols, void* drows, int64_t lddr, void* dweights, void* stream) {
    const char* what = "zero_expert_combine_grad";
    const int rc = check_experts(dy, lddy, dweights == nullptr ? dy : rows, dweights == nullptr ? lddy : ldr, place, used, dtype,
                                 tokens, k, cols, what);
    if (rc < 0) return rc;
    if (weights_dtype != dtype && weights_dtype != ZERO_F32)
        return fail(ZERO_EINVAL, "%s: weights have the rows' type or are fp32", what);
    if (drows != nullptr && lddr < cols) return fail(ZERO_ERANGE, "%s: row stride below cols", what);
    if (!aligned(weights, elem_bytes(weights_dtype)) || !aligned(dweights, elem_bytes(weights_dtype)) ||
        !aligned(drows, elem_bytes(dtype)))
        return fail(ZERO_EALIGN, "%s: weights or gradients not aligned to their elements", what);
    if (rc == 1 || (drows == nullptr && dweights == nullptr)) return ok();
    if (drows != nullptr && weights == nullptr) return fail(ZERO_EINVAL, "%s: null weights", what);
    const int64_t wbytes = tokens * k * (int64_t)elem_bytes(weights_dtype);
    const Place to[2] = {values_at(drows, dtype, tokens * k, cols, lddr), Place(dweights, wbytes)};
    for (const Place& p : to)
        if (overlap(p, values_at(dy, dtype, tokens, cols, lddy)) || overlap(p, Place(place, tokens * k * 4)) ||
            overlap(p, Place(used, 4)) || overlap(p, Place(weights, wbytes)) ||
            (dweights != nullptr && overlap(p, values_at(rows, dtype, tokens * k, cols, ldr))))
            return fail(ZERO_EINVAL, "%s: a gradient overlaps an input", what);
    if (overlap(to[0], to[1])) return fail(ZERO_EINVAL, "%s: gradients overlap", what);
    const ExpertArgs a{Vectors(1, 8), rows, dy, ldr, lddy, place, used, weights, weights_dtype == ZERO_F32, (uint32_t)tokens,
                       (uint32_t)k, cols, drows, dweights, lddr, 0};
    return with_type(dtype, [&](auto t) {
        return with_lanes(cols, [&](auto l) {
            typedef TokenOf<decltype(l)::value> Token;
            return in_launches(a, [&](const ExpertArgs& part, int64_t many) {
                return launch(expert_combine_grad_kernel<decltype(t)::value, decltype(l)::value>,
                              dim3((unsigned)ceil_div(many, Token::kTokens)), Token::kThreads, (hipStream_t)stream, part, what);
            });
        });
    });
}

}  // extern "C"
