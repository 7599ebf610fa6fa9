// sample.hip -- draws and rows under temperature, top-k, top-p and min-p on gfx950.
//
// Ids in order: logit descending, id ascending.  Each of the settings leaves a
// prefix of that order, and so does their intersection; it is kept as (key,
// ties): the ids whose logit lies above `key`, and the first `ties` that
// equal it.  Weights are whole numbers, w = rint(2^44 e^((x - m) / T)) with the
// row's largest logit m, summed in 64 bits: sums are exact, whatever order a
// launch takes them in, and so are the comparisons that a token hangs on.  (A
// row of 2^18 ids sums to 2^62 at most.)
//
// Three launches.  The first reads every row once, in chunks: largest logit,
// the few ids that a cut can lie among (candidates, listed in the order of
// ids), and for top-p an estimate of what the others weigh.  The second takes
// one workgroup a row and finds the cut in the candidates.  The estimate has
// proven bounds: where both ends of them give the same cut, that is the exact
// one.  Rows that this does not settle (flat ones, whose cut lies deep, top_k
// above kMostTopK, a cut between the bounds) are done whole by one workgroup
// in the third launch; rows that nothing cuts off are summed in the second and
// drawn from in the third, which also writes truncated rows.
#include <math.h>

#include "common.h"

namespace sv {

typedef unsigned long long u64;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRowThreads = 1024;             // threads of a row's workgroup in the third launch
constexpr int kBins = 2048;                   // of a histogram
constexpr int kListKeys = 2048;               // keys that are looked at one by one
constexpr int kChunk = 8192;                  // ids of the first launch's workgroup
constexpr int kListed = 8192;                 // candidates of a row at most
constexpr int kMostTopK = kBlock;             // largest top_k that candidates are listed for
constexpr int kSliceChunks = 16384;           // chunks that a launch takes at a time
constexpr int kWriteIds = 32768;              // ids that a writing workgroup takes
constexpr double kOne = 17592186044416.0;     // 2^44, the weight of the largest logit
// Weights below half a unit are 0: from 45 log 2 = 31.2 temperatures below m on.
constexpr double kDeepest = 31.25;
// Candidates of top-p: ids within this many temperatures of the chunk's largest
// logit (a share of e^-10 = 4.5e-5 of its).
constexpr float kHot = 10.0f;

struct ChunkRec {
    uint32_t top;                // key of the largest logit
    uint32_t n;                  // candidates
    uint32_t finite;             // ids that are not masked out
    uint32_t odd;                // a NaN or +inf is among them
    double tail;                 // estimate of sum e^((x - top) / T) over the others
    double pad;
};
enum : uint32_t { kDone, kWhole, kMany, kFault };  // a row's state after the second launch
struct RowRec {
    uint32_t state;
    uint32_t n;                  // kept ids, listed (kDone)
    float m;                     // largest logit
    uint32_t finite;
};

struct SampleArgs {
    const void *logits;          // [R][J] rows, ld elements apart
    int64_t ld;
    int R, J, V;
    const float *temperature;    // [R]
    const int32_t *top_k;        // [R] or null
    const float *top_p, *min_p;  // [R] or null
    const int32_t *rows;         // [R] or null
    const float *u;              // [R][J] (draws)
    int32_t *out_tokens;         // [R][J] (draws)
    float *out_logq;             // [R][J] or null (draws)
    void *out_logits;            // rows, out_ld elements apart (truncation)
    int64_t out_ld;
    int32_t *out_kept;           // [R][J] or null
    Control *ctl;
    int row0, rows_here;         // the slice's rows
    int chunks, room;            // chunks of a row, candidates that each may list
    ChunkRec *chunk;             // [rows_here][chunks]
    RowRec *row;                 // [rows_here]
    u64 *subs;                   // [rows_here][chunks][kChunk / 256] weights of a wave's loads (draws)
    uint32_t *ids;               // [rows_here][chunks][room] candidates, then the row's kept ids
    float *vals;                 // their logits
};

// Whole numbers in the order of the floats (-0 and 0 alike).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kNoKey = 0x007fffffu;      // of -inf: ids that are masked out

// ---------------------------------------------------------------------------
// a row's settings
// ---------------------------------------------------------------------------

struct Setting {
    bool live, ok;               // the row is in use; its settings are in their ranges
    float t, p, mp, u;
    int k;                       // 0: every id
    bool greedy, whole, many;    // one id; nothing is cut off; not by candidates
};
template <bool DRAW>
__device__ __forceinline__ Setting setting_of(const SampleArgs &a, int i) {
    Setting s;
    const int r = i / a.J, j = i - r * a.J;
    const int live = a.rows ? a.rows[r] : a.J;
    s.ok = live >= 0 && live <= a.J;
    s.live = !s.ok || j < live;
    s.t = a.temperature[r];
    s.k = a.top_k ? a.top_k[r] : 0;
    s.p = a.top_p ? a.top_p[r] : 1.f;
    s.mp = a.min_p ? a.min_p[r] : 0.f;
    s.u = DRAW ? a.u[i] : 0.f;
    s.ok = s.ok && (s.t == 0.f || (s.t >= 1e-30f && s.t <= 1e30f)) && s.p > 0.f && s.mp >= 0.f && s.mp <= 1.f;
    if (DRAW && s.t != 0.f) s.ok = s.ok && s.u >= 0.f && s.u < 1.f;
    if (s.k < 0 || s.k >= a.V) s.k = 0;
    s.greedy = s.t == 0.f || s.k == 1;
    s.many = !s.greedy && s.k > kMostTopK;
    s.whole = !s.greedy && s.k == 0 && s.p >= 1.f && s.mp == 0.f;
    return s;
}

// The least logit x with e^((x - m) / T) >= min_p, and one that is not above it.
__device__ __forceinline__ uint32_t min_p_key(float m, float t, float mp) {
    const double low = (double)m + (double)t * log((double)mp);
    const float x = (float)low;
    return key_of(x) + ((double)x < low);
}

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------

// w(x) = 2^(44 + (x - m) log2(e) / T): the exponent is cut into 64ths, whose
// powers of two stand in a table, and the rest, at most ln 2 / 128 = 0.0055, goes through the
// exponential's series to the fifth power (the next term is 4e-17).
struct Weights {
    double m, c;                 // the largest logit, 64 log2(e) / T
    const double *table;         // 2^(i / 64), i < 64 (shared memory)
};
__device__ __forceinline__ u64 weight(const Weights &w, float x) {
    constexpr double kRound = 6755399441055744.0;  // 1.5 2^52: adding it rounds to whole numbers
    constexpr double z = kLn2 / 64;
    const double y = fmax(((double)x - w.m) * w.c, -64.0 * 60.0);
    const double s = y + kRound;
    const int n = (int)(uint32_t)__double_as_longlong(s);
    const double r = y - (s - kRound);
    double p = fma(r, z * z * z * z * z / 120, z * z * z * z / 24);
    p = fma(p, r, z * z * z / 6);
    p = fma(p, r, z * z / 2);
    p = fma(p, r, z);
    p = fma(p, r, 1.0);
    p = ldexp(p * w.table[n & 63], (n >> 6) + 44);
    return (u64)(__double_as_longlong(p + kRound) - __double_as_longlong(kRound));
}

// ---------------------------------------------------------------------------
// a row's ids
// ---------------------------------------------------------------------------

template <typename T> struct Row {
    static constexpr int N = 16 / sizeof(T);  // ids of a 16-byte block
    const T *p;                  // the block that holds id 0
    int skip, V, blocks;         // elements before id 0 in it; ids; blocks
};
template <typename T>
__device__ __forceinline__ Row<T> row_of(const void *base, int64_t at, int V) {
    Row<T> r;
    const T *p = (const T *)base + at;
    r.skip = (int)(((uintptr_t)p & 15u) / sizeof(T));
    r.p = p - r.skip;
    r.V = V;
    r.blocks = (r.skip + V + Row<T>::N - 1) / Row<T>::N;
    return r;
}
template <typename T> struct Unpack;
template <> struct Unpack<float> {
    static constexpr uint32_t kMasked = 0xff800000u;
    __device__ __forceinline__ static float get(const u32x4_t &w, int i) { return __uint_as_float(w[i]); }
};
template <> struct Unpack<uint16_t> {
    static constexpr uint32_t kMasked = 0xff80ff80u;
    __device__ __forceinline__ static float get(const u32x4_t &w, int i) {
        return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
};
// Blocks b, b + stride, ..; what is not the row's becomes -inf and is not read.
// Blocks that are the row's alone come in one load each, all of them under
// way together; a row's first and last may not be (or not exist): those are
// passed by, and read one by one.
template <int NB, typename T>
__device__ __forceinline__ void load_blocks(const Row<T> &r, int b, int stride, u32x4_t (&w)[NB]) {
    constexpr int N = Row<T>::N;
    const int full0 = r.skip ? 1 : 0, full1 = (r.skip + r.V) / N;  // blocks [full0, full1) are whole
#pragma unroll
    for (int j = 0; j < NB; ++j) w[j] = u32x4_t{} + Unpack<T>::kMasked;
    if (full0 < full1) {
        const u32x4_t *p = (const u32x4_t *)r.p;
#pragma unroll
        for (int j = 0; j < NB; ++j) w[j] = p[min(max(b + j * stride, full0), full1 - 1)];
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int at = b + j * stride;
        if (at >= full0 && at < full1) continue;
        w[j] = u32x4_t{} + Unpack<T>::kMasked;
        if (at >= r.blocks) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = at * N + i - r.skip;
            if (id < 0 || id >= r.V) continue;
            if constexpr (sizeof(T) == 4) w[j][i] = __float_as_uint(r.p[(int64_t)at * N + i]);
            else {
                const uint32_t e = r.p[(int64_t)at * N + i];
                w[j][i >> 1] = i & 1 ? (w[j][i >> 1] & 0xffffu) | e << 16 : (w[j][i >> 1] & 0xffff0000u) | e;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// sums over the workgroup
// ---------------------------------------------------------------------------

struct Pair {                    // ids and their weight
    uint32_t n;
    u64 w;
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) { return {a.n + b.n, a.w + b.w}; }

// A scan's step: two 32-bit moves, the source lanes out of range reading 0.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ u64 dpp0_u64(u64 v) {
    const uint32_t lo = (uint32_t)dpp0_i<CTRL, ROW_MASK>((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)dpp0_i<CTRL, ROW_MASK>((int)(uint32_t)(v >> 32));
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_scan_u64(u64 v) {
    v += dpp0_u64<kDppRowShr1, 0xf>(v);
    v += dpp0_u64<kDppRowShr2, 0xf>(v);
    v += dpp0_u64<kDppRowShr4, 0xf>(v);
    v += dpp0_u64<kDppRowShr8, 0xf>(v);
    v += dpp0_u64<kDppRowBcast15, 0xa>(v);
    v += dpp0_u64<kDppRowBcast31, 0xc>(v);
    return v;
}
__device__ __forceinline__ u64 lane_u64(u64 v, int l) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_sum_u64(u64 v) { return lane_u64(wave_scan_u64(v), 63); }
__device__ __forceinline__ uint32_t wave_sum_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)wave_incl_scan_dpp(v), 63);
}

// Shared memory of a workgroup of B threads.
template <int B> struct Scratch {
    u64 mass[kBins];             // a histogram: weights,
    uint32_t count[kBins];       // and ids
    double table[64];
    Pair waves[2][B / 64];
    uint32_t ends[2][B / 64];
    uint32_t listed;
    uint32_t found;              // the bin of a cut,
    Pair before, there;          // what lies above it, and in it
};

// What lies in the threads before this one (in thread order), and in all.
template <int B>
__device__ __forceinline__ Pair block_before(Scratch<B> &s, Pair v, Pair &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Pair inc{wave_incl_scan_dpp(v.n), wave_scan_u64(v.w)};
    __syncthreads();
    if (lane == 63) s.waves[0][wave] = inc;
    __syncthreads();
    Pair b{inc.n - v.n, inc.w - v.w};
    all = Pair{0, 0};
    for (int w = 0; w < B / 64; ++w) {
        if (w < wave) b = b + s.waves[0][w];
        all = all + s.waves[0][w];
    }
    return b;
}
// Least and largest over the workgroup.
template <int B>
__device__ __forceinline__ void block_ends(Scratch<B> &s, uint32_t &lo, uint32_t &hi) {
    for (int o = 32; o; o >>= 1) {
        lo = min(lo, (uint32_t)__shfl_xor((int)lo, o, 64));
        hi = max(hi, (uint32_t)__shfl_xor((int)hi, o, 64));
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        s.ends[0][threadIdx.x >> 6] = lo;
        s.ends[1][threadIdx.x >> 6] = hi;
    }
    __syncthreads();
    for (int w = 0; w < B / 64; ++w) {
        lo = min(lo, s.ends[0][w]);
        hi = max(hi, s.ends[1][w]);
    }
}

// ---------------------------------------------------------------------------
// cuts
// ---------------------------------------------------------------------------

// The ids above `key` are in, and the first `ties` that equal it.
struct Cut {
    uint32_t key, ties;
};
// The shorter of two prefixes.
__device__ __forceinline__ Cut shorter(Cut a, Cut b) {
    return a.key > b.key || (a.key == b.key && a.ties < b.ties) ? a : b;
}

// A cut is asked for by its ids or by its weight: the shortest prefix with at
// least that much.
struct Want {
    bool by_weight;
    uint32_t n;
    u64 w;
    __device__ __forceinline__ bool reached(Pair p) const { return by_weight ? p.w >= w : p.n >= n; }
};
__device__ __forceinline__ Want top_p_want(float p, u64 total) {
    return Want{true, 0, (u64)ceil((double)p * (double)total)};
}

// The histogram's bin (the highest first) in which `want` is reached, counted
// from `above` on; into s.found, s.before and s.there.
template <int B>
__device__ __forceinline__ void find_bin(Scratch<B> &s, Pair above, const Want &want) {
    constexpr int EACH = kBins / B;
    Pair mine[EACH], sum{0, 0}, all;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = kBins - 1 - ((int)threadIdx.x * EACH + i);
        mine[i] = Pair{s.count[b], s.mass[b]};
        sum = sum + mine[i];
    }
    Pair at = above + block_before(s, sum, all);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (!want.reached(at) && want.reached(at + mine[i])) {
            s.found = (uint32_t)(kBins - 1 - ((int)threadIdx.x * EACH + i));
            s.before = at;
            s.there = mine[i];
        }
        at = at + mine[i];
    }
    __syncthreads();
}

template <int B>
__device__ __forceinline__ void clear_bins(Scratch<B> &s) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += B) {
        s.mass[i] = 0;
        s.count[i] = 0;
    }
    __syncthreads();
}

// The cut among keys lo .. hi, with `above` before them and `want` reached in
// them: counts over 2048 equal parts of the range, and again over the part
// that holds the cut, until it is one key.  each(f) calls f for the keys
// (others among them are passed over); masses: weights matter, be it for the
// sum up to the cut alone, which goes to weight_to_cut.
template <int B, typename F>
__device__ __forceinline__ Cut cut_among(Scratch<B> &s, const Weights &wt, uint32_t lo, uint32_t hi, Pair above,
                                         const Want &want, bool masses, u64 &weight_to_cut, F each) {
    for (int level = 0; level < 3 && hi != lo; ++level) {  // (3 times 11 bits are 32)
        const int shift = max(0, 21 - __clz((int)(hi - lo)));  // parts of 2^shift keys
        clear_bins(s);
        each([&](uint32_t k) {
            if (k < lo || k > hi) return;
            const uint32_t b = (k - lo) >> shift;
            atomicAdd(&s.count[b], 1u);
            if (masses) atomicAdd(&s.mass[b], weight(wt, of_key(k)));
        });
        find_bin(s, above, want);
        above = s.before;
        lo += s.found << shift;
        hi = min(hi, lo + ((1u << shift) - 1u));
        if (shift && s.there.n == 1) {  // (one id: its key is the part's only one)
            uint32_t l = 0xffffffffu, h = 0;
            each([&](uint32_t k) {
                if (k >= lo && k <= hi) l = h = k;
            });
            block_ends(s, l, h);
            lo = hi = h;
        }
    }
    const u64 one = weight(wt, of_key(lo));
    Cut c{lo, 0};
    if (want.by_weight) c.ties = (uint32_t)((want.w - above.w + one - 1) / one);
    else c.ties = want.n - above.n;
    weight_to_cut = above.w + one * c.ties;
    return c;
}

// ---------------------------------------------------------------------------
// first launch: chunks
// ---------------------------------------------------------------------------

// A workgroup holds its chunk in registers, 32 ids a thread; a wave's ids lie
// side by side, so that candidates come out in the order of ids.  One pass of
// HBM: 64 clocks a wave's 64 ids where a tail is estimated, about what they
// take to come.
template <typename T>
__global__ void __launch_bounds__(kBlock) chunk_kernel(SampleArgs a) {
    constexpr int N = Row<T>::N, NB = kChunk / (kBlock * N);
    __shared__ float top_s[kWaves], low_s[kWaves];
    __shared__ uint32_t group_s[kBlock], count_s[kWaves], finite_s[kWaves];
    __shared__ double tail_s[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ri = blockIdx.x / a.chunks, c = blockIdx.x - ri * a.chunks;
    const Setting g = setting_of<false>(a, a.row0 + ri);
    if (!g.live || !g.ok) return;
    const Row<T> row = row_of<T>(a.logits, (int64_t)(a.row0 + ri) * a.ld, a.V);
    const int b0 = c * (kChunk / N) + wave * 64 * NB + lane;
    u32x4_t w[NB];
    load_blocks<NB>(row, b0, 64, w);
    ChunkRec rec{kNoKey, 0, 0, 0, 0.0, 0.0};
    // ---- largest and least logit
    float top = -INFINITY, low = INFINITY;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = Unpack<T>::get(w[j], i);
            top = __builtin_elementwise_maximum(top, x);
            low = fminf(low, x);
        }
    const float own = top;
    top = wave_max(top);
    low = -wave_max(-low);
    uint32_t finite = 32;
    if (low == -INFINITY) {
        finite = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) finite += Unpack<T>::get(w[j], i) > -INFINITY;
    }
    finite = wave_sum_u32(finite);
    if (lane == 0) {
        top_s[wave] = top;
        finite_s[wave] = finite;
    }
    group_s[tid] = key_of(own);
    __syncthreads();
    rec.finite = 0;
    for (int v = 0; v < kWaves; ++v) {
        top = __builtin_elementwise_maximum(top, top_s[v]);
        rec.finite += finite_s[v];
    }
    ChunkRec *const out = a.chunk + (int64_t)ri * a.chunks + c;
    rec.odd = !(top < INFINITY);
    rec.top = key_of(top);
    if (rec.odd || top == -INFINITY || g.whole || g.many) {
        if (tid == 0) *out = rec;
        return;
    }
    // ---- where candidates begin
    float edge = top;
    if (!g.greedy) {
        if (g.k > 0) {
            // At least k of the threads' largest logits lie at or above the
            // edge, so the row's first k ids do where they lie in this chunk.
            // (20 bits of it: a few candidates more)
            uint32_t mine[kBlock / 64], at = 0;
            for (int v = 0; v < kBlock / 64; ++v) mine[v] = group_s[lane + 64 * v];
            for (int bit = 31; bit >= 12; --bit) {
                const uint32_t next = at | 1u << bit;
                int n = 0;
                for (int v = 0; v < kBlock / 64; ++v) n += __popcll(__ballot(mine[v] >= next));
                if (n >= g.k) at = next;
            }
            edge = at > kNoKey ? of_key(at) : -INFINITY;
        }
        if (g.k == 0 && g.p < 1.f) edge = top - kHot * g.t;
        if (g.mp > 0.f && (g.k == 0 || g.p >= 1.f)) {
            // (top_p's sum is over what top_k leaves)
            const float x = of_key(min_p_key(top, g.t, g.mp));
            edge = g.k == 0 && g.p >= 1.f ? x : fmaxf(edge, x);
        }
    }
    // ---- candidates, and the rest's weight
    uint32_t hits = 0;
    double tail = 0.0;
    const bool estimate = !g.greedy && g.k == 0 && g.p < 1.f;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = Unpack<T>::get(w[j], i);
            hits |= (x >= edge && x > -INFINITY ? 1u : 0u) << (j * N + i);
        }
    if (estimate) {
        // 2^a with a = d c: d = x - top, rounded, is off by 2^-24 |d|; a's whole
        // part leaves, and the rest is taken from an exact product.  (Where a
        // is far below, the rest need not be a number.)
        const double cd = kLog2e / (double)g.t;
        const float ch = (float)cd, cl = (float)(cd - (double)ch);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float d = Unpack<T>::get(w[j], i) - top;
                const float a = d * ch, n = rintf(a);
                const float f = fmaf(d, cl, fmaf(d, ch, -n));
                const float e = ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
                sum += a > -120.f && !(hits >> (j * N + i) & 1u) ? e : 0.f;
            }
            tail += (double)sum;
        }
        tail = wave_sum(tail);
    }
    uint32_t count = 0, before[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const uint32_t n = __popc(hits >> (j * N) & ((1u << N) - 1u));
        before[j] = count;
        if (__any(n != 0)) {
            const uint32_t inc = wave_incl_scan_dpp(n);
            before[j] += inc - n;
            count += (uint32_t)__builtin_amdgcn_readlane((int)inc, 63);
        }
    }
    if (lane == 0) {
        count_s[wave] = count;
        tail_s[wave] = tail;
    }
    __syncthreads();
    uint32_t base = 0;
    for (int v = 0; v < kWaves; ++v) {
        if (v < wave) base += count_s[v];
        rec.n += count_s[v];
        rec.tail += tail_s[v];
    }
    if (tid == 0) *out = rec;
    if (count == 0) return;
    const int64_t at = ((int64_t)ri * a.chunks + c) * a.room;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        uint32_t pos = base + before[j];
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (hits >> (j * N + i) & 1u) {
                if (pos < (uint32_t)a.room) {
                    a.ids[at + pos] = (uint32_t)((b0 + 64 * j) * N + i - row.skip);
                    a.vals[at + pos] = Unpack<T>::get(w[j], i);
                }
                ++pos;
            }
    }
}

// ---------------------------------------------------------------------------
// second launch: rows
// ---------------------------------------------------------------------------

// The bounds of an estimated tail: an estimate's terms are off by 2^-19 at most
// (the difference's rounding at 30 temperatures, and few of fp32 more; deeper
// ids weigh two units at most), their sums of eight by 2^-21.
constexpr double kTailError = 3.814697265625e-06;  // 2^-18
constexpr double kTailUnits = 1048576.0;           // 2^20: four units an id

template <bool DRAW>
__device__ __forceinline__ void mark_fault(const SampleArgs &a, int ri) {
    const int64_t i = a.row0 + ri;
    if constexpr (DRAW) {
        a.out_tokens[i] = -1;
        if (a.out_logq) a.out_logq[i] = NAN;
    }
    if (a.out_kept) a.out_kept[i] = -1;
    a.row[ri] = RowRec{kFault, 0, 0.f, 0};
    atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
}

__device__ __forceinline__ Weights weights_of(float m, float t, const double *table) {
    return Weights{(double)m, t == 0.f ? 0.0 : 64.0 * kLog2e / (double)t, table};
}
__device__ __forceinline__ float log_share(const Weights &wt, float x, float t, u64 total) {
    return t == 0.f ? 0.f : (float)(((double)x - wt.m) / (double)t - log((double)total / kOne));
}

template <typename T, bool DRAW>
__global__ void __launch_bounds__(kBlock) finish_kernel(SampleArgs a) {
    constexpr int N = Row<T>::N, NB = kChunk / (kBlock * N);
    __shared__ Scratch<kBlock> s;
    __shared__ float val_s[kListed];
    __shared__ uint32_t id_s[DRAW ? 1 : kListed];
    __shared__ uint32_t off_s[64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ri = DRAW ? blockIdx.x / a.chunks : blockIdx.x, c = DRAW ? blockIdx.x - ri * a.chunks : 0;
    const Setting g = setting_of<DRAW>(a, a.row0 + ri);
    if (!g.live || (c && !g.whole)) return;
    if (!g.ok) {
        if (tid == 0 && c == 0) mark_fault<DRAW>(a, ri);
        return;
    }
    // ---- the row, by every wave: lane i takes chunk i's record
    ChunkRec rec{kNoKey, 0, 0, 0, 0.0, 0.0};
    if (lane < a.chunks) rec = a.chunk[(int64_t)ri * a.chunks + lane];
    const float m = wave_max(of_key(rec.top));
    if (__any(rec.odd) || !(m > -INFINITY)) {
        if (tid == 0 && c == 0) mark_fault<DRAW>(a, ri);
        return;
    }
    const uint32_t finite = wave_sum_u32(rec.finite);
    const Weights wt = weights_of(m, g.t, s.table);
    if (tid < 64) s.table[tid] = exp2((double)tid / 64);
    const int64_t out = a.row0 + ri, list = (int64_t)ri * a.chunks * a.room;
    if (g.whole) {
        if (tid == 0 && c == 0) {
            if (a.out_kept) a.out_kept[out] = (int32_t)finite;
            a.row[ri] = RowRec{kWhole, 0, m, finite};
        }
        if constexpr (DRAW) {
            const Row<T> row = row_of<T>(a.logits, out * a.ld, a.V);
            u32x4_t w[NB];
            load_blocks<NB>(row, c * (kChunk / N) + wave * 64 * NB + lane, 64, w);
            __syncthreads();
            u64 *subs = a.subs + ((int64_t)ri * a.chunks + c) * (kChunk / 256) + wave * NB;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                u64 sum = 0;
#pragma unroll
                for (int i = 0; i < N; ++i) sum += weight(wt, Unpack<T>::get(w[j], i));
                sum = wave_sum_u64(sum);
                if (lane == 0) subs[j] = sum;
            }
        }
        return;
    }
    if (g.greedy) {
        // the first chunk that has it lists the lowest id first
        const int at = __ffsll((unsigned long long)__ballot(of_key(rec.top) == m)) - 1;
        if (tid == 0) {
            const uint32_t id = a.ids[list + (int64_t)at * a.room];
            if constexpr (DRAW) {
                a.out_tokens[out] = (int32_t)id;
                if (a.out_logq) a.out_logq[out] = 0.f;
            } else {
                a.vals[list] = a.vals[list + (int64_t)at * a.room];
                a.ids[list] = id;
            }
            if (a.out_kept) a.out_kept[out] = 1;
            a.row[ri] = RowRec{kDone, 1, m, finite};
        }
        return;
    }
    const uint32_t inc = wave_incl_scan_dpp(rec.n);
    const uint32_t n = (uint32_t)__builtin_amdgcn_readlane((int)inc, 63);
    if (wave == 0) off_s[lane] = inc - rec.n;
    if (g.many || __any(rec.n > (uint32_t)a.room) || n > (uint32_t)kListed) {
        if (tid == 0) a.row[ri] = RowRec{kMany, 0, m, finite};
        return;
    }
    __syncthreads();
    // ---- candidates, in the order of ids
    auto place = [&](uint32_t i) -> int64_t {   // of the row's candidate i
        int lo = 0, hi = a.chunks;              // the last chunk that begins at or before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (off_s[mid] <= i) lo = mid;
            else hi = mid;
        }
        return list + (int64_t)lo * a.room + (i - off_s[lo]);
    };
    uint32_t lo = 0xffffffffu, hi = 0;
    u64 sum = 0;
    for (uint32_t i = tid; i < n; i += kBlock) {
        const int64_t at = place(i);
        const float x = a.vals[at];
        val_s[i] = x;
        if (!DRAW) id_s[i] = a.ids[at];
        lo = min(lo, key_of(x));
        hi = max(hi, key_of(x));
        if (g.p < 1.f) sum += weight(wt, x);
    }
    block_ends(s, lo, hi);
    Pair all;
    block_before(s, Pair{0, sum}, all);
    u64 total = all.w;                          // of the candidates
    auto each = [&](auto f) {
        for (uint32_t i = tid; i < n; i += kBlock) f(key_of(val_s[i]));
    };
    // ---- the cut
    Cut cut{kNoKey, 0};
    // (fewer candidates than k: only ids below min_p's edge are missing, and
    // the edge comes before the k-th id)
    const bool few = g.k > 0 && (uint32_t)g.k < finite && (uint32_t)g.k <= n;
    bool many = false;
    if (few) cut = cut_among(s, wt, lo, hi, Pair{0, 0}, Want{false, (uint32_t)g.k, 0}, g.p < 1.f, total, each);
    if (g.p < 1.f) {
        u64 slack = 0;
        Want want = top_p_want(g.p, total);
        if (g.k == 0) {
            const double share = exp(((double)of_key(rec.top) - wt.m) / (double)g.t);
            const double rest = wave_sum(lane < a.chunks ? rec.tail * share : 0.0) * kOne;
            const u64 least = (u64)fmax(0.0, rest * (1.0 - kTailError) - kTailUnits);
            want = top_p_want(g.p, total + least);
            slack = top_p_want(g.p, total + (u64)(rest * (1.0 + kTailError) + kTailUnits)).w - want.w;
        }
        // Every id at or above the largest chunk's edge is a candidate, ids
        // below need not be: a cut there is not to be trusted (unless min_p's is
        // above that edge, and so the shorter one).
        const float edge = m - kHot * g.t;
        const float low = g.mp > 0.f ? of_key(min_p_key(m, g.t, g.mp)) : -INFINITY;
        Cut q{kNoKey, 0};
        u64 reached = 0;
        if (want.w + slack <= total) q = cut_among(s, wt, lo, hi, Pair{0, 0}, want, true, reached, each);
        if (g.k == 0 && of_key(q.key) < fmaxf(edge, low)) {
            many = low < edge;
        } else {
            many = reached < want.w + slack;    // the bounds' ends differ in their cuts
            cut = few ? shorter(cut, q) : q;
        }
    }
    if (many) {
        if (tid == 0) a.row[ri] = RowRec{kMany, 0, m, finite};
        return;
    }
    if (g.mp > 0.f) cut = shorter(cut, Cut{min_p_key(m, g.t, g.mp), 0xffffffffu});
    // ---- what it leaves: neighbouring candidates to a thread
    const uint32_t per = (n + kBlock - 1) / kBlock, from = min(tid * per, n), to = min(from + per, n);
    uint32_t eq = 0;
    for (uint32_t i = from; i < to; ++i) eq += key_of(val_s[i]) == cut.key;
    const uint32_t tie0 = block_before(s, Pair{eq, 0}, all).n;
    uint32_t tie = tie0;
    Pair mine{0, 0};
    auto kept = [&](uint32_t i) {
        const uint32_t k = key_of(val_s[i]);
        const bool equal = k == cut.key, in = k > cut.key || (equal && tie < cut.ties);
        tie += equal;
        return in;
    };
    for (uint32_t i = from; i < to; ++i)
        if (kept(i)) mine = mine + Pair{1, DRAW ? weight(wt, val_s[i]) : 0};
    Pair at = block_before(s, mine, all);
    tie = tie0;
    if (tid == 0) {
        if (a.out_kept) a.out_kept[out] = (int32_t)all.n;
        a.row[ri] = RowRec{kDone, all.n, m, finite};
    }
    if constexpr (DRAW) {
        const u64 target = (u64)((double)g.u * (double)all.w);
        if (at.w > target || at.w + mine.w <= target) return;
        for (uint32_t i = from; i < to; ++i) {
            if (!kept(i)) continue;
            at.w += weight(wt, val_s[i]);
            if (at.w > target) {
                a.out_tokens[out] = (int32_t)a.ids[place(i)];
                if (a.out_logq) a.out_logq[out] = log_share(wt, val_s[i], g.t, all.w);
                return;
            }
        }
    } else {
        for (uint32_t i = from; i < to; ++i) {
            if (!kept(i)) continue;
            a.ids[list + at.n] = id_s[i];       // (read from shared memory alone since the barriers)
            a.vals[list + at.n] = val_s[i];
            ++at.n;
        }
    }
}

// ---------------------------------------------------------------------------
// third launch: rows that are not settled, and truncated rows
// ---------------------------------------------------------------------------

template <typename T> __device__ __forceinline__ T masked();
template <> __device__ __forceinline__ float masked<float>() { return -INFINITY; }
template <> __device__ __forceinline__ uint16_t masked<uint16_t>() { return 0xff80; }
template <typename T> __device__ __forceinline__ T element_of(float x) {
    if constexpr (sizeof(T) == 2) return (T)(__float_as_uint(x) >> 16);
    else return x;
}

// First histogram of a whole row: bins of equal width down to the deepest
// logit with a weight, and one for the rest; the highest bin holds the largest.
// A function of the logit alone that does not rise where the logit falls.
struct Scale {
    float m, per;                // largest logit, bins per unit
};
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
    return kBins - 1 - (int)fminf((s.m - x) * s.per, (float)(kBins - 1));
}

// Calls f for each finite logit of a row, in no order.
template <typename T, typename F>
__device__ __forceinline__ void for_each_logit(const Row<T> &row, F f) {
    constexpr int N = Row<T>::N, NB = 4;
    for (int b = threadIdx.x; b < row.blocks; b += NB * kRowThreads) {
        u32x4_t w[NB];
        load_blocks<NB>(row, b, kRowThreads, w);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = Unpack<T>::get(w[j], i);
                if (x > -INFINITY) f(x);
            }
    }
}

template <typename T> struct RowShared {
    static constexpr int SUB = 64 * Row<T>::N;                // ids of a wave's load
    static constexpr int SUBS = SPEC_MAX_VERIFY_VOCAB / SUB + 1;
    static constexpr int EACH = (SUBS + kRowThreads - 1) / kRowThreads;
    Scratch<kRowThreads> s;
    uint32_t list[kListKeys];
    u64 sub_w[SUBS];             // weight above the cut, per wave's load
    uint32_t sub_n[SUBS];        // ids above it,
    uint32_t sub_e[SUBS];        // and at it
    u64 at_w;                    // of the load that holds the drawn token: weight
    uint32_t at_e;               // and ties before it
    int at_sub;
};

// Wave 0: the token in load sh.at_sub whose weights, with sh.at_w before them,
// pass the target.
template <typename T>
__device__ __forceinline__ void draw_in_load(const SampleArgs &a, const RowShared<T> &sh, const Row<T> &row,
                                             const Weights &wt, const Setting &g, Cut cut, u64 total, u64 target,
                                             int64_t out) {
    constexpr int N = Row<T>::N;
    const int b = sh.at_sub * 64 + (threadIdx.x & 63);
    u32x4_t w[1];
    load_blocks<1>(row, b, 64, w);
    float x[N];
    uint32_t at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = Unpack<T>::get(w[0], i);
        at += x[i] > -INFINITY && key_of(x[i]) == cut.key;
    }
    uint32_t tie = sh.at_e + wave_incl_scan_dpp(at) - at;
    u64 each[N], sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t k = key_of(x[i]);
        const bool equal = x[i] > -INFINITY && k == cut.key;
        each[i] = k > cut.key || (equal && tie < cut.ties) ? weight(wt, x[i]) : 0;
        tie += equal;
        sum += each[i];
    }
    u64 run = sh.at_w + wave_scan_u64(sum) - sum;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (run <= target && run + each[i] > target) {
            a.out_tokens[out] = b * N + i - row.skip;
            if (a.out_logq) a.out_logq[out] = log_share(wt, x[i], g.t, total);
        }
        run += each[i];
    }
}

// A whole row by one workgroup.
template <typename T, bool DRAW>
__device__ __forceinline__ void whole_row(const SampleArgs &a, RowShared<T> &sh, const Row<T> &row, const Setting &g,
                                          const RowRec &rec, int64_t out) {
    constexpr int N = Row<T>::N, B = kRowThreads, SUBS = RowShared<T>::SUBS, EACH = RowShared<T>::EACH;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Scratch<B> &s = sh.s;
    const Weights wt = weights_of(rec.m, g.t, s.table);
    if (tid < 64) s.table[tid] = exp2((double)tid / 64);
    const Scale scale{rec.m, (float)((kBins - 1) / (kDeepest * (double)g.t))};
    Cut cut{kNoKey, 0};                               // every id with a finite logit
    // ---- the cut
    const bool few = g.k > 0 && (uint32_t)g.k < rec.finite;
    if (few || g.p < 1.f) {
        clear_bins(s);
        for_each_logit(row, [&](float x) {
            const int b = bin_of(scale, x);
            atomicAdd(&s.count[b], 1u);
            if (g.p < 1.f) atomicAdd(&s.mass[b], weight(wt, x));
        });
        __syncthreads();
        constexpr int BINS = kBins / B;
        Pair bins[BINS], sum{0, 0}, all;              // (the cuts use the bins again)
#pragma unroll
        for (int i = 0; i < BINS; ++i) {
            bins[i] = Pair{s.count[tid * BINS + i], s.mass[tid * BINS + i]};
            sum = sum + bins[i];
        }
        block_before(s, sum, all);
        u64 total = all.w;
        auto in_bin = [&](const Want &want) -> Cut {
            find_bin(s, Pair{0, 0}, want);
            const int bin = (int)s.found;
            const Pair above = s.before, there = s.there;
            const bool listed = there.n <= (uint32_t)kListKeys;
            uint32_t lo = 0xffffffffu, hi = 0;
            if (tid == 0) s.listed = 0;
            __syncthreads();
            for_each_logit(row, [&](float x) {
                if (bin_of(scale, x) != bin) return;
                const uint32_t k = key_of(x);
                lo = min(lo, k);
                hi = max(hi, k);
                if (listed) sh.list[atomicAdd(&s.listed, 1u)] = k;  // (counted and summed alone: any order)
            });
            block_ends(s, lo, hi);
            if (listed)
                return cut_among(s, wt, lo, hi, above, want, g.p < 1.f, total, [&](auto f) {
                    for (uint32_t i = tid; i < there.n; i += B) f(sh.list[i]);
                });
            return cut_among(s, wt, lo, hi, above, want, g.p < 1.f, total, [&](auto f) {
                for_each_logit(row, [&](float x) {
                    if (bin_of(scale, x) == bin) f(key_of(x));
                });
            });
        };
        if (few) cut = in_bin(Want{false, (uint32_t)g.k, 0});
        if (g.p < 1.f) {
            const Want want = top_p_want(g.p, total);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < BINS; ++i) {
                s.count[tid * BINS + i] = bins[i].n;
                s.mass[tid * BINS + i] = bins[i].w;
            }
            const Cut q = in_bin(want);
            cut = few ? shorter(cut, q) : q;
        }
    }
    if (g.mp > 0.f) cut = shorter(cut, Cut{min_p_key(rec.m, g.t, g.mp), 0xffffffffu});
    // ---- what the cut leaves, per wave's load in the order of ids
    __syncthreads();
    const int subs = (row.blocks + 63) / 64;
    constexpr int NB = 4;
    for (int s0 = wave; s0 < subs; s0 += NB * (B / 64)) {
        u32x4_t w[NB];
        load_blocks<NB>(row, s0 * 64 + lane, B, w);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            uint32_t above = 0, at = 0;
            u64 sum = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = Unpack<T>::get(w[j], i);
                const uint32_t k = key_of(x);
                at += x > -INFINITY && k == cut.key;
                if (k > cut.key) {
                    ++above;
                    if (DRAW) sum += weight(wt, x);
                }
            }
            const uint32_t n = wave_sum_u32(at << 16 | above);
            if (DRAW) sum = wave_sum_u64(sum);
            const int sub = s0 + j * (B / 64);
            if (lane == 0 && sub < subs) {
                sh.sub_w[sub] = sum;
                sh.sub_n[sub] = n & 0xffffu;
                sh.sub_e[sub] = n >> 16;
            }
        }
    }
    __syncthreads();
    // ---- thread i: its loads; ties before them, then weights
    const u64 each = cut.ties ? weight(wt, of_key(cut.key)) : 0;
    Pair all;
    uint32_t eq[EACH], eq_sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        eq[i] = sub < subs ? sh.sub_e[sub] : 0u;
        eq_sum += eq[i];
    }
    uint32_t eq_before = block_before(s, Pair{eq_sum, 0}, all).n;
    cut.ties = min(cut.ties, all.n);
    Pair mine[EACH], sum{0, 0};
    uint32_t tie_at[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        tie_at[i] = eq_before;
        const uint32_t in = min(eq_before + eq[i], cut.ties) - min(eq_before, cut.ties);
        mine[i] = sub < subs ? Pair{sh.sub_n[sub] + in, sh.sub_w[sub] + each * in} : Pair{0, 0};
        sum = sum + mine[i];
        eq_before += eq[i];
    }
    Pair before = block_before(s, sum, all);
    if (tid == 0 && a.out_kept) a.out_kept[out] = (int32_t)all.n;
    if constexpr (DRAW) {
        const u64 target = (u64)((double)g.u * (double)all.w);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if (before.w <= target && before.w + mine[i].w > target) {
                sh.at_sub = tid * EACH + i;
                sh.at_w = before.w;
                sh.at_e = tie_at[i];
            }
            before = before + mine[i];
        }
        __syncthreads();
        if (wave == 0) draw_in_load(a, sh, row, wt, g, cut, all.w, target, out);
    } else {
        // the ties before each load
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (tid * EACH + i < subs) sh.sub_e[tid * EACH + i] = tie_at[i];
        __syncthreads();
        T *const dst = (T *)a.out_logits + out * a.out_ld;
        for (int s0 = wave; s0 < subs; s0 += NB * (B / 64)) {
            u32x4_t w[NB];
            load_blocks<NB>(row, s0 * 64 + lane, B, w);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int sub = s0 + j * (B / 64);
                if (sub >= subs) continue;
                uint32_t at = 0;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float x = Unpack<T>::get(w[j], i);
                    at += x > -INFINITY && key_of(x) == cut.key;
                }
                uint32_t tie = sh.sub_e[sub] + wave_incl_scan_dpp(at) - at;
                const int id = (sub * 64 + lane) * N - row.skip;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float x = Unpack<T>::get(w[j], i);
                    const uint32_t k = key_of(x);
                    const bool equal = x > -INFINITY && k == cut.key, in = k > cut.key || (equal && tie < cut.ties);
                    tie += equal;
                    if (id + i >= 0 && id + i < a.V) dst[id + i] = in ? element_of<T>(x) : masked<T>();
                }
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) draw_kernel(SampleArgs a) {
    constexpr int EACH = RowShared<T>::EACH, PER = kChunk / RowShared<T>::SUB;  // loads of a chunk
    __shared__ RowShared<T> sh;
    const int tid = threadIdx.x, ri = blockIdx.x;
    const Setting g = setting_of<true>(a, a.row0 + ri);
    if (!g.live) return;
    const RowRec rec = a.row[ri];
    if (rec.state == kDone || rec.state == kFault) return;
    const int64_t out = a.row0 + ri;
    const Row<T> row = row_of<T>(a.logits, out * a.ld, a.V);
    if (rec.state == kMany) {
        whole_row<T, true>(a, sh, row, g, rec, out);
        return;
    }
    const Weights wt = weights_of(rec.m, g.t, sh.s.table);
    if (tid < 64) sh.s.table[tid] = exp2((double)tid / 64);
    const int subs = (row.blocks + 63) / 64;
    const u64 *in = a.subs + (int64_t)ri * a.chunks * (kChunk / 256);
    u64 mine[EACH], sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        mine[i] = sub < subs ? in[sub / PER * (kChunk / 256) + sub % PER] : 0;
        sum += mine[i];
    }
    Pair all;
    u64 before = block_before(sh.s, Pair{0, sum}, all).w;
    const u64 target = (u64)((double)g.u * (double)all.w);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (before <= target && before + mine[i] > target) {
            sh.at_sub = tid * EACH + i;
            sh.at_w = before;
            sh.at_e = 0;
        }
        before += mine[i];
    }
    __syncthreads();
    if (tid < 64) draw_in_load(a, sh, row, wt, g, Cut{kNoKey, 0}, all.w, target, out);
}

// Truncated rows: kWriteIds ids a workgroup.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) write_kernel(SampleArgs a, int parts) {
    constexpr int N = Row<T>::N;
    __shared__ RowShared<T> sh;
    const int tid = threadIdx.x, ri = blockIdx.x / parts, part = blockIdx.x - ri * parts;
    const Setting g = setting_of<false>(a, a.row0 + ri);
    if (!g.live) return;
    const RowRec rec = a.row[ri];
    const int64_t out = a.row0 + ri;
    const Row<T> row = row_of<T>(a.logits, out * a.ld, a.V);
    if (rec.state == kMany) {
        if (part == 0) whole_row<T, false>(a, sh, row, g, rec, out);
        return;
    }
    // blocks of the output row; its first and last may be other rows' too
    const Row<T> dst = row_of<T>(a.out_logits, out * a.out_ld, a.V);
    T *const to = (T *)dst.p;
    const int b0 = part * (kWriteIds / N), b1 = min(b0 + kWriteIds / N, dst.blocks);
    const bool copy = rec.state == kWhole;
    if (copy && row.p == dst.p && row.skip == dst.skip) return;  // in place
    const T fill = rec.state == kFault ? element_of<T>(NAN) : masked<T>();
    const uint32_t nan = sizeof(T) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
    const uint32_t word = rec.state == kFault ? nan : Unpack<T>::kMasked;
    const bool alike = row.skip == dst.skip;
    for (int b = b0 + tid; b < b1; b += kRowThreads) {
        const int id = b * N - dst.skip;
        if (id >= 0 && id + N <= a.V) {
            u32x4_t w{word, word, word, word};
            if (copy) {
                if (alike) w = *(const u32x4_t *)(row.p + (int64_t)b * N);
                else {
                    T e[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) e[i] = row.p[row.skip + id + i];
                    w = __builtin_bit_cast(u32x4_t, e);
                }
            }
            *(u32x4_t *)(to + (int64_t)b * N) = w;
        } else {
            for (int i = max(id, 0); i < min(id + N, a.V); ++i)
                to[dst.skip + i] = copy ? row.p[row.skip + i] : fill;
        }
    }
    if (rec.state != kDone) return;
    __syncthreads();                            // kept ids go over what this workgroup has written
    const int64_t list = (int64_t)ri * a.chunks * a.room;
    for (uint32_t i = tid; i < rec.n; i += kRowThreads) {
        const int id = (int)a.ids[list + i], b = (id + dst.skip) / N;
        if (b >= b0 && b < b1) to[dst.skip + id] = element_of<T>(a.vals[list + i]);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static int check_rows(const void *logits, int dtype, int64_t ld, int R, int J, int V, const float *temperature) {
    if (R < 0 || J < 0 || V < 1 || ld < V) return SPEC_EINVAL;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EDTYPE;
    if (V > SPEC_MAX_VERIFY_VOCAB || (int64_t)R * J >= 1 << 22) return SPEC_EUNSUPPORTED;
    if (R == 0 || J == 0) return SPEC_OK;
    if (!logits || !temperature) return SPEC_EINVAL;
    if ((uintptr_t)logits & (dtype == SPEC_F32 ? 3u : 1u)) return SPEC_EINVAL;
    return SPEC_OK;
}

// A slice's memory.
struct Layout {
    int chunks, room, rows;      // of a row; candidates of a chunk; rows of a slice
    size_t chunk, row, subs, ids, vals, bytes;
};
static Layout layout_of(int R, int J, int V) {
    Layout l;
    l.chunks = (V + 7 + kChunk - 1) / kChunk;   // (up to 7 elements before the row in its first block)
    // a chunk lists 512 ids at least, and a row as many as the second launch
    // takes: short rows whole
    l.room = kListed / l.chunks;
    if (l.room < 512) l.room = 512;
    if (l.room > V) l.room = V;
    const int64_t rows = (int64_t)R * J;
    l.rows = kSliceChunks / l.chunks;
    if (l.rows > rows) l.rows = (int)rows;
    const size_t n = (size_t)l.rows * l.chunks;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.chunk = sizeof(Control);
    l.row = l.chunk + up(n * sizeof(ChunkRec));
    l.subs = l.row + up((size_t)l.rows * sizeof(RowRec));
    l.ids = l.subs + up(n * (kChunk / 256) * sizeof(u64));
    l.vals = l.ids + up(n * l.room * sizeof(uint32_t));
    l.bytes = l.vals + up(n * l.room * sizeof(float));
    return l;
}

template <typename T, bool DRAW>
static void launch_rows(SampleArgs a, const Layout &l, hipStream_t st) {
    const int rows = a.R * a.J, parts = (a.V + 7 + kWriteIds - 1) / kWriteIds;
    for (a.row0 = 0; a.row0 < rows; a.row0 += l.rows) {
        a.rows_here = rows - a.row0 < l.rows ? rows - a.row0 : l.rows;
        const unsigned n = (unsigned)a.rows_here, c = (unsigned)l.chunks;
        hipLaunchKernelGGL((chunk_kernel<T>), dim3(n * c), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL((finish_kernel<T, DRAW>), dim3(DRAW ? n * c : n), dim3(kBlock), 0, st, a);
        if constexpr (DRAW) hipLaunchKernelGGL((draw_kernel<T>), dim3(n), dim3(kRowThreads), 0, st, a);
        else hipLaunchKernelGGL((write_kernel<T>), dim3(n * (unsigned)parts), dim3(kRowThreads), 0, st, a, parts);
    }
}
template <bool DRAW>
static int launch_rows(SampleArgs &a, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const Layout l = layout_of(a.R, a.J, a.V);
    if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < l.bytes) return SPEC_EWORKSPACE;
    char *ws = (char *)workspace;
    a.ctl = (Control *)ws;
    a.chunks = l.chunks;
    a.room = l.room;
    a.chunk = (ChunkRec *)(ws + l.chunk);
    a.row = (RowRec *)(ws + l.row);
    a.subs = (u64 *)(ws + l.subs);
    a.ids = (uint32_t *)(ws + l.ids);
    a.vals = (float *)(ws + l.vals);
    if (dtype == SPEC_F32) launch_rows<float, DRAW>(a, l, (hipStream_t)stream);
    else launch_rows<uint16_t, DRAW>(a, l, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_sample_workspace_bytes(int R, int J, int V) {
    if (R < 0 || J < 0 || V < 1 || V > SPEC_MAX_VERIFY_VOCAB || (int64_t)R * J >= 1 << 22) return 0;
    return layout_of(R, J, V).bytes;
}

int spec_sample(const void *logits, int dtype, int64_t ld, const float *temperature, const int32_t *top_k,
                const float *top_p, const float *min_p, const int32_t *rows, const float *u, int R, int J, int V,
                int32_t *out_tokens, float *out_logq, int32_t *out_kept, void *workspace, size_t workspace_bytes,
                void *stream) {
    const int bad = check_rows(logits, dtype, ld, R, J, V, temperature);
    if (bad || R == 0 || J == 0) return bad;
    if (!u || !out_tokens) return SPEC_EINVAL;
    SampleArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.R = R;
    a.J = J;
    a.V = V;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.rows = rows;
    a.u = u;
    a.out_tokens = out_tokens;
    a.out_logq = out_logq;
    a.out_kept = out_kept;
    return launch_rows<true>(a, dtype, workspace, workspace_bytes, stream);
}

int spec_truncate_logits(const void *logits, int dtype, int64_t ld, const float *temperature, const int32_t *top_k,
                         const float *top_p, const float *min_p, const int32_t *rows, int R, int J, int V,
                         void *out_logits, int64_t out_ld, int32_t *out_kept, void *workspace,
                         size_t workspace_bytes, void *stream) {
    const int bad = check_rows(logits, dtype, ld, R, J, V, temperature);
    if (bad) return bad;
    if (out_ld < V) return SPEC_EINVAL;
    if (R == 0 || J == 0) return SPEC_OK;
    if (!out_logits || ((uintptr_t)out_logits & (dtype == SPEC_F32 ? 3u : 1u))) return SPEC_EINVAL;
    if (out_logits == logits && out_ld != ld) return SPEC_EINVAL;  // in place, or apart
    SampleArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.R = R;
    a.J = J;
    a.V = V;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.rows = rows;
    a.out_logits = out_logits;
    a.out_ld = out_ld;
    a.out_kept = out_kept;
    return launch_rows<false>(a, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
