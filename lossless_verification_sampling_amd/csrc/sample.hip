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
// Launches, over slices of rows:
//   chunks   reads every row once: largest logit, the few ids that a cut can
//            lie among (candidates, listed in the order of ids) and, for top-p, an
//            estimate of what the others weigh
//   finish   one workgroup a row: the cut among the candidates.  The estimate
//            has proven bounds; where both of their ends give the same cut, that
//            is the exact one.  Rows that this settles are done but for
//            their writing.
//   second   chunks of the other rows, from a work list: exact sums where
//            nothing is cut off, else a histogram of weights (or of ids)
//   third    the same rows where a cut is still to be found: the ids in the
//            histogram's bin that holds it are listed, what lies above is summed
//   draw     one workgroup a row that is not done: its cut and its token
//   settle, write (truncation): its cut; the rows
// A row that none of this fits (top_k above kMostTopK together with top_p, more
// equal logits than a list holds) is done whole by one workgroup at the end.
//
// Draws of bf16 rows of 151936 ids, 40 likely ones at random places above a normal floor,
// T = 0.9, in us for one row and for 256 (whose bytes alone take 15 at a copy's rate):
//   nothing cut 26, 71      top_p 0.9 27, 64       top_p 0.999 47, 166
//   min_p 0.05 26, 36       top_k 50 27, 48        top_k 200 28, 55
//   top_k 1000 37, 127      top_k 50, top_p 0.9 26, 48
//   top_k 1000, top_p 0.9 (whole rows) 101, 125
// Truncation of the 256: 49, 73, 162, 50, 61, 69, 133, 61, 168 in the same order.
#include "sample.h"

namespace sv {

constexpr int kRowThreads = 1024;             // threads of a row's workgroup in the last launches
constexpr int kListKeys = 2048;               // keys that are looked at one by one
// Ids of a chunk: 32 a lane, which stay in registers between the passes; a user's
// single row still makes a workgroup for each of 19 compute units.
constexpr int kChunk = 8192;
constexpr int kListed = 4096;                 // candidates that `finish` takes of a row at most
constexpr int kInBin = 8192;                  // ids of one bin that the last launches take
constexpr int kMostTopK = kBlock;             // largest top_k that candidates are listed for
// A chunk's histogram: bins of 16 steps (an eighth of a power of two) from
// the largest logit, bin kDeepBins - 1, to behind the last one with a weight.
constexpr int kDeepBins = 384;
// Chunks, and room for candidates, that a launch takes at a time: the workspace stays
// below 200 MB whatever the batch, and thousands of workgroups fill the card.
constexpr int kSliceChunks = 16384, kSliceListed = 1 << 24;
constexpr int kListGroups = 2048;             // workgroups of a launch over the work list: what the card holds
constexpr int kWriteIds = 32768;              // ids that a writing workgroup takes
// Candidates without top_k: ids within this many temperatures of the chunk's
// largest logit (a share of e^-8 = 3.4e-4 of its) that min_p leaves.  Where a
// wave's 2048 ids hold more than kManyHits of them (a chunk without likely ids
// has thousands of unlikely ones; more than kManyLanes lanes that hold one are taken for
// that), those below the least of the largest logits of its four rows of lanes are left
// out.  (All of them listed, 256 rows of 151936 ids took 200 us instead of 110.)
constexpr float kHot = 8.0f;
constexpr int kManyHits = 64, kManyLanes = 40;

struct ChunkRec {
    uint32_t top;                // key of the largest logit
    uint32_t n;                  // candidates
    uint32_t finite;             // ids that are not masked out, where it counts (after `second`: ids above the cut)
    uint32_t odd;                // a NaN or +inf is among them
    double tail;                 // estimate of sum e^((x - top) / T) over the others
    uint32_t share;              // key that the chunk's share of the row's first top_k ids reach
    uint32_t edge;               // key that candidates reach
};
enum : uint32_t {                // a row's state
    kDone,                       // token drawn, or kept ids listed
    kFault,
    kWhole,                      // its cut is every id at or above `key`
    kDeep,                       // its cut is looked for by histograms
    kMany,                       // by one workgroup
    kCut,                        // (truncation) its cut is `key` and ids up to `last` that equal it
    kWritten                     // (truncation) nothing is left to do
};
struct RowRec {
    uint32_t state;
    float m;                     // largest logit
    uint32_t finite;             // ids that are not masked out, where it counts
    uint32_t n;                  // kept ids, listed (kDone)
    uint32_t key;                // kWhole, kCut
    uint32_t last;               // kCut
    uint32_t by_weight;          // kDeep: top_p's cut, or top_k's
    uint32_t pad;
};
struct Listed {
    uint32_t id;
    float x;
};
struct DeepRec {                 // a kDeep row's bin (written by `third`)
    Pair above;
    Want want;
    int bin;
};
struct Work {                    // rows of the later launches, in any order
    uint32_t second, third;      // how many
    uint32_t pad[62];
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
    DeepRec *deep;               // [rows_here]
    Work *work;
    uint32_t *second, *third;    // [rows_here] rows of the slice
    u64 *hist;                   // [rows_here][chunks][kDeepBins]
    u64 *subs;                   // [rows_here][chunks][kChunk / 256] weights of a wave's loads (draws)
    Listed *list;                // [rows_here][chunks][room] candidates, then the row's kept ids
};

// ---------------------------------------------------------------------------
// a row's settings
// ---------------------------------------------------------------------------

struct Setting {
    bool live, ok;               // the row is in use; its settings are in their ranges
    float t, p, mp, u;
    int k;                       // 0: every id
    bool greedy, whole, many;    // one id; nothing is cut off; top_k is not by candidates
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

// Key of the least logit x with e^((x - m) / T) >= min_p.  (It falls with m, so
// a chunk's own largest logit gives a bound.)
__device__ __forceinline__ uint32_t min_p_key(float m, const Setting &g) {
    if (g.mp == 0.f) return kNoKey + 1;
    const double low = (double)m + (double)g.t * log((double)g.mp);
    const float x = (float)low;
    return max(key_of(x) + ((double)x < low), kNoKey + 1);
}

// Where candidates of top-p begin.  (One operation: it must not round
// differently in two places.)
__device__ __forceinline__ float hot_edge(float top, const Setting &g) { return fmaf(-kHot, g.t, top); }

__device__ __forceinline__ float log_share(const Weights &wt, float x, float t, u64 total) {
    return t == 0.f ? 0.f : (float)(((double)x - wt.m) / (double)t - log((double)total / kOne));
}

// ---------------------------------------------------------------------------
// a chunk in registers
// ---------------------------------------------------------------------------

// A workgroup of kBlock threads holds 32 ids a thread; a wave's ids lie side
// by side, N of them a lane and load.
template <typename T> struct Chunk {
    static constexpr int N = Row<T>::N, NB = kChunk / (kBlock * N);
    u32x4_t w[NB];
    int b0;                      // this lane's first block
    __device__ __forceinline__ float x(int j, int i) const { return Unpack<T>::get(w[j], i); }
    // What was unpacked before is not held for what comes: registers are waves.
    __device__ __forceinline__ void forget() {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(w[j]));
        }
    }
};
template <typename T>
__device__ __forceinline__ void load_chunk(const Row<T> &row, int c, Chunk<T> &k) {
    constexpr int N = Row<T>::N, NB = Chunk<T>::NB;
    k.b0 = c * (kChunk / N) + (threadIdx.x >> 6) * 64 * NB + (threadIdx.x & 63);
    load_blocks<NB>(row, k.b0, 64, k.w);
}

// Lists the chunk's ids whose bits are set in `hits` (bit j N + i), in their
// order; returns their number (room for fewer: the others are left out).
template <typename T>
__device__ __forceinline__ uint32_t list_hits(const SampleArgs &a, int ri, int c, const Row<T> &row, const Chunk<T> &k,
                                              uint32_t hits, uint32_t (&count_s)[kWaves]) {
    constexpr int N = Row<T>::N, NB = Chunk<T>::NB;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t count = 0, before[NB];
    if (__any(hits != 0)) {
#pragma unroll
        for (int j = 0; j < NB; j += 2) {       // (64 N at most: two loads' counts in one word)
            const uint32_t n0 = __popc(hits >> (j * N) & ((1u << N) - 1u));
            const uint32_t n1 = __popc(hits >> ((j + 1) * N) & ((1u << N) - 1u));
            const uint32_t inc = wave_incl_scan_dpp(n0 | n1 << 16), all = (uint32_t)__builtin_amdgcn_readlane((int)inc, 63);
            before[j] = count + (inc & 0xffffu) - n0;
            count += all & 0xffffu;
            before[j + 1] = count + (inc >> 16) - n1;
            count += all >> 16;
        }
    }
    if ((threadIdx.x & 63) == 0) count_s[wave] = count;
    __syncthreads();
    uint32_t base = 0, all = 0;
    for (int v = 0; v < kWaves; ++v) {
        if (v < wave) base += count_s[v];
        all += count_s[v];
    }
    if (count) {
        Listed *const out = a.list + ((int64_t)ri * a.chunks + c) * a.room;
        // few of them: each is read again (its registers have no index)
        for (uint32_t bits = hits; bits; bits &= bits - 1) {
            const uint32_t bit = (uint32_t)__ffs((int)bits) - 1u, j = bit / N;
            uint32_t pos = base + __popc((hits ^ bits) >> (j * N));
#pragma unroll
            for (int q = 0; q < NB; ++q) pos += j == q ? before[q] : 0u;
            const int at = (k.b0 + 64 * (int)j) * N + (int)(bit % N);
            if (pos < (uint32_t)a.room) out[pos] = Listed{(uint32_t)(at - row.skip), load_one(row.p, (long)at)};
        }
    }
    return all;
}

// ---------------------------------------------------------------------------
// chunks
// ---------------------------------------------------------------------------

// Largest value of each row of 16 lanes (NaN if one is), in every lane of it.
__device__ __forceinline__ float row_max(float v) {
    v = __builtin_elementwise_maximum(v, dpp_f<kDppSwap1>(v));
    v = __builtin_elementwise_maximum(v, dpp_f<kDppSwap2>(v));
    v = __builtin_elementwise_maximum(v, dpp_f<kDppHalfMirror>(v));
    return __builtin_elementwise_maximum(v, dpp_f<kDppMirror>(v));
}
__device__ __forceinline__ float of_rows(float v) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(readlane_f(v, 0), readlane_f(v, 16)),
                                         __builtin_elementwise_maximum(readlane_f(v, 32), readlane_f(v, 48)));
}

// The first launch.  Under top-p it is bound by vector instructions, 600 a wave (the
// issue slots are 90% busy): 256 rows of 151936 bf16 ids, 78 MB, in 26.5 us against 15
// for rows that nothing cuts, which are read alone.
template <typename T>
__global__ void __launch_bounds__(kBlock) chunk_kernel(SampleArgs a) {
    constexpr int N = Row<T>::N, NB = Chunk<T>::NB;
    __shared__ float top_s[kWaves];
    __shared__ uint32_t group_s[kBlock], count_s[kWaves], finite_s[kWaves], edge_s[kWaves];
    __shared__ double tail_s[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ri = blockIdx.x / a.chunks, c = blockIdx.x - ri * a.chunks;
    if (blockIdx.x == 0 && tid == 0) a.work->second = a.work->third = 0;
    const Setting g = setting_of<false>(a, a.row0 + ri);
    if (!g.live || !g.ok) return;
    const Row<T> row = row_of<T>(a.logits, (int64_t)(a.row0 + ri) * a.ld, a.V);
    Chunk<T> k;
    load_chunk(row, c, k);
    ChunkRec rec{kNoKey, 0, 0, 0, 0.0, 0xffffffffu, 0u};
    // ---- largest and least logit (the least: is an id masked out?  That counts where
    // top_k or nothing cuts)
    const bool counts = g.k > 0 || (g.p >= 1.f && g.mp == 0.f);
    float tops[NB], own = -INFINITY, low = INFINITY;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        tops[j] = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            tops[j] = __builtin_elementwise_maximum(tops[j], k.x(j, i));
            if (counts) low = __builtin_elementwise_minimum(low, k.x(j, i));
        }
        own = __builtin_elementwise_maximum(own, tops[j]);
    }
    // rows of 16 lanes first: their least is a logit that every one of them reaches
    k.forget();
    float top = row_max(own);
    float part = k.b0 - (lane & 15) < row.blocks ? top : INFINITY;  // (lanes without ids)
    part = fminf(fminf(readlane_f(part, 0), readlane_f(part, 16)), fminf(readlane_f(part, 32), readlane_f(part, 48)));
    top = of_rows(top);
    uint32_t finite = 32;
    if (__any(low == -INFINITY)) {
        finite = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) finite += k.x(j, i) > -INFINITY;
    }
    finite = wave_sum_u32(finite);
    if (lane == 0) {
        top_s[wave] = top;
        finite_s[wave] = finite;
    }
    if (g.k > 0) group_s[tid] = key_of(own);
    __syncthreads();
    for (int v = 0; v < kWaves; ++v) {
        top = __builtin_elementwise_maximum(top, top_s[v]);
        rec.finite += finite_s[v];
    }
    ChunkRec *const out = a.chunk + (int64_t)ri * a.chunks + c;
    rec.odd = !(top < INFINITY);
    rec.top = key_of(top);
    const int here = min(row.blocks - c * (kChunk / N), kChunk / N);  // blocks
    rec.share = here > 0 ? 0u : 0xffffffffu;    // (where no id is in, the share is not reached)
    if (rec.odd || top == -INFINITY || g.whole || g.many) {
        if (tid == 0) *out = rec;
        return;
    }
    // ---- where candidates begin
    float edge = top;
    const bool estimate = !g.greedy && g.k == 0 && g.p < 1.f;
    if (!g.greedy) {
        uint32_t at;
        if (g.k > 0) {
            // Groups of 8 ids; each wave finds a key that its share of k groups
            // reach with their largest logits.  So k ids of the chunk reach the least of
            // the keys, and the row's first k ids do where they lie in this chunk.  In
            // the same way, with groups of 32 ids, a key that the chunk's share of k
            // ids reach: k ids of the row reach the least of the chunks' keys.  (The keys'
            // upper 14 bits: a few candidates more.)
            constexpr int Q = 4, PER = NB / Q;  // groups of a lane, loads of a group
            auto search = [&](int n, auto reach) {
                uint32_t key = 0;
                for (int bit = 31; bit >= 18; --bit) {
                    const uint32_t next = key | 1u << bit;
                    if (reach(next) >= n) key = next;
                }
                return key;
            };
            auto of_four = [&](const uint32_t (&keys)[Q], uint32_t key) {
                int n = 0;
#pragma unroll
                for (int q = 0; q < Q; ++q) n += __popcll(__ballot(keys[q] >= key));
                return n;
            };
            // Of whole waves (or chunks) and a last one that is filled in part, that one
            // takes no share where it is filled less than half: the key of a few
            // groups strays, and the least of the keys counts.
            auto share_of = [&](int i, int blocks, int each) {
                const int all = blocks / each, rest = blocks - all * each;
                const int in = all > 0 && 2 * rest < each ? blocks - rest : blocks;
                const int mine = min(max(in - i * each, 0), each);
                return (int)(((int64_t)g.k * mine + in - 1) / in);
            };
            const int share = share_of(wave, here, 64 * NB);
            uint32_t mine[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                float t = tops[q * PER];
                if constexpr (PER == 2) t = fmaxf(t, tops[q * PER + 1]);
                mine[q] = key_of(t);
            }
            at = 0xffffffffu;
            if (share > 0) {
                if (2 * 8 * g.k <= here * N) {
                    at = search(share, [&](uint32_t key) { return of_four(mine, key); });
                } else {                        // (a short chunk: by its ids, groups would list most of it)
                    at = search(share, [&](uint32_t key) {
                        const float x = key > kNoKey ? of_key(key) : -INFINITY;
                        int n = 0;
                        k.forget();
#pragma unroll
                        for (int j = 0; j < NB; ++j)
#pragma unroll
                            for (int i = 0; i < N; ++i) n += __popcll(__ballot(k.x(j, i) >= x));
                        return n;
                    });
                }
            }
            if (lane == 0) edge_s[wave] = at;
            __syncthreads();
            for (int v = 0; v < kWaves; ++v) at = min(at, edge_s[v]);
            if (wave == 0) {                    // (which writes the record)
#pragma unroll
                for (int q = 0; q < Q; ++q) mine[q] = group_s[lane + 64 * q];
                const int n = share_of(c, row.blocks, kChunk / N);
                rec.share = n > 0 ? search(n, [&](uint32_t key) { return of_four(mine, key); }) : 0xffffffffu;
            }
        } else {
            at = kNoKey;
        }
        edge = at > kNoKey ? of_key(at) : -3.402823466e38f;  // (ids that are masked out are none)
        if (estimate) edge = fmaxf(edge, hot_edge(top, g));
        // (top_p's sum is over what top_k leaves)
        if (g.k == 0 || g.p >= 1.f) edge = fmaxf(edge, of_key(min_p_key(top, g)));
    }
    // ---- candidates, and the rest's weight
    k.forget();
    uint32_t hits = 0;
    double tail = 0.0;
    if (!g.greedy && g.k == 0) {
        // a wave that would list many leaves those below its least row's largest out
        // (where most lanes have one there is no need to count)
        int n = __popcll(__ballot(own >= edge)) > kManyLanes ? kManyHits + 1 : 0;
        if (n == 0) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if (!__any(tops[j] >= edge)) continue;
#pragma unroll
                for (int i = 0; i < N; ++i) n += __popcll(__ballot(k.x(j, i) >= edge));
            }
        }
        if (n > kManyHits) edge = fmaxf(edge, part);
        k.forget();
        if (lane == 0) edge_s[wave] = key_of(edge);
    }
    // 2^a with a = (x - top) ch, ch = log2(e) / T, in fp32: see kTailError.  In one
    // operation, x ch + b, where b = -top ch rounded is small; what that rounding took
    // (less than 2^-4) comes back with the sum.
    const float ch = estimate ? (float)(kLog2e / (double)g.t) : 0.f, b = -top * ch;
    const bool fused = fabsf(b) < 1048576.f;
    const double rounded = fused ? -(double)top * (double)ch - (double)b : 0.0;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = k.x(j, i);
        // (the first id's bit is the highest)
        if (__any(tops[j] >= edge)) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool in = x[i] >= edge;
                hits = hits + hits + in;
                x[i] = in ? -INFINITY : x[i];
            }
        } else {
            hits <<= N;
        }
        if (estimate) {
            float sum = 0.f;
            if (fused) {
#pragma unroll
                for (int i = 0; i < N; ++i) sum += __builtin_amdgcn_exp2f(fmaf(x[i], ch, b));
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) sum += __builtin_amdgcn_exp2f((x[i] - top) * ch);
            }
            tail += (double)sum;
        }
    }
    if (estimate) {
        tail = wave_sum(tail) * (double)__builtin_amdgcn_exp2f((float)rounded);
        if (lane == 0) tail_s[wave] = tail;
    }
    k.forget();
    rec.n = list_hits(a, ri, c, row, k, __brev(hits), count_s);
    if (estimate)
        for (int v = 0; v < kWaves; ++v) rec.tail += tail_s[v];
    if (!g.greedy && g.k == 0)
        for (int v = 0; v < kWaves; ++v) rec.edge = max(rec.edge, edge_s[v]);
    if (tid == 0) *out = rec;
}

// ---------------------------------------------------------------------------
// finish
// ---------------------------------------------------------------------------

// The bounds of an estimated tail.  A term's exponent is off by 3 2^-24 of
// itself (the difference's, the factor's and the product's rounding; in one operation
// the factor's and the result's), of 30 log2(e) = 43.3 at most: 5.4e-6 of the term; the
// exponential by 2.4e-7 (and again for b's rounding) and a sum of eight by 4.2e-7.  Ids
// that lie deeper weigh two units at most, and each weight is rounded to a unit: four
// units an id.
constexpr double kTailError = 7.62939453125e-06;   // 2^-17
constexpr double kTailUnits = 1048576.0;           // 2^20

// What every wave of a workgroup sees of a row's chunks: lane i chunk i's record.
struct Records {
    ChunkRec rec;
    float m;                     // largest logit
    bool ok;
    uint32_t n, off;             // candidates of the row; before this lane's chunk
    bool full;                   // more than a chunk may list
};
__device__ __forceinline__ Records records_of(const SampleArgs &a, int ri) {
    Records r;
    const int lane = threadIdx.x & 63;
    r.rec = ChunkRec{kNoKey, 0, 0, 0, 0.0, 0xffffffffu, 0u};
    if (lane < a.chunks) r.rec = a.chunk[(int64_t)ri * a.chunks + lane];
    r.m = wave_max(of_key(r.rec.top));
    r.ok = !__any(r.rec.odd) && r.m > -INFINITY;
    const uint32_t inc = wave_incl_scan_dpp(r.rec.n);
    r.n = (uint32_t)__builtin_amdgcn_readlane((int)inc, 63);
    r.off = inc - r.rec.n;
    r.full = __any(r.rec.n > (uint32_t)a.room);
    return r;
}
// Where candidate i of a row lies, off_s[c] of them before chunk c's.
__device__ __forceinline__ int64_t place_of(const SampleArgs &a, int ri, const uint32_t (&off_s)[64], uint32_t i) {
    int lo = 0, hi = a.chunks;                  // the last chunk that begins at or before it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off_s[mid] <= i) lo = mid;
        else hi = mid;
    }
    return ((int64_t)ri * a.chunks + lo) * a.room + (i - off_s[lo]);
}

template <bool DRAW>
__device__ __forceinline__ void mark_fault(const SampleArgs &a, int ri) {
    const int64_t i = a.row0 + ri;
    if constexpr (DRAW) {
        a.out_tokens[i] = -1;
        if (a.out_logq) a.out_logq[i] = NAN;
    }
    if (a.out_kept) a.out_kept[i] = -1;
    RowRec r{};
    r.state = kFault;
    a.row[ri] = r;
    atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
}

// One workgroup a row.  Up to 256 candidates are sorted, a thread's place being the number
// of those before its own; more are cut by histograms (sorted so, 512 took 32 us where
// the histograms take 23).  A thread keeps up to 32 candidates in registers from one pass
// to the next (8: 23 us against 19.6).  Bound by latency, some ten dependent steps of
// a microsecond: 12.8 us for 256 rows under top-p, 19.6 for 64 rows with top_k up to 200.
template <typename T, bool DRAW>
__global__ void __launch_bounds__(kBlock) finish_kernel(SampleArgs a) {
    __shared__ Scratch<kBlock> s;
    __shared__ float val_s[kListed];
    __shared__ uint32_t id_s[kListed];
    __shared__ uint32_t off_s[64];
    __shared__ u64 total_s;
    __shared__ uint32_t ends_s[2];
    const int tid = threadIdx.x, lane = tid & 63, ri = blockIdx.x;
    const Setting g = setting_of<DRAW>(a, a.row0 + ri);
    if (!g.live) return;
    const Records r = records_of(a, ri);
    if (!g.ok || !r.ok) {
        if (tid == 0) mark_fault<DRAW>(a, ri);
        return;
    }
    const float m = r.m;
    const uint32_t finite = wave_sum_u32(r.rec.finite);
    const int64_t out = a.row0 + ri, list = (int64_t)ri * a.chunks * a.room;
    RowRec rec{};
    rec.m = m;
    rec.finite = finite;
    auto leave = [&](uint32_t state, bool second, bool third) {
        if (tid) return;
        rec.state = state;
        a.row[ri] = rec;
        if (second) a.second[atomicAdd(&a.work->second, 1u)] = (uint32_t)ri;
        if (third) a.third[atomicAdd(&a.work->third, 1u)] = (uint32_t)ri;
    };
    if (g.greedy) {
        // the first chunk that has it lists the lowest id first
        const int at = __ffsll((unsigned long long)__ballot(of_key(r.rec.top) == m)) - 1;
        if (tid == 0) {
            const Listed first = a.list[list + (int64_t)at * a.room];
            if constexpr (DRAW) {
                a.out_tokens[out] = (int32_t)first.id;
                if (a.out_logq) a.out_logq[out] = 0.f;
            } else {
                a.list[list] = first;
            }
            if (a.out_kept) a.out_kept[out] = 1;
        }
        rec.n = 1;
        return leave(kDone, false, false);
    }
    const bool cuts = g.k > 0 && (uint32_t)g.k < finite;  // top_k leaves some out
    const uint32_t low = min_p_key(m, g);
    auto whole = [&]() {                        // at most min_p's cut
        rec.key = low;
        if (tid == 0 && g.mp == 0.f && a.out_kept) a.out_kept[out] = (int32_t)finite;
        leave(kWhole, DRAW || g.mp > 0.f, false);
    };
    auto deep = [&]() {
        const bool many = cuts && g.p < 1.f;
        rec.by_weight = !cuts;
        leave(many ? kMany : kDeep, !many, !many);
    };
    if (!cuts && g.p >= 1.f && (g.mp == 0.f || g.many || r.full)) return whole();
    if (g.many || r.full) return deep();
    // ---- candidates, in the order of ids: those at or above a key that the
    // cut cannot lie below, or from which on every id is one.  Of the others only
    // the weight counts, for top_p's sum.
    const Weights wt = weights_of(m, g.t, s.table);
    fill_table(s.table);
    if (tid < 64) off_s[tid] = r.off;
    const bool estimate = g.k == 0 && g.p < 1.f;
    uint32_t share = r.rec.share, hot = r.rec.edge;  // (no chunk: the largest number, and 0)
    for (int o = 32; o; o >>= 1) {
        share = min(share, (uint32_t)__shfl_xor((int)share, o, 64));
        hot = max(hot, (uint32_t)__shfl_xor((int)hot, o, 64));
    }
    if (g.k > 0) hot = 0;                       // every id that matters is a candidate
    if (!cuts && g.p >= 1.f && low < hot) return whole();
    const uint32_t edge = cuts ? (g.p < 1.f ? share : max(share, low)) : max(low, hot);
    __syncthreads();
    uint32_t n;
    u64 dropped = 0;
    // What top_p wants of the candidates, which weigh `total`: at least `want`,
    // at most `slack` more.
    u64 slack = 0;
    auto top_p_of = [&](u64 total) -> u64 {
        u64 least = total + dropped, most = least;
        if (estimate) {
            const double share = exp(((double)of_key(r.rec.top) - (double)m) / (double)g.t);
            const double rest = wave_sum(lane < a.chunks ? r.rec.tail * share : 0.0) * kOne;
            least += (u64)fmax(0.0, rest * (1.0 - kTailError) - kTailUnits);
            most += (u64)(rest * (1.0 + kTailError) + kTailUnits);
        }
        const u64 want = top_p_want(g.p, least).w;
        slack = top_p_want(g.p, most).w - want;
        return want;
    };
    {
        // A thread's neighbours, which stay in its registers up to kHeld of them.
        constexpr uint32_t kHeld = 32, E = 8;
        const uint32_t per = (r.n + kBlock - 1) / kBlock, from = min(tid * per, r.n), to = min(from + per, r.n);
        int c = 0, hi = a.chunks;               // the last chunk that begins at or before `from`
        while (hi - c > 1) {
            const int mid = (c + hi) >> 1;
            if (off_s[mid] <= from) c = mid;
            else hi = mid;
        }
        Listed held[kHeld];
        auto walk = [&](bool again, auto take) {
            int at = c;
            for (uint32_t i = 0; i < per; i += kHeld) {
                if (!again || per > kHeld) {
#pragma unroll
                    for (uint32_t b = 0; b < kHeld; b += E) {
                        if (i + b >= per || from >= to) continue;
#pragma unroll
                        for (uint32_t e = b; e < b + E; ++e) {
                            const uint32_t j = min(from + i + e, to - 1);
                            while (at + 1 < a.chunks && off_s[at + 1] <= j) ++at;
                            held[e] = a.list[list + (int64_t)at * a.room + (j - off_s[at])];
                        }
                    }
                }
#pragma unroll
                for (uint32_t b = 0; b < kHeld; b += E) {
                    if (i + b >= per) continue;
#pragma unroll
                    for (uint32_t e = b; e < b + E; ++e)
                        if (from + i + e < to) take(held[e]);
                }
            }
        };
        Pair mine{0, 0}, all;
        u64 inside = 0;
        walk(false, [&](Listed l) {
            const bool in = key_of(l.x) >= edge;
            mine.n += in;
            if (g.p < 1.f && !cuts) (in ? inside : mine.w) += weight(wt, l.x);
        });
        uint32_t at = block_before(s, mine, all).n;
        n = all.n;
        dropped = all.w;
        if (n > (uint32_t)kListed) {
            if (!cuts && g.p >= 1.f) return whole();
            return deep();
        }
        if (estimate && low < hot) {            // top_p's cut must lie among them
            block_before(s, Pair{0, inside}, all);
            const u64 want = top_p_of(all.w);
            if (want + slack > all.w) return deep();
        }
        walk(true, [&](Listed l) {
            if (key_of(l.x) < edge) return;
            val_s[at] = l.x;
            id_s[at++] = l.id;
        });
    }
    __syncthreads();
    // Candidates that are kept have their bit in s.count.
    auto flag = [&](uint32_t i) { atomicOr(&s.count[i >> 5], 1u << (i & 31)); };
    auto clear_flags = [&]() {
        __syncthreads();
        for (int i = tid; i < kListed / 32; i += kBlock) s.count[i] = 0u;
        __syncthreads();
    };
    const bool few = cuts && n >= (uint32_t)g.k;  // (fewer: min_p's cut comes before the k-th id)
    if (n <= kBlock) {
        // ---- sorted: a thread's place is the number of those before its own
        u64 own = ~0ull;
        if (tid < (int)n) own = (u64)~key_of(val_s[tid]) << 32 | (uint32_t)tid;
        s.mass[kBlock + tid] = own;
        __syncthreads();
        uint32_t place = 0;
        for (uint32_t i = 0; i < n; i += 4)
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) place += s.mass[kBlock + i + q] < own;
        if (tid < (int)n) s.mass[place] = own;
        __syncthreads();
        const bool in = tid < (int)n;
        const uint32_t key = in ? ~(uint32_t)(s.mass[tid] >> 32) : 0u;
        const u64 w = in && g.p < 1.f ? weight(wt, of_key(key)) : 0;
        Pair all;
        const u64 before = block_before(s, Pair{in && key >= low, w}, all).w;
        const uint32_t nk = few ? (uint32_t)g.k : n;
        uint32_t keep = min(all.n, nk);         // what min_p and top_k leave
        if (g.p < 1.f) {
            if (tid + 1 == (int)nk) total_s = before + w;
            if (tid == 0) ends_s[0] = ends_s[1] = 0;
            __syncthreads();
            const u64 want = top_p_of(total_s);
            if (before < want && before + w >= want) ends_s[0] = tid + 1;
            if (before < want + slack && before + w >= want + slack) ends_s[1] = tid + 1;
            __syncthreads();
            // Behind the candidates: then min_p's cut is the shorter one if that is
            // what ends them.  Between the bounds' cuts: not known.
            if (ends_s[0] != ends_s[1] || (ends_s[0] == 0 && low < hot)) return deep();
            if (ends_s[0]) keep = min(keep, ends_s[0]);
        }
        clear_flags();
        if (tid < (int)keep) flag((uint32_t)s.mass[tid]);
    } else {
        // ---- by histograms
        uint32_t lo = 0xffffffffu, hi = 0;
        Pair sum{0, 0}, all;
        for (uint32_t i = tid; i < n; i += kBlock) {
            const uint32_t key = key_of(val_s[i]);
            lo = min(lo, key);
            hi = max(hi, key);
            if (g.p < 1.f) sum.w += weight(wt, val_s[i]);
        }
        block_ends(s, lo, hi);
        block_before(s, sum, all);
        u64 total = all.w, reached = 0;
        auto each = [&](auto f) {
            for (uint32_t i = tid; i < n; i += kBlock) f(key_of(val_s[i]));
        };
        Cut cut{low, 0xffffffffu};
        if (few) cut = shorter(cut, cut_among(s, wt, lo, hi, Pair{0, 0}, Want{false, (uint32_t)g.k, 0}, g.p < 1.f, total, each));
        if (g.p < 1.f) {
            const u64 want = top_p_of(total);
            if (want + slack <= total) {
                cut = shorter(cut, cut_among(s, wt, lo, hi, Pair{0, 0}, Want{true, 0, want}, true, reached, each));
                if (reached < want + slack) return deep();
            } else if (want <= total || low < hot) {
                return deep();
            }
        }
        clear_flags();
        const uint32_t per = (n + kBlock - 1) / kBlock, from = min(tid * per, n), to = min(from + per, n);
        Pair mine{0, 0};
        for (uint32_t i = from; i < to; ++i) mine.n += key_of(val_s[i]) == cut.key;
        uint32_t tie = block_before(s, mine, all).n;
        for (uint32_t i = from; i < to; ++i) {
            const uint32_t key = key_of(val_s[i]);
            if (key > cut.key || (key == cut.key && tie < cut.ties)) flag(i);
            tie += key == cut.key;
        }
    }
    // ---- what is kept, in the order of ids
    __syncthreads();
    const uint32_t per = (n + kBlock - 1) / kBlock, from = min(tid * per, n), to = min(from + per, n);
    auto kept = [&](uint32_t i) { return s.count[i >> 5] >> (i & 31) & 1u; };
    Pair mine{0, 0}, all;
    for (uint32_t i = from; i < to; ++i)
        if (kept(i)) mine = mine + Pair{1, DRAW ? weight(wt, val_s[i]) : 0};
    Pair at = block_before(s, mine, all);
    if (tid == 0 && a.out_kept) a.out_kept[out] = (int32_t)all.n;
    rec.n = all.n;
    leave(kDone, false, false);
    if constexpr (DRAW) {
        const u64 target = (u64)((double)g.u * (double)all.w);
        if (at.w > target || at.w + mine.w <= target) return;
        for (uint32_t i = from; i < to; ++i) {
            if (!kept(i)) continue;
            at.w += weight(wt, val_s[i]);
            if (at.w > target) {
                a.out_tokens[out] = (int32_t)id_s[i];
                if (a.out_logq) a.out_logq[out] = log_share(wt, val_s[i], g.t, all.w);
                return;
            }
        }
    } else {
        for (uint32_t i = from; i < to; ++i) {
            if (!kept(i)) continue;
            // (candidates are read from shared memory alone by now)
            a.list[list + at.n++] = Listed{id_s[i], val_s[i]};
        }
    }
}

// ---------------------------------------------------------------------------
// second, third
// ---------------------------------------------------------------------------

__device__ __forceinline__ int deep_bin(double steps) {
    return max((int)(uint32_t)__double_as_longlong(steps) >> 4, 1 - kDeepBins) + kDeepBins - 1;
}

// Weights (DRAW) of the chunk's ids whose bits are set, per wave's load.
template <typename T>
__device__ __forceinline__ void sum_loads(const SampleArgs &a, int ri, int c, const Chunk<T> &k, uint32_t in, const Weights &wt) {
    constexpr int N = Row<T>::N, NB = Chunk<T>::NB;
    u64 *subs = a.subs + ((int64_t)ri * a.chunks + c) * (kChunk / 256) + (threadIdx.x >> 6) * NB;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        u64 sum = 0;
        if (__any(in >> (j * N) & ((1u << N) - 1u))) {
#pragma unroll
            for (int i = 0; i < N; ++i) sum += in >> (j * N + i) & 1u ? weight(wt, k.x(j, i)) : 0;
            sum = wave_sum_u64(sum);
        }
        if ((threadIdx.x & 63) == 0) subs[j] = sum;
    }
}

// Chunks of the rows that `finish` left.  Bound by fp64 instructions, 20 a weight: 256 rows
// with nothing cut, each id's weight, take 43 us; a few rows' histograms 9 us, by latency.
template <typename T, bool DRAW>
__global__ void __launch_bounds__(kBlock) second_kernel(SampleArgs a) {
    constexpr int N = Row<T>::N, NB = Chunk<T>::NB;
    __shared__ u64 hist_s[kDeepBins];
    __shared__ double table_s[kSteps];
    __shared__ uint32_t count_s[kWaves];
    const int tid = threadIdx.x;
    fill_table(table_s);
    const int items = (int)a.work->second * a.chunks;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int ri = (int)a.second[item / a.chunks], c = item % a.chunks;
        const Setting g = setting_of<DRAW>(a, a.row0 + ri);
        const RowRec rec = a.row[ri];
        const Row<T> row = row_of<T>(a.logits, (int64_t)(a.row0 + ri) * a.ld, a.V);
        const Weights wt = weights_of(rec.m, g.t, table_s);
        Chunk<T> k;
        load_chunk(row, c, k);
        __syncthreads();                        // (the item before is done with shared memory)
        if (rec.state == kWhole) {
            const float edge = of_key(rec.key);
            uint32_t in = 0;
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) in |= (k.x(j, i) >= edge ? 1u : 0u) << (j * N + i);
            if (DRAW) sum_loads(a, ri, c, k, in, wt);
            const uint32_t n = wave_sum_u32(__popc(in));
            if ((tid & 63) == 0) count_s[tid >> 6] = n;
            __syncthreads();
            if (tid == 0) {
                uint32_t all = 0;
                for (int v = 0; v < kWaves; ++v) all += count_s[v];
                a.chunk[(int64_t)ri * a.chunks + c].finite = all;
            }
        } else {
            for (int i = tid; i < kDeepBins; i += kBlock) hist_s[i] = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    double d;
                    const double steps = steps_of(wt, k.x(j, i), d);
                    const u64 w = rec.by_weight ? weight_at(wt, steps, d) : (u64)(k.x(j, i) > -INFINITY);
                    atomicAdd(&hist_s[deep_bin(steps)], w);
                }
            __syncthreads();
            u64 *h = a.hist + ((int64_t)ri * a.chunks + c) * kDeepBins;
            for (int i = tid; i < kDeepBins; i += kBlock) h[i] = hist_s[i];
        }
    }
}

// The least logit of bins `bin` and above (+infinity: none), by 64 keys at a time.
__device__ __forceinline__ float least_of_bin(const Weights &wt, int bin) {
    // keys lo - 1 and below lie lower, hi and above do not (hi: the largest logit's, or none)
    const uint32_t lane = threadIdx.x & 63, top = key_of((float)wt.m);
    if (bin >= kDeepBins) return INFINITY;
    uint32_t lo = kNoKey + 1, hi = top;
    while (hi > lo) {
        const uint32_t gap = (hi - lo) / 65 + 1, at = min(lo + lane * gap, hi);
        double d;
        const uint64_t below = __ballot(deep_bin(steps_of(wt, of_key(at), d)) < bin);
        const int n = __popcll(below);          // the first lanes: keys rise with them
        hi = n < 64 ? min(lo + n * gap, hi) : hi;
        lo = n ? min(lo + (n - 1) * gap, hi) + 1 : lo;
        if (n == 0) hi = lo;
    }
    return of_key(hi);
}

// The same chunks again where a cut is looked for.  Every workgroup adds the row's
// histograms up for itself (58 kB out of the caches), so that no launch for it comes
// between.  Bound by latency: a dozen rows of 151936 ids 11 us (12 with the histograms
// eight at a time and the rest one by one).
template <typename T, bool DRAW>
__global__ void __launch_bounds__(kBlock, 3) third_kernel(SampleArgs a) {
    constexpr int N = Row<T>::N, NB = Chunk<T>::NB;
    __shared__ u64 wave_s[kWaves], above_s;
    __shared__ int bin_s;
    __shared__ double table_s[kSteps];
    __shared__ uint32_t count_s[kWaves], above_n_s[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    fill_table(table_s);
    const int items = (int)a.work->third * a.chunks;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int ri = (int)a.third[item / a.chunks], c = item % a.chunks;
        const Setting g = setting_of<DRAW>(a, a.row0 + ri);
        const RowRec rec = a.row[ri];
        const Row<T> row = row_of<T>(a.logits, (int64_t)(a.row0 + ri) * a.ld, a.V);
        Chunk<T> k;
        load_chunk(row, c, k);
        // ---- the row's histogram, the highest bins in thread 0
        constexpr int E = (kDeepBins + kBlock - 1) / kBlock;
        const u64 *h = a.hist + (int64_t)ri * a.chunks * kDeepBins;
        u64 mine[E] = {}, sum = 0;
        const int b0 = max(kDeepBins - 1 - tid * E, 0), b1 = max(b0 - 1, 0);
        static_assert(E == 2, "two bins a thread");
        constexpr int LOADS = 10;               // chunks whose bins are under way
        for (int i0 = 0; i0 < a.chunks; i0 += LOADS) {
            u64 got[LOADS][E];
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const u64 *const of = h + min(i0 + i, a.chunks - 1) * kDeepBins;
                got[i][0] = of[b0];
                got[i][1] = of[b1];
            }
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                if (i0 + i >= a.chunks) continue;
                mine[0] += got[i][0];
                mine[1] += got[i][1];
            }
        }
        if (tid * E >= kDeepBins) mine[0] = mine[1] = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) sum += mine[e];
        const u64 inc = wave_scan_u64(sum);
        __syncthreads();                        // (the item before is done with shared memory)
        if (lane == 63) wave_s[wave] = inc;
        __syncthreads();
        u64 before = inc - sum, total = 0;
        for (int v = 0; v < kWaves; ++v) {
            if (v < wave) before += wave_s[v];
            total += wave_s[v];
        }
        const u64 want = rec.by_weight ? top_p_want(g.p, total).w : (u64)g.k;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (before < want && before + mine[e] >= want) {
                bin_s = kDeepBins - 1 - (tid * E + e);
                above_s = before;
            }
            before += mine[e];
        }
        __syncthreads();
        const int bin = bin_s;
        if (c == 0 && tid == 0) {
            DeepRec d;
            d.bin = bin;
            d.above = rec.by_weight ? Pair{0, above_s} : Pair{(uint32_t)above_s, 0};
            d.want = rec.by_weight ? Want{true, 0, want} : Want{false, (uint32_t)want, 0};
            a.deep[ri] = d;
        }
        const Weights wt = weights_of(rec.m, g.t, table_s);
        // ---- ids in it and above it, of those that min_p leaves: logits
        // from `edge` on, and from `over` on
        const float low = of_key(min_p_key(rec.m, g));
        const float edge = fmaxf(low, least_of_bin(wt, bin)), over = fmaxf(low, least_of_bin(wt, bin + 1));
        uint32_t hits = 0, above = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = k.x(j, i);
                hits |= (x >= edge ? 1u : 0u) << (j * N + i);
                above |= (x >= over ? 1u : 0u) << (j * N + i);
            }
        hits &= ~above;
        if (DRAW) sum_loads(a, ri, c, k, above, wt);
        const uint32_t n = wave_sum_u32(__popc(above));
        if (lane == 0) above_n_s[wave] = n;
        const uint32_t listed = list_hits(a, ri, c, row, k, hits, count_s);
        if (tid == 0) {
            ChunkRec &out = a.chunk[(int64_t)ri * a.chunks + c];
            out.finite = 0;
            for (int v = 0; v < kWaves; ++v) out.finite += above_n_s[v];
            out.n = listed;
        }
    }
}

// ---------------------------------------------------------------------------
// the last launches
// ---------------------------------------------------------------------------

template <typename T> __device__ __forceinline__ T masked();
template <> __device__ __forceinline__ float masked<float>() { return -INFINITY; }
template <> __device__ __forceinline__ uint16_t masked<uint16_t>() { return 0xff80; }
template <typename T> __device__ __forceinline__ T element_of(float x) {
    if constexpr (sizeof(T) == 2) return (T)(__float_as_uint(x) >> 16);
    else return x;
}

template <typename T> __device__ __forceinline__ void set_element(u32x4_t &w, int i, T e) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(e);
    else w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | (uint32_t)e << 16 : (w[i >> 1] & 0xffff0000u) | e;
}

template <typename T> struct RowShared {
    static constexpr int SUB = 64 * Row<T>::N;                // ids of a wave's load
    static constexpr int SUBS = SPEC_MAX_VERIFY_VOCAB / SUB + 1;
    static constexpr int EACH = (SUBS + kRowThreads - 1) / kRowThreads;
    Scratch<kRowThreads> s;
    float val[kInBin];           // candidates: logits,
    uint32_t id[kInBin];        // and ids
    u64 sub_w[SUBS];             // kept weight, per wave's load
    uint32_t sub_e[SUBS];        // ids at the cut's key
    uint32_t off[64];
    u64 at_w;                    // of the load that holds the drawn token: weight
    uint32_t at_e;               // and ties before it
    int at_sub;
};

// The exact cut of a kDeep row, from the ids listed in its bin; candidates
// and their tie ranks stay with the threads, n / kRowThreads neighbours each.
// False: more ids than a list holds.
struct Deep {
    Cut cut;
    uint32_t n, from, to;        // candidates; this thread's
    uint32_t tie;                // ties before its first
    uint32_t above;              // kept ids of higher bins
};
template <typename T>
__device__ __forceinline__ bool deep_cut(const SampleArgs &a, RowShared<T> &sh, int ri, const Setting &g,
                                         const RowRec &rec, const Records &r, const DeepRec &bin, const Weights &wt,
                                         Deep &d) {
    constexpr int B = kRowThreads;
    const int tid = threadIdx.x;
    if (r.full || r.n > (uint32_t)kInBin) return false;
    d.n = r.n;
    d.above = wave_sum_u32((tid & 63) < a.chunks ? r.rec.finite : 0u);
    if (tid < 64) sh.off[tid] = r.off;
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0;
    Pair sum{0, 0}, all;
    constexpr uint32_t E = 4;                   // loads under way
    for (uint32_t i0 = tid; i0 < d.n; i0 += E * B) {
        Listed l[E];
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) l[e] = a.list[place_of(a, ri, sh.off, min(i0 + e * B, d.n - 1))];
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) {
            if (i0 + e * B >= d.n) continue;
            sh.val[i0 + e * B] = l[e].x;
            sh.id[i0 + e * B] = l[e].id;
            lo = min(lo, key_of(l[e].x));
            hi = max(hi, key_of(l[e].x));
            sum = sum + Pair{1, bin.want.by_weight ? weight(wt, l[e].x) : 0};
        }
    }
    block_ends(sh.s, lo, hi);
    block_before(sh.s, sum, all);
    // (not reached where min_p left ids of the bin, or all of them, out: its cut is the shorter)
    d.cut = Cut{min_p_key(rec.m, g), 0xffffffffu};
    if (bin.want.reached(bin.above + all)) {
        u64 none;
        d.cut = shorter(d.cut, cut_among(sh.s, wt, lo, hi, bin.above, bin.want, bin.want.by_weight, none, [&](auto f) {
            for (uint32_t i = tid; i < d.n; i += B) f(key_of(sh.val[i]));
        }));
    }
    const uint32_t per = (d.n + B - 1) / B;
    d.from = min(tid * per, d.n);
    d.to = min(d.from + per, d.n);
    Pair mine{0, 0};
    for (uint32_t i = d.from; i < d.to; ++i) mine.n += key_of(sh.val[i]) == d.cut.key;
    d.tie = block_before(sh.s, mine, all).n;
    return true;
}

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

// Draws from the kept weights of sh.sub_w, a thread's loads being EACH tid on;
// the ties at the cut that each load holds stand in sh.sub_e.
template <typename T>
__device__ __forceinline__ void draw_row(const SampleArgs &a, RowShared<T> &sh, const Row<T> &row, const Weights &wt,
                                         const Setting &g, Cut cut, int64_t out) {
    constexpr int EACH = RowShared<T>::EACH;
    const int tid = threadIdx.x, subs = (row.blocks + 63) / 64;
    Pair mine[EACH], sum{0, 0}, all;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        mine[i] = sub < subs ? Pair{sh.sub_e[sub], sh.sub_w[sub]} : Pair{0, 0};
        sum = sum + mine[i];
    }
    Pair before = block_before(sh.s, sum, all);
    const u64 target = (u64)((double)g.u * (double)all.w);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (before.w <= target && before.w + mine[i].w > target) {
            sh.at_sub = tid * EACH + i;
            sh.at_w = before.w;
            sh.at_e = before.n;
        }
        before = before + mine[i];
    }
    __syncthreads();
    if (tid < 64) draw_in_load(a, sh, row, wt, g, cut, all.w, target, out);
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

// A whole row by one workgroup.
template <typename T, bool DRAW>
__device__ __forceinline__ void whole_row(const SampleArgs &a, RowShared<T> &sh, const Row<T> &row, const Setting &g,
                                          const RowRec &rec, const Weights &wt, int64_t out) {
    constexpr int N = Row<T>::N, B = kRowThreads, EACH = RowShared<T>::EACH;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Scratch<B> &s = sh.s;
    constexpr int kBins = Scratch<B>::kBins;
    uint32_t *const keys = (uint32_t *)sh.val;
    const Scale<kBins> scale(rec.m, g.t);
    __syncthreads();                                  // (the weights' table)
    Cut cut{kNoKey, 0};                               // every id with a finite logit
    // ---- the cut
    const bool few = g.k > 0 && (uint32_t)g.k < rec.finite;
    if (few || g.p < 1.f) {
        clear_bins(s);
        for_each_logit(row, [&](float x) {
            const int b = scale.bin(x);
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
                if (scale.bin(x) != bin) return;
                const uint32_t k = key_of(x);
                lo = min(lo, k);
                hi = max(hi, k);
                if (listed) keys[atomicAdd(&s.listed, 1u)] = k;  // (counted and summed alone: any order)
            });
            block_ends(s, lo, hi);
            if (listed)
                return cut_among(s, wt, lo, hi, above, want, g.p < 1.f, total, [&](auto f) {
                    for (uint32_t i = tid; i < there.n; i += B) f(keys[i]);
                });
            return cut_among(s, wt, lo, hi, above, want, g.p < 1.f, total, [&](auto f) {
                for_each_logit(row, [&](float x) {
                    if (scale.bin(x) == bin) f(key_of(x));
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
    cut = shorter(cut, Cut{min_p_key(rec.m, g), 0xffffffffu});
    // ---- what the cut leaves, per wave's load in the order of ids
    __syncthreads();
    const int subs = (row.blocks + 63) / 64;
    uint32_t *const sub_n = sh.id;
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
                sub_n[sub] = n & 0xffffu;
                sh.sub_e[sub] = n >> 16;
            }
        }
    }
    __syncthreads();
    // ---- thread i: its loads; the ties that are kept of each
    const u64 each = cut.ties ? weight(wt, of_key(cut.key)) : 0;
    Pair all;
    uint32_t eq[EACH], eq_sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        eq[i] = sub < subs ? sh.sub_e[sub] : 0u;
        eq_sum += eq[i];
    }
    uint32_t before = block_before(s, Pair{eq_sum, 0}, all).n;
    Pair kept{0, 0};
    uint32_t tie_at[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        tie_at[i] = before;
        const uint32_t in = min(before + eq[i], cut.ties) - min(before, cut.ties);
        if (sub < subs) {
            kept.n += sub_n[sub] + in;
            sh.sub_w[sub] += each * in;
        }
        before += eq[i];
    }
    block_before(s, kept, all);
    if (tid == 0 && a.out_kept) a.out_kept[out] = (int32_t)all.n;
    if constexpr (DRAW) {
        draw_row(a, sh, row, wt, g, cut, out);
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

// Tokens of the rows that are not done.  Bound by latency: 18 us for a dozen cuts
// with up to 2000 ids in the bin that holds them, 10 where nothing was cut.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) draw_kernel(SampleArgs a) {
    constexpr int PER = kChunk / RowShared<T>::SUB;    // loads of a chunk
    __shared__ RowShared<T> sh;
    const int tid = threadIdx.x, ri = blockIdx.x;
    const Setting g = setting_of<true>(a, a.row0 + ri);
    if (!g.live) return;
    const RowRec rec = a.row[ri];
    const Records r = records_of(a, ri);        // (both loaded before either is looked at)
    if (rec.state == kDone || rec.state == kFault) return;
    const DeepRec bin = a.deep[ri];             // (of kDeep rows alone)
    const int64_t out = a.row0 + ri;
    const Row<T> row = row_of<T>(a.logits, out * a.ld, a.V);
    const Weights wt = weights_of(rec.m, g.t, sh.s.table);
    fill_table(sh.s.table);
    const int subs = (row.blocks + 63) / 64;
    const u64 *in = a.subs + (int64_t)ri * a.chunks * (kChunk / 256);
    for (int i = tid; i < subs; i += kRowThreads) {
        sh.sub_w[i] = rec.state == kMany ? 0 : in[i / PER * (kChunk / 256) + i % PER];
        sh.sub_e[i] = 0;
    }
    __syncthreads();
    if (rec.state == kWhole) {
        if (g.mp > 0.f && a.out_kept && tid < 64) {
            const uint32_t n = wave_sum_u32(tid < a.chunks ? a.chunk[(int64_t)ri * a.chunks + tid].finite : 0u);
            if (tid == 0) a.out_kept[out] = (int32_t)n;
        }
        draw_row(a, sh, row, wt, g, Cut{rec.key, 0xffffffffu}, out);
        return;
    }
    Deep d;
    if (rec.state == kMany || !deep_cut(a, sh, ri, g, rec, r, bin, wt, d)) {
        __syncthreads();
        whole_row<T, true>(a, sh, row, g, rec, wt, out);
        return;
    }
    Pair mine{0, 0}, all;
    for (uint32_t i = d.from; i < d.to; ++i) {
        const uint32_t key = key_of(sh.val[i]);
        const int sub = (int)(sh.id[i] + row.skip) / RowShared<T>::SUB;
        if (key == d.cut.key) atomicAdd(&sh.sub_e[sub], 1u);
        if (key > d.cut.key || (key == d.cut.key && d.tie < d.cut.ties)) {
            atomicAdd(&sh.sub_w[sub], weight(wt, sh.val[i]));
            ++mine.n;
        }
        d.tie += key == d.cut.key;
    }
    block_before(sh.s, mine, all);
    if (tid == 0 && a.out_kept) a.out_kept[out] = (int32_t)(d.above + all.n);
    draw_row(a, sh, row, wt, g, d.cut, out);
}

// Cuts of truncated rows that are still to be found, for write_kernel; rows
// done whole.  14 us for a few rows, by latency.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) settle_kernel(SampleArgs a) {
    __shared__ RowShared<T> sh;
    const int tid = threadIdx.x, ri = blockIdx.x;
    const Setting g = setting_of<false>(a, a.row0 + ri);
    if (!g.live) return;
    RowRec rec = a.row[ri];
    const Records r = records_of(a, ri);
    const int64_t out = a.row0 + ri;
    if (rec.state == kWhole && g.mp > 0.f) {
        if (a.out_kept && tid < 64) {
            const uint32_t n = wave_sum_u32(tid < a.chunks ? a.chunk[(int64_t)ri * a.chunks + tid].finite : 0u);
            if (tid == 0) a.out_kept[out] = (int32_t)n;
        }
        return;
    }
    if (rec.state != kDeep && rec.state != kMany) return;
    const DeepRec bin = a.deep[ri];
    const Weights wt = weights_of(rec.m, g.t, sh.s.table);
    fill_table(sh.s.table);
    __syncthreads();
    Deep d;
    if (rec.state == kMany || !deep_cut(a, sh, ri, g, rec, r, bin, wt, d)) {
        __syncthreads();
        whole_row<T, false>(a, sh, row_of<T>(a.logits, out * a.ld, a.V), g, rec, wt, out);
        if (tid == 0) a.row[ri].state = kWritten;
        return;
    }
    Pair mine{0, 0}, all;
    uint32_t lo = 0xffffffffu, last = 0;
    for (uint32_t i = d.from; i < d.to; ++i) {
        const uint32_t key = key_of(sh.val[i]);
        if (key > d.cut.key || (key == d.cut.key && d.tie < d.cut.ties)) {
            ++mine.n;
            if (key == d.cut.key) last = sh.id[i];
        }
        d.tie += key == d.cut.key;
    }
    block_before(sh.s, mine, all);
    block_ends(sh.s, lo, last);
    if (tid) return;
    rec.state = kCut;
    rec.key = d.cut.key;
    // (min_p's cut may lie above the bin, and has no end)
    rec.last = d.cut.ties == 0xffffffffu ? 0xffffffffu : last;
    if (a.out_kept) a.out_kept[out] = (int32_t)(d.above + all.n);
    a.row[ri] = rec;
}

// Truncated rows: kWriteIds ids a workgroup.  Bound by HBM: 512 rows of 151936 bf16 ids,
// 156 MB written, 30.8 us, 5.1 TB/s.  (The rows that `finish` settled written beside
// the two launches after it, which wait more than they work: 129 to 132 us for the
// call against 128, those launches taking as much longer.)
template <typename T>
__global__ void __launch_bounds__(kRowThreads) write_kernel(SampleArgs a, int parts) {
    constexpr int N = Row<T>::N;
    const int tid = threadIdx.x, ri = blockIdx.x / parts, part = blockIdx.x - ri * parts;
    const Setting g = setting_of<false>(a, a.row0 + ri);
    if (!g.live) return;
    const RowRec rec = a.row[ri];
    if (rec.state == kWritten) return;
    const int64_t out = a.row0 + ri;
    // blocks of the output row; its first and last may be other rows' too
    const Row<T> row = row_of<T>(a.logits, out * a.ld, a.V), dst = row_of<T>(a.out_logits, out * a.out_ld, a.V);
    T *const to = (T *)dst.p;
    const int b0 = part * (kWriteIds / N), b1 = min(b0 + kWriteIds / N, dst.blocks);
    const bool copy = rec.state == kWhole || rec.state == kCut, alike = row.skip == dst.skip;
    if (copy && g.whole && row.p == dst.p && alike) return;  // in place
    const uint32_t nan = sizeof(T) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
    const uint32_t word = rec.state == kFault ? nan : Unpack<T>::kMasked;
    const uint32_t last = rec.state == kCut ? rec.last : 0xffffffffu;
    auto kept = [&](float x, int id) {
        const uint32_t k = key_of(x);
        return k > rec.key || (k == rec.key && (uint32_t)id <= last);
    };
    for (int b = b0 + tid; b < b1; b += kRowThreads) {
        const int id = b * N - dst.skip;
        const bool whole = id >= 0 && id + N <= a.V;
        u32x4_t w{word, word, word, word};
        if (copy) {
            if (whole && alike) w = *(const u32x4_t *)(row.p + (int64_t)b * N);
            else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (id + i >= 0 && id + i < a.V) set_element<T>(w, i, row.p[row.skip + id + i]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!kept(Unpack<T>::get(w, i), id + i)) set_element<T>(w, i, masked<T>());
        }
        if (whole) {
            *(u32x4_t *)(to + (int64_t)b * N) = w;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (id + i >= 0 && id + i < a.V) to[dst.skip + id + i] = element_of<T>(Unpack<T>::get(w, i));
        }
    }
    if (rec.state != kDone) return;
    __syncthreads();                            // kept ids go over what this workgroup has written
    const int64_t list = (int64_t)ri * a.chunks * a.room;
    for (uint32_t i = tid; i < rec.n; i += kRowThreads) {
        const Listed l = a.list[list + i];
        const int b = (int)(l.id + dst.skip) / N;
        if (b >= b0 && b < b1) to[dst.skip + l.id] = element_of<T>(l.x);
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

// Rows that share memory and are not the same rows.  (Rows that lie between each other's
// do not, as far as the same spacing shows it.)
static bool rows_overlap(const void *a, int64_t ld_a, const void *b, int64_t ld_b, int64_t rows, int64_t V, int64_t size) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    const uint64_t span_a = (uint64_t)((rows - 1) * ld_a + V) * size, span_b = (uint64_t)((rows - 1) * ld_b + V) * size;
    if (x + span_a <= y || y + span_b <= x) return false;
    if (rows > 1 && ld_a != ld_b) return true;
    if (x == y) return false;
    if (rows == 1) return true;
    const uint64_t step = (uint64_t)(ld_a * size), off = (x < y ? y - x : x - y) % step;
    return off < (uint64_t)(V * size) || step - off < (uint64_t)(V * size);
}

// A slice's memory.
struct Layout {
    int chunks, room, rows;      // of a row; candidates of a chunk; rows of a slice
    size_t chunk, row, deep, work, lists, hist, subs, list, bytes;
};
static Layout layout_of(int R, int J, int V) {
    Layout l;
    l.chunks = (V + 7 + kChunk - 1) / kChunk;   // (up to 7 elements before the row in its first block)
    // a chunk lists 512 ids at least, and a row as many as are taken: short
    // rows whole
    l.room = kListed / l.chunks;
    if (l.room < 512) l.room = 512;
    if (l.room > V) l.room = V;
    const int64_t rows = (int64_t)R * J;
    const int listed = kSliceListed / (l.chunks * l.room);
    l.rows = kSliceChunks / l.chunks;
    if (l.rows > listed) l.rows = listed;
    if (l.rows > rows) l.rows = (int)rows;
    const size_t n = (size_t)l.rows * l.chunks;
    size_t at = sizeof(Control);
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.work = take(sizeof(Work));
    l.chunk = take(n * sizeof(ChunkRec));
    l.row = take((size_t)l.rows * sizeof(RowRec));
    l.deep = take((size_t)l.rows * sizeof(DeepRec));
    l.lists = take((size_t)l.rows * 2 * sizeof(uint32_t));
    l.hist = take(n * kDeepBins * sizeof(u64));
    l.subs = take(n * (kChunk / 256) * sizeof(u64));
    l.list = take(n * l.room * sizeof(Listed));
    l.bytes = at;
    return l;
}

template <typename T, bool DRAW>
static void launch_rows(SampleArgs a, const Layout &l, hipStream_t st) {
    const int rows = a.R * a.J, parts = (a.V + 7 + kWriteIds - 1) / kWriteIds;
    for (a.row0 = 0; a.row0 < rows; a.row0 += l.rows) {
        a.rows_here = rows - a.row0 < l.rows ? rows - a.row0 : l.rows;
        const unsigned n = (unsigned)a.rows_here, c = n * (unsigned)l.chunks;
        const unsigned w = c < (unsigned)kListGroups ? c : (unsigned)kListGroups;
        hipLaunchKernelGGL((chunk_kernel<T>), dim3(c), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL((finish_kernel<T, DRAW>), dim3(n), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL((second_kernel<T, DRAW>), dim3(w), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL((third_kernel<T, DRAW>), dim3(w), dim3(kBlock), 0, st, a);
        if constexpr (DRAW) {
            hipLaunchKernelGGL((draw_kernel<T>), dim3(n), dim3(kRowThreads), 0, st, a);
        } else {
            hipLaunchKernelGGL((settle_kernel<T>), dim3(n), dim3(kRowThreads), 0, st, a);
            hipLaunchKernelGGL((write_kernel<T>), dim3(n * (unsigned)parts), dim3(kRowThreads), 0, st, a, parts);
        }
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
    a.work = (Work *)(ws + l.work);
    a.chunk = (ChunkRec *)(ws + l.chunk);
    a.row = (RowRec *)(ws + l.row);
    a.deep = (DeepRec *)(ws + l.deep);
    a.second = (uint32_t *)(ws + l.lists);
    a.third = a.second + l.rows;
    a.hist = (u64 *)(ws + l.hist);
    a.subs = (u64 *)(ws + l.subs);
    a.list = (Listed *)(ws + l.list);
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
    if (rows_overlap(logits, ld, out_logits, out_ld, (int64_t)R * J, V, dtype == SPEC_F32 ? 4 : 2)) return SPEC_EINVAL;
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
