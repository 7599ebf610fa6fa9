// sample.hip -- draws and rows under temperature, top-k, top-p and min-p on gfx950.
//
// Ids in order: logit descending, id ascending.  Each of the settings leaves a
// prefix of that order, and so does their intersection; it is kept as (key,
// ties): the ids whose logit lies above `key`, and the first `ties` that
// equal it.  Weights are whole numbers, w = rint(2^44 e^((x - m) / T)) with the
// row's largest logit m, summed in 64 bits: sums are exact, whatever order a
// launch takes them in, and so are the comparisons that a token hangs on.  (A
// row of 2^18 ids sums to 2^62 at most.)
#include <math.h>

#include "common.h"

namespace sv {

typedef unsigned long long u64;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRowThreads = 1024;             // threads of a row's workgroup
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBins = 2 * kRowThreads;        // of a histogram
constexpr int kListKeys = 2048;               // keys that are looked at one by one
constexpr double kOne = 17592186044416.0;     // 2^44, the weight of the largest logit
// Weights below half a unit are 0: from 45 log 2 = 31.2 temperatures below m on.
constexpr double kDeepest = 31.25;

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
// A block's logits; elements that are not the row's become -inf and are not read.
template <typename T>
__device__ __forceinline__ void load_block(const Row<T> &r, int b, float (&x)[Row<T>::N]) {
    constexpr int N = Row<T>::N;
    const int id = b * N - r.skip;
    if (id >= 0 && id + N <= r.V) {
        VecLoad<T, N>::run(r.p, (long)b * N, x);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = id + i >= 0 && id + i < r.V ? load_one(r.p, (long)b * N + i) : -INFINITY;
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

__device__ __forceinline__ u64 wave_sum_u64(u64 v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ u64 wave_scan_u64(u64 v) {
    for (int o = 1; o < 64; o <<= 1) {
        const u64 x = __shfl_up(v, o, 64);
        if ((int)(threadIdx.x & 63) >= o) v += x;
    }
    return v;
}

struct Scratch {
    u64 mass[kBins];             // a histogram: weights,
    uint32_t count[kBins];       // and ids
    uint32_t list[kListKeys];    // keys
    double table[64];
    Pair waves[kRowWaves];
    uint32_t ends[2][kRowWaves];
    uint32_t listed;
    uint32_t found;              // the bin of a cut,
    Pair before, there;          // what lies above it, and in it
};

// What lies in the threads before this one (in thread order), and in all.
__device__ __forceinline__ Pair block_before(Scratch &s, Pair v, Pair &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Pair inc{wave_incl_scan_dpp(v.n), wave_scan_u64(v.w)};
    __syncthreads();
    if (lane == 63) s.waves[wave] = inc;
    __syncthreads();
    Pair b{inc.n - v.n, inc.w - v.w};
    all = Pair{0, 0};
    for (int w = 0; w < kRowWaves; ++w) {
        if (w < wave) b = b + s.waves[w];
        all = all + s.waves[w];
    }
    return b;
}
__device__ __forceinline__ uint32_t block_max(Scratch &s, uint32_t v) {
    for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.ends[0][threadIdx.x >> 6] = v;
    __syncthreads();
    for (int w = 0; w < kRowWaves; ++w) v = max(v, s.ends[0][w]);
    return v;
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

// The histogram's bin (the highest first) in which `want` is reached, counted
// from `above` on; into s.found, s.before and s.there.
__device__ __forceinline__ void find_bin(Scratch &s, Pair above, const Want &want) {
    constexpr int EACH = kBins / kRowThreads;
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

__device__ __forceinline__ void clear_bins(Scratch &s) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kRowThreads) {
        s.mass[i] = 0;
        s.count[i] = 0;
    }
    __syncthreads();
}

// First histogram of a row: bins of equal width down to the deepest logit
// with a weight, and one for the rest; the highest bin holds the largest.  A
// function of the logit alone that does not rise where the logit falls.
struct Scale {
    float m, per;                // largest logit, bins per unit
};
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
    return kBins - 1 - (int)fminf((s.m - x) * s.per, (float)(kBins - 1));
}

template <typename T, typename F>
__device__ __forceinline__ void for_each_logit(const Row<T> &row, F f) {
    constexpr int N = Row<T>::N;
    for (int b = threadIdx.x; b < row.blocks; b += kRowThreads) {
        float x[N];
        load_block(row, b, x);
#pragma unroll
        for (int i = 0; i < N; ++i) f(x[i]);
    }
}

// The cut inside bin `bin` of the row's first histogram, with `above` before
// it and `there` in it.  Few keys go to a list, many are counted again from
// the row, over 2048 equal parts of their range until one key is left.
// masses: weights matter, be it for the sum up to the cut alone.
template <typename T>
__device__ __forceinline__ Cut cut_in_bin(Scratch &s, const Row<T> &row, const Scale &scale, const Weights &wt,
                                          int bin, Pair above, Pair there, const Want &want, bool masses,
                                          u64 &weight_to_cut) {
    const bool listed = there.n <= kListKeys;
    __syncthreads();
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
    uint32_t hi = 0, lo = 0xffffffffu;
    for_each_logit(row, [&](float x) {
        if (x > -INFINITY && bin_of(scale, x) == bin) {
            const uint32_t k = key_of(x);
            hi = max(hi, k);
            lo = min(lo, k);
            if (listed) s.list[atomicAdd(&s.listed, 1u)] = k;  // (counted and summed alone: any order)
        }
    });
    hi = block_max(s, hi);
    lo = ~block_max(s, ~lo);
    while (true) {
        if (hi == lo) {
            const u64 each = weight(wt, of_key(lo));
            Cut c{lo, 0};
            if (want.by_weight) c.ties = (uint32_t)((want.w - above.w + each - 1) / each);
            else c.ties = want.n - above.n;
            weight_to_cut = above.w + each * c.ties;
            return c;
        }
        const int shift = max(0, 21 - __clz((int)(hi - lo)));  // parts of 2^shift keys
        clear_bins(s);
        auto add = [&](uint32_t k) {
            if (k < lo || k > hi) return;
            const uint32_t b = (k - lo) >> shift;
            atomicAdd(&s.count[b], 1u);
            if (masses) atomicAdd(&s.mass[b], weight(wt, of_key(k)));
        };
        if (listed) {
            for (uint32_t i = threadIdx.x; i < there.n; i += kRowThreads) add(s.list[i]);
        } else {
            for_each_logit(row, [&](float x) {
                if (x > -INFINITY && bin_of(scale, x) == bin) add(key_of(x));
            });
        }
        find_bin(s, above, want);
        above = s.before;
        lo += s.found << shift;
        hi = min(hi, lo + ((1u << shift) - 1u));
        if (shift && s.there.n == 1) {
            // (one id: its key is the part's only one)
            uint32_t k = 0;
            if (listed) {
                for (uint32_t i = threadIdx.x; i < there.n; i += kRowThreads)
                    if (s.list[i] >= lo && s.list[i] <= hi) k = s.list[i];
            } else {
                for_each_logit(row, [&](float x) {
                    if (x > -INFINITY && bin_of(scale, x) == bin && key_of(x) >= lo && key_of(x) <= hi) k = key_of(x);
                });
            }
            hi = lo = block_max(s, k);
        }
    }
}

// ---------------------------------------------------------------------------
// the launch
// ---------------------------------------------------------------------------

// One workgroup a row.
template <typename T, bool DRAW>
__global__ void __launch_bounds__(kRowThreads) sample_kernel(SampleArgs a) {
    constexpr int N = Row<T>::N, SUB = 64 * N;        // ids of a wave's load
    constexpr int kSubs = SPEC_MAX_VERIFY_VOCAB / SUB + 1;
    __shared__ Scratch s;
    __shared__ u64 sub_w[kSubs];                      // weight above the cut, per wave's load
    __shared__ uint32_t sub_n[kSubs], sub_e[kSubs];   // ids above it, and at it
    __shared__ u64 at_w;
    __shared__ int at_sub;
    __shared__ uint32_t at_e;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = blockIdx.x / a.J, j = blockIdx.x - r * a.J;
    const int live = a.rows ? a.rows[r] : a.J;
    // ---- settings
    const float t = a.temperature[r];
    const int k = a.top_k ? a.top_k[r] : 0;
    const float p = a.top_p ? a.top_p[r] : 1.f, mp = a.min_p ? a.min_p[r] : 0.f;
    const float u = DRAW ? a.u[blockIdx.x] : 0.f;
    bool ok = live >= 0 && live <= a.J;
    if (ok && j >= live) return;
    ok = ok && (t == 0.f || (t >= 1e-30f && t <= 1e30f)) && p > 0.f && mp >= 0.f && mp <= 1.f;
    if (DRAW && t != 0.f) ok = ok && u >= 0.f && u < 1.f;
    const Row<T> row = row_of<T>(a.logits, (int64_t)blockIdx.x * a.ld, a.V);
    // ---- the largest logit
    Scale scale;
    uint32_t finite = 0, first = 0;
    {
        uint32_t top = 0;
        bool odd = false;
        if (ok)
            for_each_logit(row, [&](float x) {
                odd |= !(x < INFINITY);
                finite += x > -INFINITY;
                top = max(top, key_of(x));
            });
        ok = !__syncthreads_or(odd) && ok;
        top = block_max(s, top);
        ok = ok && top > kNoKey;
        scale.m = of_key(top);
    }
    const int64_t out = (int64_t)blockIdx.x;
    T *const dst = DRAW ? nullptr : (T *)a.out_logits + out * a.out_ld;
    if (!ok) {
        if (tid == 0) {
            if (DRAW) a.out_tokens[out] = -1;
            if (DRAW && a.out_logq) a.out_logq[out] = NAN;
            if (a.out_kept) a.out_kept[out] = -1;
            atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        }
        if constexpr (!DRAW)
            for (int i = tid; i < a.V; i += kRowThreads) dst[i] = sizeof(T) == 2 ? (T)0x7fc0 : (T)NAN;
        return;
    }
    // ---- the cut
    Weights wt;
    wt.m = (double)scale.m;
    wt.c = t == 0.f ? 0.0 : 64.0 * kLog2e / (double)t;
    wt.table = s.table;
    if (tid < 64) s.table[tid] = exp2((double)tid / 64);
    scale.per = t == 0.f ? 0.f : (float)((kBins - 1) / (kDeepest * (double)t));
    Cut cut{kNoKey, 0};                               // every id with a finite logit
    {
        Pair all;
        block_before(s, Pair{finite, 0}, all);
        finite = all.n;
    }
    if (t == 0.f) {
        cut = Cut{key_of(scale.m), 1};
    } else {
        const bool few = k > 0 && (uint32_t)k < finite;
        if (few || p < 1.f) {
            clear_bins(s);
            for_each_logit(row, [&](float x) {
                if (x > -INFINITY) {
                    const int b = bin_of(scale, x);
                    atomicAdd(&s.count[b], 1u);
                    if (p < 1.f) atomicAdd(&s.mass[b], weight(wt, x));
                }
            });
            __syncthreads();
            constexpr int EACH = kBins / kRowThreads;
            // (the bins are used again by the cuts)
            Pair bins[EACH], sum{0, 0}, all;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                bins[i] = Pair{s.count[tid * EACH + i], s.mass[tid * EACH + i]};
                sum = sum + bins[i];
            }
            block_before(s, sum, all);
            u64 total = all.w;
            if (few) {
                const Want want{false, (uint32_t)k, 0};
                find_bin(s, Pair{0, 0}, want);
                cut = cut_in_bin(s, row, scale, wt, (int)s.found, s.before, s.there, want, p < 1.f, total);
            }
            if (p < 1.f) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    s.count[tid * EACH + i] = bins[i].n;
                    s.mass[tid * EACH + i] = bins[i].w;
                }
                const Want want{true, 0, (u64)ceil((double)p * (double)total)};
                find_bin(s, Pair{0, 0}, want);
                const Cut c = cut_in_bin(s, row, scale, wt, (int)s.found, s.before, s.there, want, p < 1.f, total);
                cut = few ? shorter(cut, c) : c;
            }
        }
        if (mp > 0.f) {
            // the least logit x with e^((x - m) / T) >= min_p
            const double low = (double)scale.m + (double)t * log((double)mp);
            float x = (float)low;
            uint32_t kx = key_of(x);
            if ((double)x < low) ++kx;
            if (kx > kNoKey) cut = shorter(cut, Cut{kx, 0xffffffffu});
        }
    }
    // ---- what the cut leaves, per wave's load in the order of ids
    __syncthreads();
    const int subs = (row.blocks + 63) / 64;
    const float edge = of_key(cut.key);
    for (int sub = wave; sub < subs; sub += kRowWaves) {
        const int b = sub * 64 + lane;
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = -INFINITY;
        if (b < row.blocks) load_block(row, b, x);
        uint32_t above = 0, at = 0;
        u64 w = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            at += x[i] == edge;
            if (x[i] > edge) {
                ++above;
                if (DRAW) w += weight(wt, x[i]);
            }
        }
        const uint64_t n = wave_sum_u64((u64)at << 32 | above);
        if (DRAW) w = wave_sum_u64(w);
        if (lane == 0) {
            sub_w[sub] = w;
            sub_n[sub] = (uint32_t)n;
            sub_e[sub] = cut.key > kNoKey ? (uint32_t)(n >> 32) : 0u;
        }
    }
    __syncthreads();
    // ---- thread i: loads 2 i and 2 i + 1; ties before them, then weights
    constexpr int EACH = (kSubs + kRowThreads - 1) / kRowThreads;
    const u64 each = cut.ties ? weight(wt, edge) : 0;
    Pair all;
    uint32_t eq[EACH], eq_sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        eq[i] = sub < subs ? sub_e[sub] : 0u;
        eq_sum += eq[i];
    }
    uint32_t eq_before = block_before(s, Pair{eq_sum, 0}, all).n;
    const uint32_t ties = min(cut.ties, all.n);
    Pair mine[EACH], sum{0, 0};
    uint32_t tie_at[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int sub = tid * EACH + i;
        tie_at[i] = eq_before;
        const uint32_t in = min(eq_before + eq[i], ties) - min(eq_before, ties);
        mine[i] = sub < subs ? Pair{sub_n[sub] + in, sub_w[sub] + each * in} : Pair{0, 0};
        sum = sum + mine[i];
        eq_before += eq[i];
    }
    Pair before = block_before(s, sum, all);
    if (tid == 0 && a.out_kept) a.out_kept[out] = (int32_t)all.n;
    if constexpr (DRAW) {
        const u64 target = t == 0.f ? 0 : (u64)((double)u * (double)all.w);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if (before.w <= target && before.w + mine[i].w > target) {
                at_sub = tid * EACH + i;
                at_w = before.w;
                at_e = tie_at[i];
            }
            before = before + mine[i];
        }
        __syncthreads();
        if (wave) return;
        const int b = at_sub * 64 + lane;
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = -INFINITY;
        if (b < row.blocks) load_block(row, b, x);
        uint32_t at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) at += cut.key > kNoKey && x[i] == edge;
        uint32_t tie = at_e + wave_incl_scan_dpp(at) - at;
        u64 w[N], w_sum = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool equal = cut.key > kNoKey && x[i] == edge;
            w[i] = x[i] > edge || (equal && tie < ties) ? weight(wt, x[i]) : 0;
            tie += equal;
            w_sum += w[i];
        }
        u64 run = at_w + wave_scan_u64(w_sum) - w_sum;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (run <= target && run + w[i] > target) {
                a.out_tokens[out] = b * N + i - row.skip;
                if (a.out_logq)
                    a.out_logq[out] = t == 0.f ? 0.f : (float)(((double)x[i] - wt.m) / (double)t - log((double)all.w / kOne));
            }
            run += w[i];
        }
    } else {
        // the ties that each load may keep
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (tid * EACH + i < subs) sub_e[tid * EACH + i] = tie_at[i];
        __syncthreads();
        const bool some = ties != 0 || cut.key > kNoKey;
        for (int sub = wave; sub < subs; sub += kRowWaves) {
            const int b = sub * 64 + lane;
            float x[N];
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = -INFINITY;
            if (b < row.blocks) load_block(row, b, x);
            uint32_t at = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) at += some && x[i] == edge;
            uint32_t tie = sub_e[sub] + wave_incl_scan_dpp(at) - at;
            const int id = b * N - row.skip;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool equal = some && x[i] == edge;
                const bool in = x[i] > edge || (equal && tie < ties);
                tie += equal;
                if (id + i >= 0 && id + i < a.V) {
                    if constexpr (sizeof(T) == 2) dst[id + i] = in ? (T)(__float_as_uint(x[i]) >> 16) : (T)0xff80;
                    else dst[id + i] = in ? x[i] : -INFINITY;
                }
            }
        }
    }
}

static int check_rows(const void *logits, int dtype, int64_t ld, int R, int J, int V, const float *temperature,
                      const void *workspace, size_t workspace_bytes) {
    if (R < 0 || J < 0 || V < 1 || ld < V) return SPEC_EINVAL;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EDTYPE;
    if (V > SPEC_MAX_VERIFY_VOCAB || (int64_t)R * J >= 1 << 22) return SPEC_EUNSUPPORTED;
    if (R == 0 || J == 0) return SPEC_OK;
    if (!logits || !temperature) return SPEC_EINVAL;
    if ((uintptr_t)logits & (dtype == SPEC_F32 ? 3u : 1u)) return SPEC_EINVAL;
    if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < sizeof(Control)) return SPEC_EWORKSPACE;
    return SPEC_OK;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_sample_workspace_bytes(int R, int J, int V) {
    if (R < 0 || J < 0 || V < 1 || V > SPEC_MAX_VERIFY_VOCAB || (int64_t)R * J >= 1 << 22) return 0;
    return sizeof(Control);
}

int spec_sample(const void *logits, int dtype, int64_t ld, const float *temperature, const int32_t *top_k,
                const float *top_p, const float *min_p, const int32_t *rows, const float *u, int R, int J, int V,
                int32_t *out_tokens, float *out_logq, int32_t *out_kept, void *workspace, size_t workspace_bytes,
                void *stream) {
    const int bad = check_rows(logits, dtype, ld, R, J, V, temperature, workspace, workspace_bytes);
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
    a.ctl = (Control *)workspace;
    const dim3 grid((unsigned)(R * J));
    if (dtype == SPEC_F32) hipLaunchKernelGGL((sample_kernel<float, true>), grid, dim3(kRowThreads), 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL((sample_kernel<uint16_t, true>), grid, dim3(kRowThreads), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_truncate_logits(const void *logits, int dtype, int64_t ld, const float *temperature, const int32_t *top_k,
                         const float *top_p, const float *min_p, const int32_t *rows, int R, int J, int V,
                         void *out_logits, int64_t out_ld, int32_t *out_kept, void *workspace,
                         size_t workspace_bytes, void *stream) {
    const int bad = check_rows(logits, dtype, ld, R, J, V, temperature, workspace, workspace_bytes);
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
    a.ctl = (Control *)workspace;
    const dim3 grid((unsigned)(R * J));
    if (dtype == SPEC_F32) hipLaunchKernelGGL((sample_kernel<float, false>), grid, dim3(kRowThreads), 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL((sample_kernel<uint16_t, false>), grid, dim3(kRowThreads), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
