// sample.h -- rows of logits, whole-number weights, and cuts found by histograms:
// what the launches of sample.hip are made of (internal).
#pragma once

#include <math.h>

#include "common.h"

namespace sv {

typedef unsigned long long u64;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr double kOne = 17592186044416.0;     // 2^44, the weight of the largest logit
// Weights below half a unit are 0: from 45 log 2 = 31.2 temperatures below m on.
constexpr double kDeepest = 31.25;

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

// w(x) = 2^(44 + (x - m) log2(e) / T): the exponent is rounded to a 128th, whose
// power of two stands in a table, and the rest, at most ln 2 / 256 = 0.0027, goes through
// the exponential's series to the fourth power (the next term is 1.2e-15, a
// fiftieth of a unit; with the roundings a weight is within 0.025 units of its value before
// it is rounded, over 10^8 random logits, and one in a thousand is rounded the other way).
constexpr int kSteps = 128;
struct Weights {
    double m, c, least;          // the largest logit, 128 log2(e) / T, x - m of 2^-60 of its weight
    double k1, k2, k3, k4;       // (ln 2 / 128)^i / i!
    const double *table;         // 2^(44 + i / 128), i < 128 (shared memory)
};
// A constant in scalar registers, opaque to the compiler, which would write
// its 64 bits into vector registers before every use.
__device__ __forceinline__ double constant(double v) {
    asm volatile("" : "+s"(v));
    return v;
}
__device__ __forceinline__ Weights weights_of(float m, float t, const double *table) {
    constexpr double z = kLn2 / kSteps;
    const double c = kSteps * kLog2e / (double)t;
    return Weights{readlane_d((double)m, 0), readlane_d(c, 0), readlane_d(-60.0 * kSteps / c, 0), constant(z),
                   constant(z * z / 2), constant(z * z * z / 6), constant(z * z * z * z / 24), table};
}
__device__ __forceinline__ void fill_table(double *table) {
    for (int i = threadIdx.x; i < kSteps; i += blockDim.x) table[i] = kOne * exp2((double)i / kSteps);
}
// (x - m) log2(e) / T in 128ths, rounded: a whole number that does not rise where x falls.
constexpr double kRound = 6755399441055744.0;  // 1.5 2^52: adding it rounds to whole numbers
__device__ __forceinline__ double steps_of(const Weights &w, float x, double &d) {
    d = fmax((double)x - w.m, w.least);
    return fma(d, w.c, kRound);
}
__device__ __forceinline__ u64 weight_at(const Weights &w, double s, double d) {
    const int n = (int)(uint32_t)__double_as_longlong(s);
    const double r = fma(d, w.c, -(s - kRound));
    double p = fma(r, w.k4, w.k3);
    p = fma(p, r, w.k2);
    p = fma(p, r, w.k1);
    p = fma(p, r, 1.0);
    p = ldexp(p * w.table[n & (kSteps - 1)], n >> 7) + kRound;
    const u64 bits = (u64)__double_as_longlong(p);
    return (u64)((uint32_t)(bits >> 32) - 0x43380000u) << 32 | (uint32_t)bits;  // (less kRound's)
}
__device__ __forceinline__ u64 weight(const Weights &w, float x) {
    double d;
    const double s = steps_of(w, x, d);
    return weight_at(w, s, d);
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
    static constexpr int kLog = B > 256 ? 11 : 10, kBins = 1 << kLog;
    u64 mass[kBins];             // a histogram: weights,
    uint32_t count[kBins];       // and ids
    double table[kSteps];
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
    constexpr int kBins = Scratch<B>::kBins, EACH = kBins / B;
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
    for (int i = threadIdx.x; i < Scratch<B>::kBins; i += B) {
        s.mass[i] = 0;
        s.count[i] = 0;
    }
    __syncthreads();
}

// The cut among keys lo .. hi, with `above` before them and `want` reached in
// them: counts over equal parts of the range, and again over the part that
// holds the cut, until it is one key.  each(f) calls f for the keys
// (others among them are passed over); masses: weights matter, be it for the
// sum up to the cut alone, which goes to weight_to_cut.
template <int B, typename F>
__device__ __forceinline__ Cut cut_among(Scratch<B> &s, const Weights &wt, uint32_t lo, uint32_t hi, Pair above,
                                         const Want &want, bool masses, u64 &weight_to_cut, F each) {
    for (int level = 0; level < 4 && hi != lo; ++level) {  // (4 times 10 bits are 32)
        const int shift = max(0, 32 - Scratch<B>::kLog - __clz((int)(hi - lo)));  // parts of 2^shift keys
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
        if (shift) {                            // (often one key's, or nearly)
            uint32_t l = 0xffffffffu, h = 0;
            each([&](uint32_t k) {
                if (k < lo || k > hi) return;
                l = min(l, k);
                h = max(h, k);
            });
            block_ends(s, l, h);
            lo = l;
            hi = h;
        }
    }
    const u64 one = weight(wt, of_key(lo));
    Cut c{lo, 0};
    if (want.by_weight) c.ties = (uint32_t)((want.w - above.w + one - 1) / one);
    else c.ties = want.n - above.n;
    weight_to_cut = above.w + one * c.ties;
    return c;
}

// Histograms of a row's logits: BINS bins of equal width down to the deepest
// logit with a weight (the lowest bin holds the rest, the highest the largest).
// A function of the logit alone that does not rise where the logit falls.
template <int BINS> struct Scale {
    float m, per;                // largest logit, bins per unit
    __device__ __forceinline__ Scale(float m, float t) : m(m), per((float)((BINS - 1) / (kDeepest * (double)t))) {}
    __device__ __forceinline__ int bin(float x) const {
        return BINS - 1 - (int)fminf((m - x) * per, (float)(BINS - 1));
    }
};

}  // namespace sv
