// page_select.hip -- key bounds of cache pages and the choice of pages that a
// drafting step attends to, on gfx950.
//
// lo_d and hi_d are the least and the largest value of key dimension d in a
// page of one key head.  For any query q and key k of the page q . k is at
// most sum_d max(q_d lo_d, q_d hi_d), and summed over the query rows that share
// the key head (nodes, and heads of the group) that is
//   score = sum_d U_d hi_d + N_d lo_d,  U = sum of max(q, 0), N of min(q, 0):
// two products a dimension whatever the number of rows.  (lo and hi are kept in bf16.
// Those of bf16 pages are values of theirs; those of e4m3 pages are rounded to nearest,
// and the score may lie below what it bounds by 2^-8 of its terms: it chooses
// pages, and outward rounding would double the bounds' error.)  Sums are in 64 bits:
// the products of bf16 values with U and N are close to exact there, so that
// which pages are chosen does not hang on the order of the sums.
#include "cache.h"
#include "page_cut.h"

namespace sv {

// ---------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------

struct BoundsArgs {
    Pages c;                     // (k only)
    const int32_t *start, *len;  // [R]
    int max_len;
    uint16_t *lo, *hi;           // [num_pages][heads][D] bf16
    Control *ctl;
};

// Least and largest of three, NaN if one is (v_minimum3, v_maximum3).
__device__ __forceinline__ float least(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float most(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Of a and the P-lane partner's a in lanes whose bit P is 0, of b in the others.
template <int P>
__device__ __forceinline__ float least_of_pair(float a, float b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    if constexpr (P == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        return least(__uint_as_float(r[0]), __uint_as_float(r[1]));
    } else {
        const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
        return least(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
}
constexpr int kDppRowRor4 = 0x124, kDppRowRor8 = 0x128;  // from lane i + 4, i + 8 of a row of 16

template <bool FP8> struct KeyVec;  // 16 bytes of one token's key
template <> struct KeyVec<false> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void run(u32x4_t w, float, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <> struct KeyVec<true> {
    static constexpr int N = 16;
    __device__ __forceinline__ static void run(u32x4_t w, float scale, float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            x[4 * i] = a[0] * scale;
            x[4 * i + 1] = a[1] * scale;
            x[4 * i + 2] = b[0] * scale;
            x[4 * i + 3] = b[1] * scale;
        }
    }
};

// One wave per page and head (SPLIT: the four waves of a workgroup divide the
// page's tokens).  A token's row is LPR lanes of 16 bytes; a lane keeps the
// bounds of its N dimensions over the tokens it meets, up to four loads at a time.
// Tokens behind the last one stand for it.  The lanes that hold the same dimensions are
// joined at the end: as all bounds are least values (largest ones negated), an
// exchange with the other half of the wave, then with the other row of 16, leaves each
// lane half of its values, then a quarter.  (By shuffles of all of them through shared
// memory the prompts below took 29.5 us, and e4m3 pages of 16 tokens 1.7 times as
// long.)  Bound by HBM: 8 prompts of up to 12 k tokens, 110 MB of e4m3 keys, scales and
// bounds, 22 us, 5 TB/s; a step's few pages by latency, 3.4 us.
constexpr int kBoundLoads = 4;

template <bool FP8, int D, bool SPLIT>
__global__ void __launch_bounds__(kBlock) bounds_kernel(BoundsArgs a) {
    typedef KeyVec<FP8> V;
    constexpr int N = V::N, LPR = D / N, TPL = 64 / LPR;  // lanes a row, tokens a load
    __shared__ float join_s[SPLIT ? kWaves : 1][2][SPLIT ? D : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = blockIdx.y;
    const int start = a.start[r], len = a.len[r];
    const int64_t unit = SPLIT ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kWaves + wave;
    if (len < 0 || len > a.max_len || !in_table(start, len, a.c.max_pages, a.c.shift)) {
        if (tid == 0 && blockIdx.x == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        return;
    }
    if (len == 0) return;
    const int index = (start >> a.c.shift) + (int)(unit / a.c.heads), h = (int)(unit % a.c.heads);
    if (index > (start + len - 1) >> a.c.shift) return;
    const int page = a.c.table[(int64_t)r * a.c.max_pages + index];
    if ((unsigned)page >= (unsigned)a.c.num_pages) {
        if (lane == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        return;
    }
    const int last = min(start + len - 1 - (index << a.c.shift), a.c.size - 1);  // in the page
    const int64_t row = ((int64_t)page * a.c.heads + h) * a.c.size;
    const int sub = lane % LPR, grp = lane / LPR;
    const char *k = (const char *)a.c.k + (row * D) * (FP8 ? 1 : 2) + sub * 16;
    float lo[N], hi[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        lo[i] = INFINITY;
        hi[i] = -INFINITY;
    }
    for (int t = (SPLIT ? wave * TPL * kBoundLoads : 0); t <= last; t += (SPLIT ? kWaves : 1) * TPL * kBoundLoads) {
        u32x4_t w[kBoundLoads];
        float sc[kBoundLoads];
#pragma unroll
        for (int i = 0; i < kBoundLoads; ++i) {
            if (!SPLIT && t + i * TPL > last) continue;
            const int tok = min(t + i * TPL + grp, last);
            w[i] = *(const u32x4_t *)(k + tok * (D * (FP8 ? 1 : 2)));
            sc[i] = FP8 ? a.c.k_scale[row + tok] : 1.f;
        }
#pragma unroll
        for (int i = 0; i < kBoundLoads; ++i) {
            if (!SPLIT && t + i * TPL > last) continue;
            float x[N];
            V::run(w[i], sc[i], x);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                lo[j] = least(lo[j], x[j]);
                hi[j] = most(hi[j], x[j]);
            }
        }
    }
    // ---- lanes 0 .. 31 go on with the least values, the others with the largest
    constexpr int C = LPR <= 16 ? N / 2 : N;    // of a row: its first or second half
#pragma unroll
    for (int j = 0; j < N; ++j) lo[j] = least_of_pair<32>(lo[j], -hi[j]);
    if constexpr (LPR <= 16) {
#pragma unroll
        for (int j = 0; j < C; ++j) lo[j] = least_of_pair<16>(lo[j], lo[j + C]);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
        if constexpr (LPR <= 8) lo[j] = least(lo[j], dpp_f<kDppRowRor8>(lo[j]));
        if constexpr (LPR <= 4) lo[j] = least(lo[j], dpp_f<kDppRowRor4>(lo[j]));
    }
    const int largest = lane >> 5, at = sub * N + (LPR <= 16 ? (lane >> 4 & 1) * C : 0);
    if constexpr (SPLIT) {
#pragma unroll
        for (int j = 0; j < C; ++j) join_s[wave][largest][at + j] = lo[j];  // (the same from every lane that has it)
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int w = 1; w < kWaves; ++w) lo[j] = least(lo[j], join_s[w][largest][at + j]);
    }
    if (LPR < 16 && (lane & 15) >= LPR) return;
    uint16_t *out = (largest ? a.hi : a.lo) + ((int64_t)page * a.c.heads + h) * D + at;
    const float sign = largest ? -1.f : 1.f;
    uint32_t w[C / 2];
#pragma unroll
    for (int j = 0; j < C; j += 2) w[j / 2] = pack_bf16(lo[j] * sign, lo[j + 1] * sign);
    if constexpr (C == 8) *(u32x4_t *)out = u32x4_t{w[0], w[1], w[2], w[3]};
    else *(uint2 *)out = uint2{w[0], w[1]};
}

// A workgroup's waves divide a page where it holds more than two rounds of one
// wave's loads (8 prompts of 4096 tokens, 8 heads of 128, a wave a page against four:
// e4m3 pages of 64 tokens, two rounds, 9.2 against 12.1 us, of 128 9.6 against 8.7, of
// 1024 31.5 against 10.1; bf16 of 32 13.0 against 13.5, of 64 13.8 against 12.3, of 1024
// 40.8 against 12.3).
template <bool FP8, int D>
static void launch_bounds(const BoundsArgs &a, int64_t units, int R, hipStream_t st) {
    constexpr int round = 64 / (D / KeyVec<FP8>::N) * kBoundLoads;
    if (a.c.size > 2 * round)
        hipLaunchKernelGGL((bounds_kernel<FP8, D, true>), dim3((unsigned)units, (unsigned)R), dim3(kBlock), 0, st, a);
    else
        hipLaunchKernelGGL((bounds_kernel<FP8, D, false>), dim3((unsigned)((units + kWaves - 1) / kWaves), (unsigned)R),
                           dim3(kBlock), 0, st, a);
}
template <bool FP8>
static void launch_bounds(const BoundsArgs &a, int D, int64_t units, int R, hipStream_t st) {
    if (D == 64) launch_bounds<FP8, 64>(a, units, R, st);
    else if (D == 128) launch_bounds<FP8, 128>(a, units, R, st);
    else launch_bounds<FP8, 256>(a, units, R, st);
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------

struct SelectArgs {
    const uint16_t *q;           // [R][M][Hq][D] bf16
    const uint16_t *lo, *hi;     // [num_pages][heads][D] bf16
    const int32_t *table;        // [R][max_pages]
    const int32_t *ctx_len, *n_nodes;
    int num_pages, max_pages, heads, shift;
    int M, Hq, G;
    int budget, first, last;
    int32_t *lists, *list_len;   // [R][heads][width], [R]
    int width;
    double *sums;                // [R][heads][2][D] U and N
    uint64_t *keys;              // [R][heads][max_pages] ordered scores
    Control *ctl;
};

struct Context {
    int n, ctx, full, take;      // full pages of context, of which `take` are listed
    bool ok;
};
__device__ __forceinline__ Context context_of(const SelectArgs &a, int r) {
    Context c;
    c.n = a.n_nodes[r];
    c.ctx = a.ctx_len[r];
    c.ok = c.n >= 0 && c.n <= a.M && in_table(c.ctx, c.n, a.max_pages, a.shift);
    c.full = c.ok && c.n ? c.ctx >> a.shift : 0;
    c.take = min(c.full, a.budget);
    return c;
}

// U and N of one request and key head.  (A launch of its own: sums that every wave of
// the score launch makes for itself took 41.8 against 33.5 us for 32 requests of 16 k
// tokens and 4 query rows a head, 72 against 33.6 for 16 rows; 15.5 against 16.1 for
// one request of 32 k tokens and 4 rows.)
template <int D>
__global__ void __launch_bounds__(kBlock) query_sums_kernel(SelectArgs a) {
    constexpr int LPR = D / 8, GRP = kBlock / LPR;
    __shared__ double part[GRP][2][D];
    const int tid = threadIdx.x, sub = tid % LPR, grp = tid / LPR, h = blockIdx.x, r = blockIdx.y;
    const Context c = context_of(a, r);
    if (c.full <= a.budget) return;
    double up[8], dn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = dn[i] = 0.0;
    for (int i = grp; i < c.n * a.G; i += GRP) {
        const int node = i / a.G;
        const uint16_t *row = a.q + (((int64_t)r * a.M + node) * a.Hq + h * a.G + (i - node * a.G)) * D;
        const u32x4_t w = *(const u32x4_t *)(row + sub * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {           // (a NaN goes to both)
            const float x = j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
            up[j] += (double)most(x, 0.f);
            dn[j] += (double)least(x, 0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        part[grp][0][sub * 8 + i] = up[i];
        part[grp][1][sub * 8 + i] = dn[i];
    }
    __syncthreads();
    for (int d = tid; d < 2 * D; d += kBlock) {
        double s = 0.0;
        for (int g = 0; g < GRP; ++g) s += part[g][d / D][d % D];
        a.sums[((int64_t)r * a.heads + h) * 2 * D + d] = s;
    }
}

// Sum over LANES neighbours, the same in each of them.
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
    v += dpp_d<kDppSwap1>(v);
    v += dpp_d<kDppSwap2>(v);
    v += dpp_d<kDppHalfMirror>(v);
    if constexpr (LANES >= 16) v += dpp_d<kDppMirror>(v);
    if constexpr (LANES >= 32) {
        const long long b = __double_as_longlong(v);
        uint32_t l0, l1, h0, h1;
        lane_pair<16>((uint32_t)(b & 0xffffffffLL), l0, l1);
        lane_pair<16>((uint32_t)(b >> 32), h0, h1);
        v = __longlong_as_double((long long)((uint64_t)h0 << 32 | l0)) +
            __longlong_as_double((long long)((uint64_t)h1 << 32 | l1));
    }
    return v;
}

// A score as a whole number in the same order; NaN stands with +infinity, for
// a page that could hold anything.
__device__ __forceinline__ uint64_t key_of(double s) {
    s = s != s ? (double)INFINITY : s + 0.0;  // (-0 becomes 0)
    const uint64_t b = (uint64_t)__double_as_longlong(s);
    return b >> 63 ? ~b : b | 1ull << 63;
}

// Scores of a request's full pages.  A page's bounds, all key heads of them,
// lie side by side: SPAN lanes take 8 values each of them (the launch's y axis goes
// over rows of more than 64 lanes), so that a wave reads pieces of up to a
// kilobyte; D / 8 lanes share a head.  The largest values go with U, then the
// least with N: one of the two sums is in registers at a time.  Bound by HBM:
// 171 MB of bounds (64 requests of up to 16 k tokens, 8 heads of 128, 16-token pages) in
// 26.7 us.  Two pages of one head a lane pair and eight loads a side took longer (80 us
// for the call against 58, and 44 us for this launch against 42, where each wave still
// summed its queries).
constexpr int kScoreLoads = 4;      // of 16 bytes a lane and side, all under way

// U (or, LEAST, N) of this lane's 8 dimensions.
template <int D, bool LEAST>
__device__ __forceinline__ void query_sums(const SelectArgs &a, int r, int h, int sub, double (&q)[8]) {
    const double *s = a.sums + ((int64_t)r * a.heads + h) * 2 * D + (LEAST ? D : 0) + sub * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s[i];
}

template <int D, int SPAN>
__global__ void __launch_bounds__(kBlock) score_kernel(SelectArgs a) {
    constexpr int PPL = 64 / SPAN;              // pages a load
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = blockIdx.z;
    const Context c = context_of(a, r);
    const int first = (blockIdx.x * kWaves + wave) * (kScoreLoads * PPL), p0 = first + lane / SPAN;
    if (c.full <= a.budget || first >= c.full) return;
    const int at = blockIdx.y * 512 + lane % SPAN * 8;      // value of a page's row
    const bool in = at < a.heads * D;
    const int h = in ? at / D : 0, sub = in ? at % D / 8 : 0;
    int page[kScoreLoads];
#pragma unroll
    for (int t = 0; t < kScoreLoads; ++t)
        page[t] = a.table[(int64_t)r * a.max_pages + min(p0 + t * PPL, c.full - 1)];
    u32x4_t hi[kScoreLoads], lo[kScoreLoads];
    uint32_t bad = 0;
#pragma unroll
    for (int t = 0; t < kScoreLoads; ++t) {
        if ((unsigned)page[t] >= (unsigned)a.num_pages) {
            bad |= 1u << t;                     // (the request is a faulty one: see select_kernel)
            page[t] = 0;
        }
        const int64_t e = ((int64_t)page[t] * a.heads + h) * D + sub * 8;
        hi[t] = *(const u32x4_t *)(a.hi + e);
        lo[t] = *(const u32x4_t *)(a.lo + e);
    }
    double s[kScoreLoads], q[8];
    auto add = [&](const u32x4_t (&x)[kScoreLoads]) {
#pragma unroll
        for (int t = 0; t < kScoreLoads; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[t] = fma(q[i], (double)(i & 1 ? bf16_hi(x[t][i >> 1]) : bf16_lo(x[t][i >> 1])), s[t]);
    };
#pragma unroll
    for (int t = 0; t < kScoreLoads; ++t) s[t] = 0.0;
    query_sums<D, false>(a, r, h, sub, q);
    add(hi);
    query_sums<D, true>(a, r, h, sub, q);
    add(lo);
    uint64_t *keys = a.keys + ((int64_t)r * a.heads + h) * a.max_pages;
#pragma unroll
    for (int t = 0; t < kScoreLoads; ++t) {
        const double sum = lanes_sum<D / 8>(s[t]);
        const int p = p0 + t * PPL;
        if (in && sub == 0 && p < c.full) keys[p] = bad >> t & 1u ? 0ull : key_of(sum);
    }
}

// Sum over the workgroup and prefix before this thread, of two counts in one
// word's halves (each total below 2^32).
__device__ __forceinline__ uint64_t block_prefix(uint64_t v, uint64_t (&wave_s)[kWaves], uint64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t lo = wave_incl_scan_dpp((uint32_t)v), hi = wave_incl_scan_dpp((uint32_t)(v >> 32));
    const uint64_t inc = (uint64_t)hi << 32 | lo;
    __syncthreads();
    if (lane == 63) wave_s[wave] = inc;
    __syncthreads();
    uint64_t before = inc - v;
    total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += wave_s[w];
        total += wave_s[w];
    }
    return before;
}

// (min and max of unlike 64-bit types are taken as doubles, which round.)
__device__ __forceinline__ uint64_t lower(uint64_t a, uint64_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint64_t higher(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The best pages of one request and key head, and its list.  The cut is found
// by counts over 2048 equal parts of the keys' range, and again over the part that
// holds it (page_cut.h; of one key the lowest pages that have it are taken).  Keys of
// up to kHeldKeys pages stay in shared memory.  Bound by latency: a handful of
// dependent passes over a few keys a thread (10.4 us for eight lists of 1875 pages, 9.2 for 512 of up to 1000).
constexpr int kHeldKeys = 4096;

__global__ void __launch_bounds__(kBlock) select_kernel(SelectArgs a) {
    __shared__ uint64_t held[kHeldKeys];
    __shared__ uint32_t count_s[kParts];
    __shared__ uint64_t wave_s[kWaves], cut_s[2], ends_s[2][kWaves];
    const int tid = threadIdx.x, h = blockIdx.x, r = blockIdx.y;
    const Context c = context_of(a, r);
    const int32_t *table = a.table + (int64_t)r * a.max_pages;
    int32_t *list = a.lists + ((int64_t)r * a.heads + h) * a.width;
    // pages of the request's tokens, the nodes' among them
    const int pages = c.ok && c.n ? (int)(((int64_t)c.ctx + c.n - 1) >> a.shift) + 1 : 0;
    const int from = a.first, to = c.full - a.last;  // pages that compete
    const uint64_t *keys = a.keys + ((int64_t)r * a.heads + h) * a.max_pages;
    const bool choose = c.full > a.budget;
    const bool in_lds = c.full <= kHeldKeys;
    bool ok = c.ok;
    uint64_t lo = ~0ull, hi = 0ull;
    constexpr int E = 8;                             // loads under way
    for (int p0 = tid; p0 < pages; p0 += E * kBlock) {
        int page[E];
        uint64_t k[E];
#pragma unroll
        for (int e = 0; e < E; ++e) page[e] = table[min(p0 + e * kBlock, pages - 1)];
        if (choose) {
#pragma unroll
            for (int e = 0; e < E; ++e) k[e] = keys[min(p0 + e * kBlock, c.full - 1)];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int p = p0 + e * kBlock;
            ok = ok && (unsigned)page[e] < (unsigned)a.num_pages;
            if (!choose || p < from || p >= to) continue;
            if (in_lds) held[p] = k[e];
            lo = lower(lo, k[e]);
            hi = higher(hi, k[e]);
        }
    }
    ok = __syncthreads_and(ok);
    if (!ok) {
        for (int i = tid; i < a.width; i += kBlock) list[i] = -1;
        if (tid == 0 && h == 0) {
            a.list_len[r] = -1;
            atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        }
        return;
    }
    // ---- the cut: keys above `cut` are taken, and the first `ties` that equal it
    uint64_t cut = 0;
    uint32_t ties = 0xffffffffu;
    auto key = [&](int p) -> uint64_t { return in_lds ? held[p] : keys[p]; };
    if (choose) {
        for (int o = 32; o; o >>= 1) {
            lo = lower(lo, __shfl_xor((unsigned long long)lo, o, 64));
            hi = higher(hi, __shfl_xor((unsigned long long)hi, o, 64));
        }
        if ((tid & 63) == 0) {
            ends_s[0][tid >> 6] = lo;
            ends_s[1][tid >> 6] = hi;
        }
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) {
            lo = lower(lo, ends_s[0][w]);
            hi = higher(hi, ends_s[1][w]);
        }
        const uint32_t want = (uint32_t)(a.budget - a.first - a.last);
        if (want == 0) {
            cut = ~0ull;  // above every key: +infinity's is below
        } else {
            const KeyCut found = key_cut(lo, hi, want, [&](uint64_t lo, uint64_t hi, int shift, uint32_t want) {
                for (int i = tid; i < kParts; i += kBlock) count_s[i] = 0u;
                __syncthreads();
                for (int p = from + tid; p < to; p += kBlock) {
                    const uint64_t k = key(p);
                    if (k >= lo && k <= hi) atomicAdd(&count_s[(k - lo) >> shift], 1u);
                }
                __syncthreads();
                // thread tid sums its parts, the highest first
                constexpr int EACH = kParts / kBlock;
                uint32_t mine[EACH], sum = 0;
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    mine[i] = count_s[kParts - 1 - (tid * EACH + i)];
                    sum += mine[i];
                }
                uint64_t total;
                uint32_t before = (uint32_t)block_prefix(sum, wave_s, total);
                if (before < want && before + sum >= want) {
#pragma unroll
                    for (int i = 0; i < EACH; ++i) {
                        if (before < want && before + mine[i] >= want) {
                            cut_s[0] = (uint64_t)(kParts - 1 - (tid * EACH + i));
                            cut_s[1] = (uint64_t)mine[i] << 32 | (want - before);
                        }
                        before += mine[i];
                    }
                }
                __syncthreads();
                const CutPart part{cut_s[0], (uint32_t)(cut_s[1] >> 32), (uint32_t)cut_s[1]};
                __syncthreads();
                return part;
            });
            cut = found.key;              // (above 0: no score's key is 0)
            ties = found.ties;
        }
    }
    // ---- the list, in the order of the context: a thread takes neighbouring pages
    const int each = (c.full + kBlock - 1) / kBlock;
    const int b = min(tid * each, c.full), e = min(b + each, c.full);
    uint32_t above = 0, equal = 0;
    for (int p = b; p < e; ++p) {
        if (!choose || p < from || p >= to) {
            ++above;
        } else {
            const uint64_t k = key(p);
            above += k > cut;
            equal += k == cut;
        }
    }
    uint64_t total;
    const uint64_t before = block_prefix((uint64_t)equal << 32 | above, wave_s, total);
    uint32_t tie = (uint32_t)(before >> 32);
    int at = (int)((uint32_t)before + min(tie, ties));
    for (int p = b; p < e; ++p) {
        bool in = true;
        if (choose && p >= from && p < to) {
            const uint64_t k = key(p);
            in = k > cut || (k == cut && tie < ties);
            tie += k == cut;
        }
        if (in && at < c.take) list[at++] = table[p];
    }
    const int tail = pages - c.full;
    for (int i = c.take + tid; i < a.width; i += kBlock)
        list[i] = i - c.take < tail ? table[c.full + i - c.take] : -1;
    if (tid == 0 && h == 0) a.list_len[r] = c.n ? (c.take << a.shift) + (c.ctx & ((1 << a.shift) - 1)) : 0;
}

template <int D>
static void launch_select(const SelectArgs &a, int R, hipStream_t st) {
    if (a.max_pages > a.budget) {
        hipLaunchKernelGGL((query_sums_kernel<D>), dim3((unsigned)a.heads, (unsigned)R), dim3(kBlock), 0, st, a);
        // lanes of a page's row, the next power of two
        const int64_t row = (int64_t)a.heads * D / 8;
        const int span = row <= D / 8 ? D / 8 : row <= 16 ? 16 : row <= 32 ? 32 : 64;
        const int per = kScoreLoads * (64 / span) * kWaves;
        const dim3 grid((unsigned)((a.max_pages + per - 1) / per), (unsigned)((row + 63) / 64), (unsigned)R);
        if constexpr (D == 64) {
            if (span == 8) hipLaunchKernelGGL((score_kernel<D, 8>), grid, dim3(kBlock), 0, st, a);
        }
        if constexpr (D <= 128) {
            if (span == 16) hipLaunchKernelGGL((score_kernel<D, 16>), grid, dim3(kBlock), 0, st, a);
        }
        if (span == 32) hipLaunchKernelGGL((score_kernel<D, 32>), grid, dim3(kBlock), 0, st, a);
        if (span == 64) hipLaunchKernelGGL((score_kernel<D, 64>), grid, dim3(kBlock), 0, st, a);
    }
    hipLaunchKernelGGL(select_kernel, dim3((unsigned)a.heads, (unsigned)R), dim3(kBlock), 0, st, a);
}

}  // namespace sv

using namespace sv;

extern "C" {

int spec_page_bounds(const void *k_cache, int cache_dtype, const float *k_scale, int num_pages,
                     int page_size, const int32_t *page_table, int max_pages, const int32_t *start,
                     const int32_t *len, int R, int max_len, int Hkv, int D, void *k_min,
                     void *k_max, void *workspace, size_t workspace_bytes, void *stream) {
    if (R < 0 || max_len < 0) return SPEC_EINVAL;
    const int bad = check_pages(k_cache, k_cache, cache_dtype, k_scale, k_scale, num_pages,
                                page_size, max_pages, Hkv, D);
    if (bad) return bad;
    if (R > 65535) return SPEC_EUNSUPPORTED;
    // pages that max_len tokens can lie in, whatever the first one's place is
    int64_t units = max_len ? ((int64_t)max_len + page_size - 2) / page_size + 1 : 0;
    if (units > max_pages) units = max_pages;
    if (units > (int64_t)0x7fffffff / Hkv) return SPEC_EUNSUPPORTED;
    units *= Hkv;
    if (units >= kMaxBlocks) return SPEC_EUNSUPPORTED;
    if (R == 0 || max_len == 0) return SPEC_OK;
    if (!start || !len || !k_min || !k_max || (max_pages > 0 && !page_table)) return SPEC_EINVAL;
    if (((uintptr_t)k_min | (uintptr_t)k_max) & 15u) return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, sizeof(Control))) return SPEC_EWORKSPACE;
    BoundsArgs a{};
    a.c = make_pages(k_cache, nullptr, k_scale, nullptr, num_pages, page_size, page_table,
                     max_pages, Hkv);
    a.start = start;
    a.len = len;
    a.max_len = max_len;
    a.lo = (uint16_t *)k_min;
    a.hi = (uint16_t *)k_max;
    a.ctl = (Control *)workspace;
    if (units == 0) units = 1;  // (no table: every request with tokens is a faulty one)
    if (cache_dtype == SPEC_E4M3) launch_bounds<true>(a, D, units, R, (hipStream_t)stream);
    else launch_bounds<false>(a, D, units, R, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

size_t spec_page_select_workspace_bytes(int R, int Hkv, int D, int max_pages) {
    if (R < 0 || R > 65535 || Hkv < 1 || Hkv > 65535 || (D != 64 && D != 128 && D != 256) ||
        max_pages < 0)
        return 0;
    return sizeof(Control) + (size_t)R * Hkv * ((size_t)max_pages + 2 * (size_t)D) * sizeof(double);
}

int spec_page_select(const void *q, int q_dtype, const void *k_min, const void *k_max,
                     int num_pages, int page_size, const int32_t *page_table, int max_pages,
                     const int32_t *ctx_len, const int32_t *n_nodes, int budget, int first,
                     int last, int R, int M, int Hq, int Hkv, int D, int32_t *out_lists,
                     int list_pages, int32_t *out_len, void *workspace, size_t workspace_bytes,
                     void *stream) {
    if (R < 0 || M < 1 || Hq < 1 || budget < 0 || first < 0 || last < 0 ||
        (int64_t)first + last > budget)
        return SPEC_EINVAL;
    if (q_dtype != SPEC_BF16) return SPEC_EDTYPE;
    const int bad = check_pages(k_min, k_max, SPEC_BF16, nullptr, nullptr, num_pages, page_size,
                                max_pages, Hkv, D);
    if (bad) return bad;
    if (Hq % Hkv) return SPEC_EINVAL;
    const size_t need = spec_page_select_workspace_bytes(R, Hkv, D, max_pages);
    if (!need || M > SPEC_TREE_MAX_NODES || Hq / Hkv > 64) return SPEC_EUNSUPPORTED;
    // the chosen pages, and those that hold the context's end and the nodes
    if ((int64_t)list_pages < (int64_t)(budget < max_pages ? budget : max_pages) +
                                  ((int64_t)M + page_size - 2) / page_size + 1)
        return SPEC_EINVAL;
    if (R == 0) return SPEC_OK;
    if (!q || !ctx_len || !n_nodes || !out_lists || !out_len || (max_pages > 0 && !page_table))
        return SPEC_EINVAL;
    if ((uintptr_t)q & 15u) return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, need)) return SPEC_EWORKSPACE;
    SelectArgs a{};
    a.q = (const uint16_t *)q;
    a.lo = (const uint16_t *)k_min;
    a.hi = (const uint16_t *)k_max;
    a.table = page_table;
    a.ctx_len = ctx_len;
    a.n_nodes = n_nodes;
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.heads = Hkv;
    a.shift = __builtin_ctz((unsigned)page_size);
    a.M = M;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.budget = budget;
    a.first = first;
    a.last = last;
    a.lists = out_lists;
    a.list_len = out_len;
    a.width = list_pages;
    a.ctl = (Control *)workspace;
    a.keys = (uint64_t *)((char *)workspace + sizeof(Control));
    a.sums = (double *)(a.keys + (size_t)R * Hkv * max_pages);
    if (D == 64) launch_select<64>(a, R, (hipStream_t)stream);
    else if (D == 128) launch_select<128>(a, R, (hipStream_t)stream);
    else launch_select<256>(a, R, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
