// tree_attn.hip -- attention of drafted tokens over the paged cache on gfx950.
//
// Row (v, h) of request r: s_j = scale q . k_j over the tokens j the node sees,
// o = sum_j e^{s_j} v_j / sum_j e^{s_j}, in one pass over the tokens with the
// running maximum m, sum l and product o; scores are kept in units of log 2.
//
// Tiles.  The n G query rows that share a key head (row = node G + head in the
// group) are cut into row tiles of 16 RT rows; a wave takes 32 tokens a step.
//   S^T = K Q^T     v_mfma_f32_16x16x32_bf16, A = 16 tokens, B = 16 rows: lane
//                   (g = lane / 16, c = lane % 16) gets tokens 4 g + i of row c
//   O^T += V^T P^T  A = V^T, B = P^T: lane wants 8 tokens of row c as its B
//                   operand, and has them from S^T without a move if the
//                   contraction index (g, j) stands for token 4 g + j (j < 4) or
//                   16 + 4 g + j - 4; V is loaded by the same rule
// so a row's maximum, sum, weights and accumulators all live in the lanes with
// its c, and rescaling is one multiply by a lane's own value.  K's rows are
// read straight into the A operand's layout (16 bytes of one token a lane).
// V's rows are read 8 tokens by D / 16 values a lane and transposed in
// registers (v_perm_b32); output tile j then holds d = (D / 16) m + j, a
// permutation that the store undoes.  No shared memory and no barrier until
// the waves' results are joined.  e4m3 codes become bf16 exactly; their K
// scale multiplies the score, their V scale the weight before it is rounded.
//
// Split.  All (request, key head, row tile) items' token units (128 tokens)
// are laid end to end and cut into equal ranges, one per workgroup, whatever
// the lengths in the batch are; an item cut by a range border leaves partial
// (m, l, o) in the workspace, joined in order by a second launch.  Every
// workgroup finds its range from ctx_len and n_nodes by one scan.
#include <math.h>

#include "cache.h"

namespace sv {

struct Cut;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kStep = 32;              // tokens a wave takes at a time
constexpr int kUnit = kStep * kWaves;  // tokens of one unit of work
constexpr int kMaxGroups = 512;        // workgroups of the attention launch
constexpr int kFewUnits = 2048;        // below, one workgroup per compute unit
constexpr float kLazy = 8.0f;          // a maximum may lag by this many powers of two

struct AttnArgs {
    const uint16_t *q;           // [R][M][Hq][D] bf16
    Pages c;
    const int32_t *ctx_len, *n_nodes;
    const uint32_t *mask;        // [R][M][W], null: chain
    const int32_t *positions;    // [R][M], null: ctx + v
    float scale2;                // |scale| * log2(e), above 0
    uint32_t flip;               // sign bits for q where scale is negative
    int window, R, M, W, Hq, G;
    uint16_t *out;
    float *lse;
    Control *ctl;
    float *part;                 // [2 groups][part_stride]
    Cut *cuts;                   // [groups]
    int *n_cuts;                 // cuts that the launch wrote
    int groups, part_stride;
};

// ---------------------------------------------------------------------------
// the work list
// ---------------------------------------------------------------------------

struct Req {
    int n, ctx, rows, tiles;     // live nodes, context, query rows per key head, row tiles
    int lo;                      // the 16 tokens with the first one that any row sees
    bool ok;
};

template <int TR>
__device__ __forceinline__ Req request_of(const AttnArgs &a, int r) {
    Req q;
    q.n = a.n_nodes[r];
    q.ctx = a.ctx_len[r];
    q.ok = q.n >= 0 && q.n <= a.M && in_table(q.ctx, q.n, a.c.max_pages, a.c.shift);
    if (!q.ok) {
        q.n = a.M;               // every row of a faulty request is marked
        q.ctx = 0;
    }
    q.rows = q.n * a.G;
    q.tiles = (q.rows + TR - 1) / TR;
    // (no lower: 16 tokens always share a page, 32 need not, and the page before
    // the first token seen may have been given back)
    q.lo = a.window ? max(0, q.ctx - a.window + 1) & ~15 : 0;
    return q;
}

// Tokens [q.lo, end) of row tile t; a chain's rows see nothing behind their last node.
template <int TR>
__device__ __forceinline__ int tile_end(const AttnArgs &a, const Req &q, int t) {
    if (!q.ok) return q.lo + 1;
    if (a.mask) return q.ctx + q.n;
    return q.ctx + (min((t + 1) * TR, q.rows) - 1) / a.G + 1;
}
template <int TR>
__device__ __forceinline__ int tile_units(const AttnArgs &a, const Req &q, int t) {
    return (tile_end<TR>(a, q, t) - q.lo + kUnit - 1) / kUnit;
}
// Units of one key head.
template <int TR>
__device__ __forceinline__ int head_units(const AttnArgs &a, const Req &q) {
    if (q.tiles == 0) return 0;
    if (a.mask || !q.ok) return q.tiles * tile_units<TR>(a, q, 0);
    int s = 0;
    for (int t = 0; t < q.tiles; ++t) s += tile_units<TR>(a, q, t);
    return s;
}

// Ranges of the batch's `total` units (below 2^31, checked on the host): the
// first `extra` of `parts` ranges have `each` + 1 of them.  There are as many
// ranges as compute units, or two for each (fewer parts to join, against waits
// that hide each other): one user's 30 k tokens, 1880 units, take 29.2 us with
// 256 ranges and 32.6 with 512, 8 users of 4 k 22.7 and 24.7, 16 users (2300
// units) 35.3 and 34.6, 32 users 78 (288 ranges) and 65.0 (all bf16, D = 128).
// Numbers between leave some compute units twice the work of others.
struct Place {
    int r;                       // the request of the range's first unit
    int off;                     // units into it
    int total, parts, each, extra;
};

// The first unit of range `num` of `parts`.
__device__ __forceinline__ int border(const Place &p, int num) {
    return p.each * num + min(num, p.extra);
}

// The request that the first unit of this workgroup's range falls into.
// Neighbouring ranges, which often share a key head's pages, go to one XCD
// (workgroups are dealt to the eight in turn); num becomes the range, or -1.
// Every thread of the workgroup gets the same answer.
template <int TR>
__device__ __forceinline__ Place find_unit(const AttnArgs &a, int &num) {
    __shared__ int sum_s[kWaves];
    __shared__ int r_s, off_s;
    const int tid = threadIdx.x;
    const int chunk = (a.R + kBlock - 1) / kBlock;
    const int r0 = min(tid * chunk, a.R), r1 = min(r0 + chunk, a.R);
    int mine = 0;
    for (int r = r0; r < r1; ++r) mine += head_units<TR>(a, request_of<TR>(a, r)) * a.c.heads;
    // scan inside the wave, then over the four waves
    const int inc = (int)wave_incl_scan_dpp((uint32_t)mine);
    if ((tid & 63) == 63) sum_s[tid >> 6] = inc;
    __syncthreads();
    int base = 0;
    Place p;
    p.total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < (tid >> 6)) base += sum_s[w];
        p.total += sum_s[w];
    }
    p.total = __builtin_amdgcn_readfirstlane(p.total);
    p.parts = min(min(a.groups, p.total < kFewUnits ? kMaxGroups / 2 : kMaxGroups), p.total);
    p.each = p.parts ? p.total / p.parts : 0;
    p.extra = p.total - p.each * p.parts;
    p.r = a.R;
    p.off = 0;
    const int per = (p.parts + 7) >> 3, in = num >> 3;
    num = in < per ? (num & 7) * per + in : a.groups;
    if (num >= p.parts) {
        num = -1;
        return p;
    }
    const int at = border(p, num);
    const int first = base + inc - mine;
    if (at >= first && at < first + mine) {
        int left = at - first;
        int r = r0;
        for (; r < r1; ++r) {
            const int u = head_units<TR>(a, request_of<TR>(a, r)) * a.c.heads;
            if (left < u) break;
            left -= u;
        }
        r_s = r;
        off_s = left;
    }
    __syncthreads();
    p.r = __builtin_amdgcn_readfirstlane(r_s);
    p.off = __builtin_amdgcn_readfirstlane(off_s);
    return p;
}

struct Item {
    int h, t, u;                 // key head, row tile, unit in the item
};
template <int TR>
__device__ __forceinline__ Item item_of(const AttnArgs &a, const Req &rq, int off) {
    const int hu = head_units<TR>(a, rq);
    Item i;
    i.h = off / hu;
    i.t = 0;
    i.u = off - i.h * hu;
    if (a.mask || !rq.ok) {
        const int units = tile_units<TR>(a, rq, 0);
        i.t = i.u / units;
        i.u -= i.t * units;
    } else {
        for (int units; i.u >= (units = tile_units<TR>(a, rq, i.t)); ++i.t) i.u -= units;
    }
    return i;
}

// What a range left of the item it began and did not finish, for the join.
struct Cut {
    int node0, h, row0;          // first node of the request, key head, first row
    int rows;                    // rows of the item; 0: none
    int parts;                   // ranges that hold its units, from this one on
    int pad[3];
};

// Range `grp`'s entry; `rest` units of the item are behind the range.
template <int TR>
__device__ __forceinline__ void write_cut(const AttnArgs &a, const Place &p, int grp, bool cuts,
                                          int r, const Req &rq, int h, int t, int rest) {
    Cut cut{r * a.M, h, t * TR, cuts ? min(TR, rq.rows - t * TR) : 0, 1, {0, 0, 0}};
    const int last = border(p, grp + 1) + rest;
    while (grp + cut.parts < p.parts && border(p, grp + cut.parts) < last) ++cut.parts;
    a.cuts[grp] = cut;
    if (grp == 0) *a.n_cuts = p.parts - 1;  // the last range cuts nothing
}

// ---------------------------------------------------------------------------
// one wave's step
// ---------------------------------------------------------------------------

// v, opaque to the compiler: what is derived from it stays where it is used
// instead of being computed ahead of the token loop, whose registers are short.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

template <bool FP8, int D> struct Tile {
    static constexpr int KS = D / 32;              // contraction steps of Q K^T
    static constexpr int DV = D / 16;              // values of V a lane holds per token
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int KV = D * EB / 64;         // 16-byte K loads per 16 tokens
    static constexpr int VW = DV * EB / 4;         // 32-bit words of V per token
    u32x4_t k[2][KV];
    uint32_t v[8][VW];
    float sc;                                      // scales (FP8), see load_scale
};

// N consecutive 32-bit words (N a multiple of 4, or 1 or 2: aligned to them).
template <int N>
__device__ __forceinline__ void load_words(const char *p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *(const uint32_t *)p;
    } else if constexpr (N == 2) {
        const u32x2_t x = *(const u32x2_t *)p;
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4_t x = *(const u32x4_t *)(p + 4 * i);
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
    }
}

// Element offsets of the step's two 16-token halves: rows, and scales.
struct Half {
    int64_t row[2];              // (page * heads + head) * size + offset
    int bad;                     // bit h: half h lies in a bad page
};

// The row of the page table that request r's key head h reads by: the
// request's, or (LISTS) a page list of its own.  A template argument, so that
// the launches over tables hold nothing of it: their scalar registers are short.
template <bool LISTS>
__device__ __forceinline__ int table_row(const AttnArgs &a, int r, int h) {
    return LISTS ? r * a.c.heads + h : r;
}
// A page number, by a scalar load (the index is the wave's, and nothing in a
// launch writes the table).
__device__ __forceinline__ int page_number(const AttnArgs &a, int row, int index) {
    typedef const __attribute__((address_space(4))) int32_t *table_t;
    return ((table_t)(uintptr_t)(a.c.table + (int64_t)row * a.c.max_pages))[index];
}

// The page numbers of a step's halves, one load ahead of their use: a wave
// that waited for them before it could ask for the rows stood still for a
// memory round trip each step.
struct Numbers {
    int page[2];
};
__device__ __forceinline__ Numbers numbers_of(const AttnArgs &a, int row, int t, int L) {
    Numbers x;
    t = min(t, L - 1);                                  // a step behind the end is not used
    x.page[0] = page_number(a, row, t >> a.c.shift);
    x.page[1] = page_number(a, row, min(t + 16, L - 1) >> a.c.shift);
    return x;
}
__device__ __forceinline__ Half halves_of(const AttnArgs &a, const Numbers &num, int h, int t, int L) {
    Half x;
    x.bad = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int tt = t + 16 * s < L ? t + 16 * s : t;  // nor is a half
        int page = t + 16 * s < L ? num.page[s] : num.page[0];
        if ((unsigned)page >= (unsigned)a.c.num_pages) {
            x.bad |= 1 << s;
            page = 0;
        }
        x.row[s] = ((int64_t)page * a.c.heads + h) * a.c.size + (tt & (a.c.size - 1));
    }
    return x;
}

template <bool FP8, int D>
__device__ __forceinline__ void load_k(const AttnArgs &a, const Half &x, int lane, Tile<FP8, D> &t) {
    const int hl = here(lane), c = hl & 15, g = hl >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        // a wave's base, and a lane's 32-bit offset
        const char *p = (const char *)a.c.k + x.row[s] * (D * Tile<FP8, D>::EB);
        const uint32_t lane_at = c * (D * Tile<FP8, D>::EB) + g * 16;
#pragma unroll
        for (int i = 0; i < Tile<FP8, D>::KV; ++i) t.k[s][i] = *(const u32x4_t *)(p + lane_at + i * 64);
    }
}
template <bool FP8, int D>
__device__ __forceinline__ void load_v(const AttnArgs &a, const Half &x, int lane, Tile<FP8, D> &t) {
    typedef Tile<FP8, D> TT;
    const int hl = here(lane), c = hl & 15, g = hl >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const char *p = (const char *)a.c.v + x.row[s] * (D * TT::EB);
        const uint32_t lane_at = g * (4 * D * TT::EB) + c * (TT::VW * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words(p + lane_at + i * (D * TT::EB), t.v[4 * s + i]);
    }
}

// A step's 64 scales, one a lane: lane group g holds those of its own tokens,
// K's of its eight in lanes 0-7 and V's in lanes 8-15, for row_times to take by row broadcasts.
__device__ __forceinline__ float load_scale(const AttnArgs &a, const Half &x, int lane) {
    const int hl = here(lane), c = hl & 15, g = hl >> 4;
    const float *k = a.c.k_scale + x.row[0], *v = a.c.v_scale + x.row[0];
    const int64_t at = (c & 4 ? x.row[1] - x.row[0] : 0) + 4 * g + (c & 3);
    return (c & 8 ? v : k)[at];
}

// The A operand of contraction step ks of the 16 tokens of half s.
template <bool FP8, int D>
__device__ __forceinline__ bf16x8_t k_frag(const Tile<FP8, D> &t, int s, int ks) {
    if constexpr (!FP8) {
        return __builtin_bit_cast(bf16x8_t, t.k[s][ks]);
    } else {
        const u32x4_t w = t.k[s][ks >> 1];
        const uint32_t x = ks & 1 ? w.z : w.x, y = ks & 1 ? w.w : w.y;
        return __builtin_bit_cast(bf16x8_t, u32x4_t{e4m3_bf16<false>(x), e4m3_bf16<true>(x),
                                                       e4m3_bf16<false>(y), e4m3_bf16<true>(y)});
    }
}
// First of the 8 values of q that lane group g pairs with it.
template <bool FP8> __device__ __forceinline__ int q_chunk(int ks, int g) {
    return FP8 ? 16 * (4 * (ks >> 1) + g) + 8 * (ks & 1) : 8 * (4 * ks + g);
}

// Packed bf16 words of V: tok[t] holds values 2 w and 2 w + 1 of token t.
template <bool FP8, int D>
__device__ __forceinline__ uint32_t v_word(const Tile<FP8, D> &t, int tok, int w) {
    if constexpr (!FP8) return t.v[tok][w];
    else return w & 1 ? e4m3_bf16<true>(t.v[tok][w >> 1]) : e4m3_bf16<false>(t.v[tok][w >> 1]);
}

// The low k bits, k clamped to 0 .. 32.
__device__ __forceinline__ uint32_t ones(int k) {
    return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u;
}
// Node and position of query row `row` of request r (rows past the last
// stand for it).
struct Query {
    int node, pos;
};
__device__ __forceinline__ Query query_of(const AttnArgs &a, const Req &rq, int r, int row) {
    Query q;
    q.node = min(row, rq.rows - 1) / a.G;
    q.pos = a.positions ? a.positions[(size_t)r * a.M + q.node] : rq.ctx + q.node;
    return q;
}
// The low k bits of 64, k clamped to 0 .. 64.
__device__ __forceinline__ uint64_t ones64(int k) {
    return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1ull;
}
// Tokens tok .. tok + 63 that a row sees, one bit each: the row's node v (its
// tree bits from slot ctx - tok on in `tree`, for a mask) at position pos.
__device__ __forceinline__ uint64_t sees(const AttnArgs &a, const Req &rq, int tok, int v, int pos,
                                         uint64_t tree) {
    const int k = rq.ctx - tok;  // tokens of the context
    const uint64_t old = ones64(k);
    if (a.mask) {
        tree &= ones64(k + rq.n);
    } else {
        tree = ones64(k + v + 1);
        if (a.window) tree &= ~ones64(max(k + v + 1, 0) - a.window);
    }
    const uint64_t near = a.window ? old & ~ones64(max(pos - a.window + 1, 0) - tok) : old;
    return near | (tree & ~old);
}
// Bit i: token i of this lane group's eight.
__device__ __forceinline__ uint32_t lane_bits(uint32_t seen, int g) {
    return (seen >> (4 * g) & 15u) | (seen >> (4 * g + 16) & 15u) << 4;
}

// The B operands of query row `row`: lane group g holds its values of every
// contraction step.
template <bool FP8, int D>
__device__ __forceinline__ void load_q(const AttnArgs &a, const Req &rq, int r, int h, int row, int lane,
                                       bf16x8_t (&qf)[D / 32]) {
    row = min(here(row), rq.rows - 1);
    const int node = row / a.G, g = here(lane) >> 4;
    const uint16_t *qp = a.q + (((size_t)r * a.M + node) * a.Hq + h * a.G + (row - node * a.G)) * D;
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks)
        qf[ks] = __builtin_bit_cast(bf16x8_t, *(const u32x4_t *)(qp + q_chunk<FP8>(ks, g)) ^ a.flip);
}

// Maximum (NaN if one is) of a lane's eight scores, and over the four lanes
// that share a column; the latter's sum.
__device__ __forceinline__ float max2(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float max8(const float (&p)[8]) {
    return max2(max2(max2(p[0], p[1]), max2(p[2], p[3])), max2(max2(p[4], p[5]), max2(p[6], p[7])));
}
__device__ __forceinline__ float column_max(float v) {
    uint32_t lo, hi;
    lane_pair<16>(__float_as_uint(v), lo, hi);
    v = max2(__uint_as_float(lo), __uint_as_float(hi));
    lane_pair<32>(__float_as_uint(v), lo, hi);
    return max2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ float column_sum(float v) {
    uint32_t lo, hi;
    lane_pair<16>(__float_as_uint(v), lo, hi);
    v = __uint_as_float(lo) + __uint_as_float(hi);
    lane_pair<32>(__float_as_uint(v), lo, hi);
    return __uint_as_float(lo) + __uint_as_float(hi);
}

// p[i] times the value that lane FIRST + i of the lane group holds (the
// broadcast is an operand modifier of the multiply).
template <int N>
__device__ __forceinline__ float row_lane(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x150 + N, 0xf, 0xf, true));
}
template <int FIRST>
__device__ __forceinline__ void row_times(float (&p)[8], float v) {
    p[0] *= row_lane<FIRST>(v);
    p[1] *= row_lane<FIRST + 1>(v);
    p[2] *= row_lane<FIRST + 2>(v);
    p[3] *= row_lane<FIRST + 3>(v);
    p[4] *= row_lane<FIRST + 4>(v);
    p[5] *= row_lane<FIRST + 5>(v);
    p[6] *= row_lane<FIRST + 6>(v);
    p[7] *= row_lane<FIRST + 7>(v);
}

// The running softmax's step for a lane's eight tokens of each of its RT
// columns, in three parts, so that a caller can lay the products of one column
// between the exponents of the next.
//
// Scores s become p, ready for the exponent but for scale2 (bf16), and top
// their maximum.  seen: bit i, the row sees token i; bad: bit h, tokens
// 4 h .. 4 h + 3 lie in a bad page (both only where masked).
template <bool FP8>
__device__ __forceinline__ float peak(const f32x4_t (&s)[2], float sc, float scale2, bool masked,
                                      uint32_t seen, int bad, float (&p)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3];
    if constexpr (FP8) row_times<0>(p, sc * scale2);
    if (masked) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = !(seen >> i & 1u) ? -INFINITY : bad >> (i >> 2) & 1 ? NAN : p[i];
    }
    const float top = max8(p);  // m is the column's, so a lane's own maximum tells
    return FP8 ? top : top * scale2;
}
// The maximum may lag by kLazy: weights then reach 2^kLazy, which costs no
// precision, and most steps rescale nothing.
template <int RT, int DV>
__device__ __forceinline__ void lift(const float (&top)[RT], float (&m)[RT], float (&l)[RT],
                                     f32x4_t (&acc)[RT][DV]) {
    bool up = false;
#pragma unroll
    for (int x = 0; x < RT; ++x) up |= top[x] > m[x] + kLazy;
    if (!__any(up)) return;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const float most = column_max(top[x]);
        const bool due = most > m[x] + kLazy;  // a row's own affair, whatever its neighbours do
        const float al = due ? __builtin_amdgcn_exp2f(m[x] - most) : 1.f;
        l[x] *= al;
#pragma unroll
        for (int j = 0; j < DV; ++j) acc[x][j] *= al;
        m[x] = due ? most : m[x];
    }
}
// The weights (bf16, 2^-8 relative like the output's own rounding; V's scale
// goes in first), and their sum into l.
template <bool FP8>
__device__ __forceinline__ u32x4_t weigh(float (&p)[8], float sc, float scale2, float m, float &l) {
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(FP8 ? p[i] - ref : fmaf(p[i], scale2, -ref));
        l += p[i];
    }
    if constexpr (FP8) row_times<8>(p, sc);
    return u32x4_t{pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]),
                   pack_bf16(p[6], p[7])};
}

// NaN and infinities in V or its scale.  A weight of 0 would not cancel them in
// a product, and rows that do not see such a token must not meet it: where
// some row does not see a token, the values leave the operand (take_rare) and
// are added after the token loop to the rows that do (add_rare).  Few calls ever hold
// one; what matters is that the loop has no part in it but the look.
template <bool FP8, int N>
__device__ __forceinline__ bool take_rare(uint32_t (&w)[N], bool live) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t v = live ? w[i] : 0u;
        if constexpr (!FP8) {
            const bool lo = (v & 0x7f80u) == 0x7f80u, hi = (v & 0x7f800000u) == 0x7f800000u;
            odd |= lo || hi;
            v &= (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
        } else {
#pragma unroll
            for (int s = 0; s < 32; s += 8) {  // e4m3: seven ones are a NaN
                const bool nan = (v >> s & 0x7fu) == 0x7fu;
                odd |= nan;
                v &= nan ? ~(0xffu << s) : ~0u;
            }
        }
        w[i] = v;
    }
    return odd;
}
// The same of a token's scale.
__device__ __forceinline__ bool take_rare(float &sc, bool live) {
    const bool odd = !(fabsf(sc) < INFINITY);
    sc = odd ? 0.f : sc;
    return odd && live;
}
// Tokens [from, to) of the request, for the row whose sums acc holds.
template <bool FP8, int D>
__device__ __forceinline__ void add_rare(const AttnArgs &a, const Req &rq, int r, int h, int trow, int row,
                                         int from, int to, int lane, f32x4_t (&acc)[D / 16]) {
    constexpr int DV = D / 16;
    const int g = here(lane) >> 4;
    const Query q = query_of(a, rq, r, here(row));
    const uint32_t *mrow = a.mask ? a.mask + ((size_t)r * a.M + q.node) * a.W : nullptr;
#pragma unroll 1
    for (int t = from; t < to; ++t) {
        const int page = page_number(a, trow, t >> a.c.shift), u = t - rq.ctx;
        if ((unsigned)page >= (unsigned)a.c.num_pages) continue;
        const uint64_t tree = mrow && u >= 0 && u < rq.n ? mrow[u >> 5] >> (u & 31) & 1u : 0u;
        const bool see = sees(a, rq, t, q.node, q.pos, tree) & 1u;
        const int64_t slot = ((int64_t)page * a.c.heads + h) * a.c.size + (t & (a.c.size - 1)), at = slot * D;
        const float sc = FP8 ? a.c.v_scale[slot] : 1.f;
#pragma unroll
        for (int j = 0; j < DV; ++j) {
            __builtin_amdgcn_sched_barrier(0);  // few loads at a time: registers are short
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t e = at + DV * (4 * g + i) + j;
                float val;
                if constexpr (FP8) val = sc * bf16_lo(e4m3_bf16<false>(((const uint8_t *)a.c.v)[e]));
                else val = bf16_lo(((const uint16_t *)a.c.v)[e]);
                acc[j][i] += see && !(fabsf(val) < INFINITY) ? val : 0.f;
            }
        }
    }
}

// Tokens that every row of a wave sees: steps inside need no mask.
struct Plain {
    int lo, hi;
};
// For the 16 RT rows from `row0` on, up to token t1.
template <int RT>
__device__ __forceinline__ Plain plain_of(const AttnArgs &a, const Req &rq, int r, int row0, int c,
                                          int t1) {
    Plain p;
    p.lo = 0;
    p.hi = rq.ctx;
    if (!a.mask && !a.window) p.hi += row0 / a.G + 1;
    if (a.window) {
        int far = 0;
#pragma unroll
        for (int x = 0; x < RT; ++x) far = max(far, query_of(a, rq, r, row0 + x * 16 + c).pos);
        // (a position may be anything up to 2^31 - 1: inside the item, lo can be
        // rounded up to a tile in 32 bits)
        p.lo = min(max(wave_max_i(far) - a.window + 1, 0), t1);
    }
    p.hi = min(p.hi, t1);
    return p;
}

// ---------------------------------------------------------------------------
// the attention launch
// ---------------------------------------------------------------------------

// Bound by HBM: a workgroup's waves keep one step of K and V each in flight.
// One token behind 30011 (bf16): 27.8 us, 4.4 TB/s; 64 chains of 8 behind up to
// 4 k (e4m3): 83 us, 3.8 TB/s (two waves a SIMD, for the registers).
template <int D, int RT> constexpr int waves_per_simd() {
    return D <= 128 && D * RT <= 256 ? 2 : 1;
}

template <bool FP8, int D, int RT, bool LISTS>
__global__ void __launch_bounds__(kBlock, (waves_per_simd<D, RT>())) attn_kernel(AttnArgs a) {
    typedef Tile<FP8, D> TT;
    constexpr int KS = TT::KS, DV = TT::DV, TR = 16 * RT;
    constexpr int LD = D + 4;    // row pitch of the join buffer
    __shared__ float o_s[kWaves][16][LD];
    __shared__ float m_s[kWaves][16], l_s[kWaves][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    int grp = blockIdx.x;
    const Place at = find_unit<TR>(a, grp);
    if (grp < 0) {
        if (at.parts == 0 && blockIdx.x == 0 && tid == 0) *a.n_cuts = 0;
        return;
    }
    int left = border(at, grp + 1) - border(at, grp);
    int r = at.r;
    Req rq = request_of<TR>(a, r);
    const Item it = item_of<TR>(a, rq, at.off);
    int h = it.h, t = it.t, u0 = it.u;
    while (true) {
        // ---- one item (r, h, t), its units from u0 on
        const int end = tile_end<TR>(a, rq, t);
        const int units = tile_units<TR>(a, rq, t);
        const int u1 = min(units, u0 + left);
        const int t0 = rq.lo + u0 * kUnit, t1 = min(end, rq.lo + u1 * kUnit);
        const int trow = table_row<LISTS>(a, r, h);
        const bool whole = u0 == 0 && u1 == units;
        // ---- the rows of this lane's column
        bf16x8_t qf[RT][KS];
#pragma unroll
        for (int x = 0; x < RT; ++x) load_q<FP8, D>(a, rq, r, h, t * TR + x * 16 + c, lane, qf[x]);
        // the rows' tree bits (at most 32 nodes here) and positions, for masks
        uint32_t bits[RT];
        Query at_row[RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            at_row[x] = query_of(a, rq, r, t * TR + x * 16 + c);
            bits[x] = a.mask ? a.mask[((size_t)r * a.M + at_row[x].node) * a.W] : 0u;
        }
        f32x4_t acc[RT][DV];
        float m[RT], l[RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            m[x] = -INFINITY;
            l[x] = 0.f;
#pragma unroll
            for (int j = 0; j < DV; ++j) acc[x][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        const Plain plain = plain_of<RT>(a, rq, r, t * TR, c, t1);
        int tok = t0 + wave * kStep;
        int bad = 0;        // a bad page was met
        bool rare = false;  // values left the products
        // (no load but the next step's is under way inside the loop.  A load
        // that a branch may issue makes the compiler wait for all of them
        // where the branch joins.)
        if (rq.ok && tok < t1) {
            TT kv;
            Half cur = halves_of(a, numbers_of(a, trow, tok, end), h, tok, end);
            Numbers num = numbers_of(a, trow, tok + kUnit, end);
            load_k<FP8, D>(a, cur, lane, kv);
            if constexpr (FP8) kv.sc = load_scale(a, cur, lane);
            load_v<FP8, D>(a, cur, lane, kv);
            while (true) {
                const int nxt = tok + kUnit;
                const bool more = nxt < t1;
                Half nh = cur;
                if (more) nh = halves_of(a, num, h, nxt, end);
                num = numbers_of(a, trow, nxt + kUnit, end);
                // ---- scores
                f32x4_t s[RT][2];
#pragma unroll
                for (int x = 0; x < RT; ++x)
                    for (int hf = 0; hf < 2; ++hf) s[x][hf] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const bf16x8_t kf = k_frag<FP8, D>(kv, hf, ks);
#pragma unroll
                        for (int x = 0; x < RT; ++x)
                            s[x][hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[x][ks], s[x][hf], 0, 0, 0);
                    }
                }
                float sc = FP8 ? kv.sc : 0.f;
                if (more) {
                    load_k<FP8, D>(a, nh, lane, kv);
                    if constexpr (FP8) kv.sc = load_scale(a, nh, lane);
                }
                __builtin_amdgcn_sched_barrier(0);
                const bool masked = tok < plain.lo || tok + kStep > plain.hi || cur.bad;
                uint32_t seen[RT];  // bit i: the row sees this lane's token i
                float p[RT][8], top[RT];
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    seen[x] = 0xffu;
                    if (masked) {
                        const int k = rq.ctx - tok;  // tree slot 0 is bit k
                        const uint64_t tree = k >= 64 ? 0ull : k >= 0 ? (uint64_t)bits[x] << k
                                            : k > -32 ? bits[x] >> -k : 0u;
                        seen[x] = lane_bits((uint32_t)sees(a, rq, tok, at_row[x].node, at_row[x].pos, tree), g);
                    }
                    top[x] = peak<FP8>(s[x], sc, a.scale2, masked, seen[x], cur.bad, p[x]);
                }
                lift(top, m, l, acc);
                if (masked) {
                    bool odd = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        odd |= take_rare<FP8>(kv.v[i], tok + 16 * (i >> 2) + 4 * g + (i & 3) < t1);
                    if constexpr (FP8) {
                        if (lane & 8) odd |= take_rare(sc, tok + 16 * (lane >> 2 & 1) + 4 * g + (lane & 3) < t1);
                    }
                    rare |= __any(odd);
                }
                u32x4_t pw[RT];
#pragma unroll
                for (int x = 0; x < RT; ++x) pw[x] = weigh<FP8>(p[x], sc, a.scale2, m[x], l[x]);
                // ---- product
#pragma unroll
                for (int w = 0; w < DV / 2; ++w) {
                    __builtin_amdgcn_sched_barrier(0);  // one word's operands in registers at a time
                    uint32_t b[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[i] = v_word<FP8, D>(kv, i, w);
                    u32x4_t f0, f1;
                    f0.x = __builtin_amdgcn_perm(b[1], b[0], 0x05040100);
                    f0.y = __builtin_amdgcn_perm(b[3], b[2], 0x05040100);
                    f0.z = __builtin_amdgcn_perm(b[5], b[4], 0x05040100);
                    f0.w = __builtin_amdgcn_perm(b[7], b[6], 0x05040100);
                    f1.x = __builtin_amdgcn_perm(b[1], b[0], 0x07060302);
                    f1.y = __builtin_amdgcn_perm(b[3], b[2], 0x07060302);
                    f1.z = __builtin_amdgcn_perm(b[5], b[4], 0x07060302);
                    f1.w = __builtin_amdgcn_perm(b[7], b[6], 0x07060302);
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        const bf16x8_t pf = __builtin_bit_cast(bf16x8_t, pw[x]);
                        acc[x][2 * w] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, f0), pf, acc[x][2 * w], 0, 0, 0);
                        acc[x][2 * w + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, f1), pf, acc[x][2 * w + 1], 0, 0, 0);
                    }
                }
                bad |= cur.bad;
                if (!more) break;
                load_v<FP8, D>(a, nh, lane, kv);
                __builtin_amdgcn_sched_barrier(0);
                cur = nh;
                tok = nxt;
            }
        }
        if (rare) {
#pragma unroll 1
            for (int s = t0 + wave * kStep; s < t1; s += kUnit) {
                if (s >= plain.lo && s + kStep <= plain.hi) continue;
#pragma unroll
                for (int x = 0; x < RT; ++x)
                    add_rare<FP8, D>(a, rq, r, h, trow, t * TR + x * 16 + c, s, min(s + kStep, t1), lane, acc[x]);
            }
        }
        if (bad && lane == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        // ---- join the four waves, 16 rows at a time
        const int et = here(tid), ec = et & 15, eg = et >> 4 & 3;
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            l[x] = column_sum(l[x]);
            if (!rq.ok || query_of(a, rq, r, t * TR + x * 16 + ec).pos < rq.ctx) {
                l[x] = NAN;
                atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < DV; j += 4)
                    *(f32x4_t *)&o_s[wave][ec][DV * (4 * eg + i) + j] =
                        f32x4_t{acc[x][j][i], acc[x][j + 1][i], acc[x][j + 2][i], acc[x][j + 3][i]};
            if (eg == 0) {
                m_s[wave][ec] = m[x];
                l_s[wave][ec] = l[x];
            }
            __syncthreads();
            const int jr = et >> 4, e0 = (et & 15) * DV;  // this thread's row and values
            const int row = t * TR + x * 16 + jr;
            float mm = fmaxf(fmaxf(m_s[0][jr], m_s[1][jr]), fmaxf(m_s[2][jr], m_s[3][jr]));
            const float ref = mm == -INFINITY ? 0.f : mm;
            float sum = 0.f, o[DV];
#pragma unroll
            for (int j = 0; j < DV; ++j) o[j] = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(m_s[w][jr] - ref);
                sum += f * l_s[w][jr];
#pragma unroll
                for (int j = 0; j < DV; ++j) o[j] += f * o_s[w][jr][e0 + j];
            }
            if (row < rq.rows) {
                if (whole) {
                    const int nd = row / a.G;
                    const size_t orow = ((size_t)r * a.M + nd) * a.Hq + h * a.G + (row - nd * a.G);
                    if (sum == 0.f) {  // no weight at all: o is 0, whatever V holds
                        sum = 1.f;
                        mm = -INFINITY;
#pragma unroll
                        for (int j = 0; j < DV; ++j) o[j] = 0.f;
                    }
                    const float inv = 1.f / sum;
                    uint16_t *op = a.out + orow * D + e0;
#pragma unroll
                    for (int j = 0; j < DV; j += 4)
                        *(u32x2_t *)(op + j) = u32x2_t{pack_bf16(o[j] * inv, o[j + 1] * inv),
                                                        pack_bf16(o[j + 2] * inv, o[j + 3] * inv)};
                    if ((et & 15) == 0) {
                        if (a.lse) a.lse[orow] = (mm + log2f(sum)) * (float)kLn2;
                    }
                } else {
                    float *pp = a.part + (size_t)(2 * grp + (u0 == 0)) * a.part_stride;
                    float *po = pp + (size_t)(x * 16 + jr) * D + e0;
#pragma unroll
                    for (int j = 0; j < DV; j += 4) *(f32x4_t *)(po + j) = f32x4_t{o[j], o[j + 1], o[j + 2], o[j + 3]};
                    if ((et & 15) == 0) {
                        pp[TR * D + x * 16 + jr] = mm;
                        pp[TR * D + TR + x * 16 + jr] = sum;
                    }
                }
            }
        }
        // ---- the next item
        left -= u1 - u0;
        if (left <= 0) {
            if (tid == 0) write_cut<TR>(a, at, grp, u0 == 0 && !whole, r, rq, h, t, units - u1);
            return;
        }
        u0 = 0;
        if (++t >= rq.tiles) {
            t = 0;
            if (++h >= a.c.heads) {
                h = 0;
                do {
                    if (++r >= a.R) return;
                    rq = request_of<TR>(a, r);
                } while (rq.tiles == 0);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// many rows to a key head
// ---------------------------------------------------------------------------

constexpr int kTile = 64;              // tokens staged at a time

// The same arithmetic with the waves side by side in the rows (16 RT each)
// instead of the tokens: 64 tokens of K and V go to shared memory once per
// workgroup, already in operand layout (converted and transposed on the way),
// while the previous 64 are multiplied, and every wave reads them from there.
// Bound by HBM for trees (64 of 48 nodes behind up to 4 k tokens, bf16: 176 us,
// 3.6 TB/s; with the arithmetic left out 150), by the issue of matrix and
// vector instructions for prompt chunks (4 of 1000 behind 12 k, five heads a
// key head, e4m3: 771 us, 831 TFLOP/s, the matrix pipes 33% busy).
template <bool FP8, int D> struct Stage {
    typedef Tile<FP8, D> TT;
    u32x4_t k[TT::KV];
    uint32_t v[4][TT::VW];
    float sc;
    int flags;                         // bit 1: the 16 tokens lie in a bad page
    uint32_t bits[3];                  // tree bits of this thread's row, see stage_sight
};
template <bool FP8, int D, int TR> struct Shared {
    u32x4_t k[2][4][D / 32][64];         // [buffer][16 tokens][contraction step][lane]
    u32x2_t v[2][2][D / 16][2][64];      // [buffer][32 tokens][output tile][half][lane]
    float sc[2][2][64];                // [buffer][32 tokens][lane], as load_scale's
    int flags[2][4];                   // per 16 tokens: bit 0 rare values left V, bit 1 a bad page
    uint64_t sight[2][TR];             // per row: the tokens of the tile that it sees
};

// The page number of this wave's 16 tokens of the tile at token t0; those
// behind the end take the last token's page, and are not used.
__device__ __forceinline__ int stage_page(const AttnArgs &a, int row, int t0, int end, int wave) {
    return page_number(a, row, min(t0 + 16 * wave, end - 1) >> a.c.shift);
}

// Loads this wave's 16 tokens of the tile at token t0 (rows [t0, end) exist).
template <bool FP8, int D>
__device__ __forceinline__ void stage_load(const AttnArgs &a, int page, int h, int t0, int end, int wave,
                                           int lane, Stage<FP8, D> &s) {
    typedef Tile<FP8, D> TT;
    const int hl = here(lane), c = hl & 15, g = hl >> 4;
    const int tt = t0 + 16 * wave < end ? t0 + 16 * wave : (end - 1) & ~15;
    s.flags = 0;
    if ((unsigned)page >= (unsigned)a.c.num_pages) {
        s.flags = 2;
        page = 0;
    }
    const int64_t row = ((int64_t)page * a.c.heads + h) * a.c.size + (tt & (a.c.size - 1));
    const char *kp = (const char *)a.c.k + row * (D * TT::EB);
    const uint32_t k_at = c * (D * TT::EB) + g * 16;
#pragma unroll
    for (int i = 0; i < TT::KV; ++i) s.k[i] = *(const u32x4_t *)(kp + k_at + i * 64);
    const char *vp = (const char *)a.c.v + row * (D * TT::EB);
    const uint32_t v_at = g * (4 * D * TT::EB) + c * (TT::VW * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_words(vp + v_at + i * (D * TT::EB), s.v[i]);
    if constexpr (FP8) s.sc = lane & 16 ? (a.c.v_scale + row)[c] : (a.c.k_scale + row)[c];
}

// A row's mask words that hold the tree slots of the 64 tokens from t0 on.
template <bool FP8, int D>
__device__ __forceinline__ void load_bits(const AttnArgs &a, const Req &rq, int r, int node, int t0,
                                          Stage<FP8, D> &s) {
    const uint32_t *row = a.mask + ((size_t)r * a.M + node) * a.W;
    const int w = (t0 - rq.ctx) >> 5;  // of slot t0 - ctx
#pragma unroll
    for (int i = 0; i < 3; ++i) s.bits[i] = w + i >= 0 && w + i < a.W ? row[w + i] : 0u;
}
// Which of them the row sees (thread `tid`'s, of the workgroup's row tile).
template <bool FP8, int D>
__device__ __forceinline__ uint64_t stage_sight(const AttnArgs &a, const Req &rq, int t0, Query q,
                                                const Stage<FP8, D> &s) {
    uint64_t tree = 0ull;
    if (a.mask) {
        const int sh = (t0 - rq.ctx) & 31;
        const uint32_t b0 = here(s.bits[0]), b1 = here(s.bits[1]), b2 = here(s.bits[2]);  // not waited for before
        tree = ((uint64_t)b1 << 32 | b0) >> sh;
        if (sh) tree |= (uint64_t)b2 << (64 - sh);
    }
    return sees(a, rq, t0, q.node, q.pos, tree);
}

// Writes them to buffer b.  `part`: the tile holds tokens that some row does
// not see, or that do not exist (from `end` on, V becomes 0): values of V that
// a weight of 0 would not cancel are looked for.
template <bool FP8, int D, typename SH>
__device__ __forceinline__ void stage_store(const AttnArgs &a, SH &sh, int b, int t0, int end,
                                            bool part, int wave, int lane, Stage<FP8, D> &s) {
    typedef Tile<FP8, D> TT;
    const int g = lane >> 4;
#pragma unroll
    for (int i = 0; i < TT::KV; ++i) {
        if constexpr (!FP8) {
            sh.k[b][wave][i][lane] = s.k[i];
        } else {
            const u32x4_t w = s.k[i];
            sh.k[b][wave][2 * i][lane] = u32x4_t{e4m3_bf16<false>(w.x), e4m3_bf16<true>(w.x),
                                                    e4m3_bf16<false>(w.y), e4m3_bf16<true>(w.y)};
            sh.k[b][wave][2 * i + 1][lane] = u32x4_t{e4m3_bf16<false>(w.z), e4m3_bf16<true>(w.z),
                                                        e4m3_bf16<false>(w.w), e4m3_bf16<true>(w.w)};
        }
    }
    int flags = s.flags;
    if (part) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= take_rare<FP8>(s.v[i], t0 + 16 * wave + 4 * g + i < end);
        if constexpr (FP8) {
            if (lane & 16) odd |= take_rare(s.sc, t0 + 16 * wave + (lane & 15) < end);
        }
        flags |= __any(odd) ? 1 : 0;
    }
    uint32_t v[4][TT::DV / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < TT::DV / 2; ++w) {
            if constexpr (!FP8) v[i][w] = s.v[i][w];
            else v[i][w] = w & 1 ? e4m3_bf16<true>(s.v[i][w >> 1]) : e4m3_bf16<false>(s.v[i][w >> 1]);
        }
#pragma unroll
    for (int w = 0; w < TT::DV / 2; ++w) {
        sh.v[b][wave >> 1][2 * w][wave & 1][lane] =
            u32x2_t{__builtin_amdgcn_perm(v[1][w], v[0][w], 0x05040100),
                       __builtin_amdgcn_perm(v[3][w], v[2][w], 0x05040100)};
        sh.v[b][wave >> 1][2 * w + 1][wave & 1][lane] =
            u32x2_t{__builtin_amdgcn_perm(v[1][w], v[0][w], 0x07060302),
                       __builtin_amdgcn_perm(v[3][w], v[2][w], 0x07060302)};
    }
    if constexpr (FP8) {
        // lane c of K's (0-15) or V's (16-31): token c of the wave's 16
        const int c = lane & 15;
        if (lane < 32)
            sh.sc[b][wave >> 1][16 * (c >> 2) + (lane & 16 ? 8 : 0) + 4 * (wave & 1) + (c & 3)] = s.sc;
    }
    if (lane == 0) sh.flags[b][wave] = flags;
}

template <bool FP8, int D, int RT, bool LISTS>
__global__ void __launch_bounds__(kBlock, D <= 128 ? 2 : 1) attn_wide_kernel(AttnArgs a) {
    typedef Tile<FP8, D> TT;
    constexpr int KS = TT::KS, DV = TT::DV, TR = 64 * RT;
    __shared__ Shared<FP8, D, TR> sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    int grp = blockIdx.x;
    const Place at = find_unit<TR>(a, grp);
    if (grp < 0) {
        if (at.parts == 0 && blockIdx.x == 0 && tid == 0) *a.n_cuts = 0;
        return;
    }
    int left = border(at, grp + 1) - border(at, grp);
    int r = at.r;
    Req rq = request_of<TR>(a, r);
    const Item it = item_of<TR>(a, rq, at.off);
    int h = it.h, t = it.t, u0 = it.u;
    while (true) {
        const int end = tile_end<TR>(a, rq, t);
        const int units = tile_units<TR>(a, rq, t);
        const int u1 = min(units, u0 + left);
        const int t0 = rq.lo + u0 * kUnit, t1 = min(end, rq.lo + u1 * kUnit);
        const int trow = table_row<LISTS>(a, r, h);
        const bool whole = u0 == 0 && u1 == units;
        const int row0 = t * TR + wave * 16 * RT;  // the wave's rows
        bf16x8_t qf[RT][KS];
#pragma unroll
        for (int x = 0; x < RT; ++x) load_q<FP8, D>(a, rq, r, h, row0 + x * 16 + c, lane, qf[x]);
        f32x4_t acc[RT][DV];
        float m[RT], l[RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            m[x] = -INFINITY;
            l[x] = 0.f;
#pragma unroll
            for (int j = 0; j < DV; ++j) acc[x][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        // tiles [mid0, mid1) are seen whole by every row of the workgroup
        const Plain plain = plain_of<RT * kWaves>(a, rq, r, t * TR, c, t1);
        const int mid0 = min(t0 + max(0, plain.lo - t0 + kTile - 1) / kTile * kTile, t1);
        const int mid1 = max(mid0, t0 + (max(plain.hi, t0) - t0) / kTile * kTile);
        // a chain's wave sees nothing behind its last row's node
        const int wend = a.mask ? t1 : min(t1, rq.ctx + (min(row0 + 16 * RT, rq.rows) - 1) / a.G + 1);
        const bool idle = row0 >= rq.rows || !rq.ok;
        int bad = 0;        // a bad page was met
        bool rare = false;  // values left the products
        // (no load but the next tile's is under way while this one is worked
        // on: masks are laid beside the tile.  A load that a branch may issue
        // makes the compiler wait for all of them where the branch joins.)
        if (rq.ok) {
            Stage<FP8, D> st;
            // the next tile's, and this thread's row's sight of it
            const auto ask = [&](int page, int t_at) {
                stage_load<FP8, D>(a, page, h, t_at, end, wave, lane, st);
                if (a.mask && tid < TR && (t_at < mid0 || t_at >= mid1))
                    load_bits<FP8, D>(a, rq, r, query_of(a, rq, r, t * TR + here(tid)).node, t_at, st);
            };
            const auto keep = [&](int buf, int t_at) {
                const bool part = t_at < mid0 || t_at >= mid1;
                stage_store<FP8, D>(a, sh, buf, t_at, end, part, wave, lane, st);
                if (part && tid < TR)
                    sh.sight[buf][tid] = stage_sight<FP8, D>(a, rq, t_at, query_of(a, rq, r, t * TR + here(tid)), st);
            };
            ask(stage_page(a, trow, t0, end, wave), t0);
            int page = stage_page(a, trow, t0 + kTile, end, wave);
            __syncthreads();  // the last item's reads are done
            keep(0, t0);
            __syncthreads();
            int b = 0;
            for (int tile = t0; tile < t1; tile += kTile, b ^= 1) {
                const bool more = tile + kTile < t1;
                const bool part = tile < mid0 || tile >= mid1;
                if (more) ask(page, tile + kTile);
                page = stage_page(a, trow, tile + 2 * kTile, end, wave);  // in time for the next load
                int flags[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) flags[i] = __builtin_amdgcn_readfirstlane(sh.flags[b][i]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int tok = tile + kStep * half;
                    if (idle || tok >= wend) break;
                    // ---- scores
                    f32x4_t s[RT][2];
#pragma unroll
                    for (int x = 0; x < RT; ++x)
                        for (int hf = 0; hf < 2; ++hf) s[x][hf] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                    // operands come from shared memory well ahead of their products
                    u32x4_t kf[2][KS];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) kf[hf][ks] = sh.k[b][2 * half + hf][ks][lane];
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                            for (int x = 0; x < RT; ++x)
                                s[x][hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8_t, kf[hf][ks]), qf[x][ks], s[x][hf], 0, 0, 0);
                    const float sc = FP8 ? sh.sc[b][half][lane] : 0.f;
                    const int fl0 = half ? flags[2] : flags[0], fl1 = half ? flags[3] : flags[1];
                    const int off = fl0 >> 1 | (fl1 & 2);  // halves in a bad page
                    bad |= off;
                    const bool masked = part || off;
                    uint32_t seen[RT];
                    float p[RT][8], top[RT];
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        seen[x] = 0xffu;
                        if (part) {
                            const uint64_t sight = sh.sight[b][wave * 16 * RT + x * 16 + c];
                            seen[x] = lane_bits((uint32_t)(half ? sight >> 32 : sight), g);
                        }
                        top[x] = peak<FP8>(s[x], sc, a.scale2, masked, seen[x], off, p[x]);
                    }
                    rare |= (fl0 | fl1) & 1;
                    lift(top, m, l, acc);
                    // ---- product; the first operands come while the weights are made
                    const auto load_vf = [&](int j0, u32x4_t (&vf)[4]) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const u32x2_t lo = sh.v[b][half][j0 + j][0][lane], hi = sh.v[b][half][j0 + j][1][lane];
                            vf[j] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
                        }
                    };
                    u32x4_t vf[DV / 4][4];
                    load_vf(0, vf[0]);
                    __builtin_amdgcn_sched_barrier(0);
                    u32x4_t pw[RT];
#pragma unroll
                    for (int x = 0; x < RT; ++x) pw[x] = weigh<FP8>(p[x], sc, a.scale2, m[x], l[x]);
#pragma unroll
                    for (int q = 0; q < DV / 4; ++q) {
                        __builtin_amdgcn_sched_barrier(0);
                        if (q + 1 < DV / 4) load_vf(4 * (q + 1), vf[q + 1]);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int x = 0; x < RT; ++x)
                                acc[x][4 * q + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8_t, vf[q][j]), __builtin_bit_cast(bf16x8_t, pw[x]),
                                    acc[x][4 * q + j], 0, 0, 0);
                    }
                }
                if (more) keep(b ^ 1, tile + kTile);
                __syncthreads();
            }
        }
        if (rare) {
#pragma unroll 1
            for (int s = t0; s < wend; s += kTile) {
                if (s >= mid0 && s < mid1) continue;
#pragma unroll
                for (int x = 0; x < RT; ++x)
                    add_rare<FP8, D>(a, rq, r, h, trow, row0 + x * 16 + c, s, min(s + kTile, wend), lane, acc[x]);
            }
        }
        if (bad && lane == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        // ---- the wave's rows
        const int el = here(lane), ec = el & 15, eg = el >> 4;
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            l[x] = column_sum(l[x]);
            const int lr = wave * 16 * RT + x * 16 + ec, row = t * TR + lr;
            if (row >= rq.rows) continue;
            const Query q = query_of(a, rq, r, row);
            if (!rq.ok || q.pos < rq.ctx) {
                l[x] = NAN;
                if (eg == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
            }
            if (whole) {
                const size_t orow = ((size_t)r * a.M + q.node) * a.Hq + h * a.G + (row - q.node * a.G);
                if (l[x] == 0.f) {  // no weight at all: o is 0, whatever V holds
                    l[x] = 1.f;
                    m[x] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < DV; ++j) acc[x][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
                const float inv = 1.f / l[x];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint16_t *op = a.out + orow * D + DV * (4 * eg + i);
#pragma unroll
                    for (int j = 0; j < DV; j += 4)
                        *(u32x2_t *)(op + j) = u32x2_t{pack_bf16(acc[x][j][i] * inv, acc[x][j + 1][i] * inv),
                                                        pack_bf16(acc[x][j + 2][i] * inv, acc[x][j + 3][i] * inv)};
                }
                if (eg == 0 && a.lse) a.lse[orow] = (m[x] + log2f(l[x])) * (float)kLn2;
            } else {
                // as the lanes hold it, a kilobyte a store (rows side by side, as the
                // output has them, were 16 bytes a line: 24.0 us against 19.4 for one
                // tree of 48 nodes behind 4 k tokens)
                float *pp = a.part + (size_t)(2 * grp + (u0 == 0)) * a.part_stride;
                float *po = pp + (wave * RT + x) * 16 * D + 4 * el;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < DV; j += 4)
                        *(f32x4_t *)(po + (i * (DV / 4) + j / 4) * 256) =
                            f32x4_t{acc[x][j][i], acc[x][j + 1][i], acc[x][j + 2][i], acc[x][j + 3][i]};
                if (eg == 0) {
                    pp[TR * D + lr] = m[x];
                    pp[TR * D + TR + lr] = l[x];
                }
            }
        }
        // ---- the next item
        left -= u1 - u0;
        if (left <= 0) {
            if (tid == 0) write_cut<TR>(a, at, grp, u0 == 0 && !whole, r, rq, h, t, units - u1);
            return;
        }
        u0 = 0;
        if (++t >= rq.tiles) {
            t = 0;
            if (++h >= a.c.heads) {
                h = 0;
                do {
                    if (++r >= a.R) return;
                    rq = request_of<TR>(a, r);
                } while (rq.tiles == 0);
            }
        }
    }
}

template <int E>
__device__ __forceinline__ void load_part(const float *p, float (&x)[E]) {
    VecLoad<float, E>::run(p, 0, x);
}

// Joins the parts of the item that range blockIdx.x began and did not finish,
// in token order; a wave's lanes take D / 64 values each of one row.  The
// parts come from other XCDs' memory, a long way off: one load for the cut,
// then every load of up to kJoinParts parts at once.  SPLIT: the four waves
// divide one row's parts (few rows cut into many parts); otherwise each takes
// rows of its own (many rows, in two or three parts).
constexpr int kJoinParts = 16;

template <int D, int TR, bool SPLIT>
__global__ void __launch_bounds__(kBlock) attn_join_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    __shared__ float o_s[kWaves][D], m_s[kWaves], l_s[kWaves];
    const int f = blockIdx.x, n_cuts = *a.n_cuts;
    const Cut cut = a.cuts[f];
    if (f >= n_cuts || cut.rows == 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = SPLIT ? blockIdx.y : blockIdx.y * kWaves + wave;
    if (lr >= cut.rows) return;
    const int n = cut.parts;
    auto slot = [&](int i) -> const float * {
        return a.part + (size_t)(2 * (f + i) + (i == 0)) * a.part_stride;
    };
    float m = -INFINITY, sum = 0.f, o[E];
    for (int q = 0; q < E; ++q) o[q] = 0.f;
    for (int i0 = SPLIT ? wave * kJoinParts : 0; i0 < n; i0 += SPLIT ? kBlock / 64 * kJoinParts : kJoinParts) {
        const int cnt = min(kJoinParts, n - i0);
        const float *p = slot(min(i0 + lane, n - 1)) + TR * D + lr;
        const float mi = lane < cnt ? p[0] : -INFINITY, li = lane < cnt ? p[TR] : 0.f;
        float x[kJoinParts][E];
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k)
            if (k < cnt) load_part(slot(i0 + k) + (size_t)lr * D + lane * E, x[k]);
        const float top = fmaxf(wave_max(mi), m);
        const float ref = top == -INFINITY ? 0.f : top;
        const float w = __builtin_amdgcn_exp2f(mi - ref), back = __builtin_amdgcn_exp2f(m - ref);
        sum = sum * back + wave_sum_f(w * li);
        for (int q = 0; q < E; ++q) o[q] *= back;
        m = top;
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k)
            if (k < cnt) {
                const float wk = readlane_f(w, k);
#pragma unroll
                for (int q = 0; q < E; ++q) o[q] += wk * x[k][q];
            }
    }
    if constexpr (SPLIT) {
        for (int q = 0; q < E; ++q) o_s[wave][lane * E + q] = o[q];
        if (lane == 0) {
            m_s[wave] = m;
            l_s[wave] = sum;
        }
        __syncthreads();
        if (wave) return;
        m = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
        const float ref = m == -INFINITY ? 0.f : m;
        sum = 0.f;
        for (int q = 0; q < E; ++q) o[q] = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float wk = __builtin_amdgcn_exp2f(m_s[w] - ref);
            sum += wk * l_s[w];
            for (int q = 0; q < E; ++q) o[q] += wk * o_s[w][lane * E + q];
        }
    }
    const int row = cut.row0 + lr, nd = row / a.G;
    const size_t orow = (size_t)(cut.node0 + nd) * a.Hq + cut.h * a.G + (row - nd * a.G);
    if (sum == 0.f) {  // no weight at all: o is 0, whatever V holds
        sum = 1.f;
        m = -INFINITY;
        for (int q = 0; q < E; ++q) o[q] = 0.f;
    }
    const float inv = 1.f / sum;
    uint16_t *op = a.out + orow * D + lane * E;
    if constexpr (E == 1) op[0] = (uint16_t)pack_bf16(o[0] * inv, 0.f);
    else if constexpr (E == 2) *(uint32_t *)op = pack_bf16(o[0] * inv, o[1] * inv);
    else *(uint2 *)op = make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    if (lane == 0 && a.lse) a.lse[orow] = (m + log2f(sum)) * (float)kLn2;
}

// The same for attn_wide_kernel's parts, which lie as its lanes held them: a
// wave takes 16 rows by 16 of their values, a kilobyte of each part.
template <int D, int TR>
__global__ void __launch_bounds__(kBlock) attn_wide_join_kernel(AttnArgs a) {
    constexpr int DV = D / 16;
    const int f = blockIdx.x, n_cuts = *a.n_cuts;
    const Cut cut = a.cuts[f];
    if (f >= n_cuts) return;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int unit = blockIdx.y * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rb = unit / DV, piece = unit - rb * DV, lr = 16 * rb + c;
    if (16 * rb >= cut.rows) return;
    const int n = cut.parts;
    float m = -INFINITY, sum = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < n; i0 += kJoinParts) {
        const int cnt = min(kJoinParts, n - i0);
        float mi[kJoinParts], li[kJoinParts];
        f32x4_t x[kJoinParts];
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) {
            mi[k] = -INFINITY;
            if (k < cnt) {
                const float *p = a.part + (size_t)(2 * (f + i0 + k) + (i0 + k == 0)) * a.part_stride;
                mi[k] = p[TR * D + lr];
                li[k] = p[TR * D + TR + lr];
                x[k] = *(const f32x4_t *)(p + unit * 256 + 4 * lane);
            }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) top = fmaxf(top, mi[k]);
        const float ref = top == -INFINITY ? 0.f : top, back = __builtin_amdgcn_exp2f(m - ref);
        sum *= back;
        o *= back;
        m = top;
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k)
            if (k < cnt) {
                const float w = __builtin_amdgcn_exp2f(mi[k] - ref);
                sum += w * li[k];
                o += w * x[k];
            }
    }
    if (lr >= cut.rows) return;
    const int row = cut.row0 + lr, nd = row / a.G;
    const size_t orow = (size_t)(cut.node0 + nd) * a.Hq + cut.h * a.G + (row - nd * a.G);
    if (sum == 0.f) {  // no weight at all: o is 0, whatever V holds
        sum = 1.f;
        m = -INFINITY;
        o = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    o *= 1.f / sum;
    // piece = i (DV / 4) + j / 4: the lane's values d = DV (4 g + i) + j on
    const int i = piece / (DV / 4), j = 4 * (piece - i * (DV / 4));
    *(u32x2_t *)(a.out + orow * D + DV * (4 * g + i) + j) = u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    if (piece == 0 && g == 0 && a.lse) a.lse[orow] = (m + log2f(sum)) * (float)kLn2;
}

// Which launch a call takes and its row tile.  A request's largest count of
// rows per key head decides.  Up to 16 the waves of a workgroup divide the
// tokens; more rows divide the waves, which read K and V from HBM once for all
// of them.  For e4m3 the first form holds up to 32 rows (two tiles a wave) and
// is the faster one there (64 users, 32 rows, 4 k tokens: 91.6 us, the other
// 95; the other way round for bf16, 136.5 and 134.3), but for D = 256, where two
// tiles leave too few registers (24 rows: 162 us, the other 156).
// Beside each other three 16-row tiles a wave reach 781 TFLOP/s on long chunks
// against 649 with two (D = 128, e4m3: each operand from shared memory serves
// three products), so two are taken where they leave over 13% fewer rows
// empty (16 trees of 64 nodes, 256 rows: 97 us against 104; 192 rows: 81.8
// against 80.3).  A small batch, up to 48 rows to a compute unit, takes one:
// more workgroups with less to store for the join, for pages read again from
// L2 (one tree of 48 nodes behind 200 tokens 14.0 us against 20.1, behind 4 k
// 27.7 and 31.4, but behind 30 k 72 and 68; 8 trees, the rule's last, 50.3 and
// 53.6, 16 trees 93 and 81; between them it is not measured).
struct Shape {
    bool wide;
    int RT, TR, groups;
};
constexpr int64_t kSmallBatch = 48 * (kMaxGroups / 2);
// rows: a request's per key head; heads: key heads of all requests.
inline Shape shape_of(int64_t rows, int64_t heads, int D, bool fp8) {
    Shape s;
    s.wide = rows > (fp8 && D <= 128 ? 32 : 16);
    if (!s.wide) s.RT = rows <= 16 ? 1 : 2;
    else if (D == 256 || rows <= 64 || rows * heads <= kSmallBatch) s.RT = 1;
    else {
        const int64_t two = (rows + 127) / 128 * 128, three = (rows + 191) / 192 * 192;
        s.RT = two * 100 < three * 87 ? 2 : 3;
    }
    s.TR = 16 * s.RT * (s.wide ? kWaves : 1);
    s.groups = D <= 128 ? kMaxGroups : kMaxGroups / 2;
    return s;
}

template <bool LISTS, bool FP8, int D, int RT, bool WIDE>
static void launch_attn(const AttnArgs &a, hipStream_t st) {
    constexpr int TR = 16 * RT * (WIDE ? kWaves : 1);
    if constexpr (WIDE) {
        hipLaunchKernelGGL((attn_wide_kernel<FP8, D, RT, LISTS>), dim3(a.groups), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL((attn_wide_join_kernel<D, TR>), dim3(a.groups - 1, TR * D / 256 / kWaves), dim3(kBlock), 0, st, a);
    } else {
        hipLaunchKernelGGL((attn_kernel<FP8, D, RT, LISTS>), dim3(a.groups), dim3(kBlock), 0, st, a);
        // items enough for every eighth range: eight parts an item at most, on
        // the average; fewer items: more parts than one wave reads at a time
        // (one user's 30 k tokens: 32.6 us with the parts divided, 36.0
        // without; 64 users, 32 rows: 141.5 and 137.2)
        const int64_t items = (int64_t)a.R * a.c.heads * ((a.M * a.G + TR - 1) / TR);
        if (items * 8 >= a.groups)
            hipLaunchKernelGGL((attn_join_kernel<D, TR, false>), dim3(a.groups - 1, TR / kWaves), dim3(kBlock), 0, st, a);
        else
            hipLaunchKernelGGL((attn_join_kernel<D, TR, true>), dim3(a.groups - 1, TR), dim3(kBlock), 0, st, a);
    }
}
template <bool LISTS, bool FP8, int D>
static void launch_attn(const AttnArgs &a, const Shape &s, hipStream_t st) {
    if (s.wide) {
        if (s.RT == 1) launch_attn<LISTS, FP8, D, 1, true>(a, st);
        else if constexpr (D <= 128) {
            if (s.RT == 2) launch_attn<LISTS, FP8, D, 2, true>(a, st);
            else launch_attn<LISTS, FP8, D, 3, true>(a, st);
        }
    } else {
        if (s.RT == 1) launch_attn<LISTS, FP8, D, 1, false>(a, st);
        else if constexpr (FP8 && D <= 128) launch_attn<LISTS, FP8, D, 2, false>(a, st);
    }
}
template <bool LISTS, bool FP8>
static void launch_attn(const AttnArgs &a, int D, const Shape &s, hipStream_t st) {
    if (D == 64) launch_attn<LISTS, FP8, 64>(a, s, st);
    else if (D == 128) launch_attn<LISTS, FP8, 128>(a, s, st);
    else launch_attn<LISTS, FP8, 256>(a, s, st);
}

// Both entry points: pages by the requests' tables, or (LISTS) by the lists of
// every request's key heads.
template <bool LISTS>
static int attend(const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                  int cache_dtype, const float *k_scale, const float *v_scale,
                  int num_pages, int page_size, const int32_t *page_table, int max_pages,
                  const int32_t *ctx_len, const int32_t *n_nodes, const uint32_t *mask,
                  const int32_t *positions, float scale, int window, int R, int M, int Hq,
                  int Hkv, int D, void *out, float *out_lse, void *workspace,
                  size_t workspace_bytes, void *stream) {
    if (R < 0 || M < 1 || Hq < 1 || window < 0 || !isfinite(scale)) return SPEC_EINVAL;
    if (q_dtype != SPEC_BF16) return SPEC_EDTYPE;
    const int bad = check_pages(k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                                page_size, max_pages, Hkv, D);
    if (bad) return bad;
    if (Hq % Hkv) return SPEC_EINVAL;
    const size_t need = spec_tree_attention_workspace_bytes(R, M, Hq, Hkv, D);
    if (!need || R > 65535) return SPEC_EUNSUPPORTED;
    if (LISTS && (int64_t)R * Hkv > 0x7fffffff) return SPEC_EUNSUPPORTED;  // rows of the lists
    if (R == 0) return SPEC_OK;
    if (!q || !ctx_len || !n_nodes || !out || (max_pages > 0 && !page_table)) return SPEC_EINVAL;
    if (mask && window > 0 && !positions) return SPEC_EINVAL;  // a node's index is not its level
    if (((uintptr_t)q | (uintptr_t)out) & 15u) return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, need)) return SPEC_EWORKSPACE;
    AttnArgs a{};
    a.q = (const uint16_t *)q;
    a.c = make_pages(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, page_table,
                     max_pages, Hkv);
    a.ctx_len = ctx_len;
    a.n_nodes = n_nodes;
    a.mask = mask;
    a.positions = positions;
    // a positive factor, so that the largest score is the largest product; 0
    // becomes the smallest normal number (-inf times it is still -inf)
    a.scale2 = fmaxf((float)(fabs((double)scale) * kLog2e), 1.17549435e-38f);
    a.flip = scale < 0.0f ? 0x80008000u : 0u;
    a.R = R;
    a.window = window;
    a.M = M;
    a.W = (M + 31) / 32;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.out = (uint16_t *)out;
    a.lse = out_lse;
    a.ctl = (Control *)workspace;
    a.cuts = (Cut *)((char *)workspace + sizeof(Control));
    a.n_cuts = (int *)(a.cuts + kMaxGroups);
    a.part = (float *)(a.cuts + kMaxGroups + 1);
    const Shape s = shape_of((int64_t)M * a.G, (int64_t)R * Hkv, D, cache_dtype == SPEC_E4M3);
    a.groups = s.groups;
    a.part_stride = s.TR * (D + 2);
    // the batch's units must count in 31 bits
    const int64_t tiles = ((int64_t)M * a.G + s.TR - 1) / s.TR;
    const int64_t units = (((int64_t)max_pages << a.c.shift) + kUnit - 1) / kUnit + 1;
    if ((double)R * Hkv * (double)tiles * (double)units >= 2147483647.0) return SPEC_EUNSUPPORTED;
    if (cache_dtype == SPEC_E4M3) launch_attn<LISTS, true>(a, D, s, (hipStream_t)stream);
    else launch_attn<LISTS, false>(a, D, s, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_tree_attention_workspace_bytes(int R, int M, int Hq, int Hkv, int D) {
    if (R < 0 || M < 1 || M > SPEC_TREE_MAX_NODES || Hkv < 1 || Hq < 1 || Hq % Hkv ||
        Hq / Hkv > 64 || (D != 64 && D != 128 && D != 256))
        return 0;
    // the largest tiles that these sizes or smaller ones take
    const int rows = M * (Hq / Hkv);
    const size_t TR = rows <= 16 ? 16 : D == 256 || rows <= 64 ? 64 : 192;
    const size_t groups = D <= 128 ? kMaxGroups : kMaxGroups / 2;
    return sizeof(Control) + sizeof(Cut) * (kMaxGroups + 1) + 2 * groups * TR * (D + 2) * sizeof(float);
}

int spec_tree_attention(const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                        int cache_dtype, const float *k_scale, const float *v_scale,
                        int num_pages, int page_size, const int32_t *page_table, int max_pages,
                        const int32_t *ctx_len, const int32_t *n_nodes, const uint32_t *mask,
                        const int32_t *positions, float scale, int window, int R, int M, int Hq,
                        int Hkv, int D, void *out, float *out_lse, void *workspace,
                        size_t workspace_bytes, void *stream) {
    return attend<false>(q, q_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                         page_size, page_table, max_pages, ctx_len, n_nodes, mask, positions, scale,
                         window, R, M, Hq, Hkv, D, out, out_lse, workspace, workspace_bytes, stream);
}

int spec_page_attention(const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                        int cache_dtype, const float *k_scale, const float *v_scale,
                        int num_pages, int page_size, const int32_t *page_lists, int list_pages,
                        const int32_t *list_len, const int32_t *n_nodes, const uint32_t *mask,
                        float scale, int R, int M, int Hq, int Hkv, int D, void *out,
                        float *out_lse, void *workspace, size_t workspace_bytes, void *stream) {
    return attend<true>(q, q_dtype, k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                        page_size, page_lists, list_pages, list_len, n_nodes, mask, nullptr, scale,
                        0, R, M, Hq, Hkv, D, out, out_lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
