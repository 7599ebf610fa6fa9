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

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStep = 32;              // tokens a wave takes at a time
constexpr int kUnit = kStep * kWaves;  // tokens of one unit of work
constexpr int kMaxGroups = 512;        // workgroups of the attention launch
constexpr float kLazy = 8.0f;          // a maximum may lag by this many powers of two

struct AttnArgs {
    const uint16_t *q;           // [R][M][Hq][D] bf16
    Pages c;
    const int32_t *ctx_len, *n_nodes;
    const uint32_t *mask;        // [R][M][W], null: chain
    const int32_t *positions;    // [R][M], null: ctx + v
    float scale2;                // scale * log2(e)
    int window, R, M, W, Hq, G;
    uint16_t *out;
    float *lse;
    Control *ctl;
    float *part;                 // [2 groups][part_stride]
    int groups, part_stride;
};

// ---------------------------------------------------------------------------
// the work list
// ---------------------------------------------------------------------------

struct Req {
    int n, ctx, rows, tiles;     // live nodes, context, query rows per key head, row tiles
    int lo;                      // first token any row sees
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
    q.lo = a.window ? max(0, q.ctx - a.window + 1) & ~(kStep - 1) : 0;
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
__device__ __forceinline__ int64_t head_units(const AttnArgs &a, const Req &q) {
    if (q.tiles == 0) return 0;
    if (a.mask || !q.ok) return (int64_t)q.tiles * tile_units<TR>(a, q, 0);
    int64_t s = 0;
    for (int t = 0; t < q.tiles; ++t) s += tile_units<TR>(a, q, t);
    return s;
}

struct Place {
    int r;                       // request
    int64_t off;                 // units into it
    int64_t total;               // units of the whole batch
    int parts;                   // ranges with work: min(groups, total)
};

__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The first unit of range `num` of `parts`.
__device__ __forceinline__ int64_t border(const Place &p, int num) {
    return p.total * num / p.parts;
}

// The request that the first unit of a range falls into: of range `num`, or,
// with XCD, of the range of workgroup `num` when neighbouring ranges, which
// often share a key head's pages, go to one XCD (num becomes the range; -1:
// none).  Every thread of the workgroup gets the same answer.
template <int TR, bool XCD>
__device__ __forceinline__ Place find_unit(const AttnArgs &a, int &num) {
    __shared__ int64_t sum_s[kWaves];
    __shared__ int r_s;
    __shared__ int64_t off_s;
    const int tid = threadIdx.x;
    const int chunk = (a.R + kBlock - 1) / kBlock;
    const int r0 = min(tid * chunk, a.R), r1 = min(r0 + chunk, a.R);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += head_units<TR>(a, request_of<TR>(a, r)) * a.c.heads;
    // scan inside the wave, then over the four waves
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t up = __shfl_up(inc, o, 64);
        if ((tid & 63) >= o) inc += up;
    }
    if ((tid & 63) == 63) sum_s[tid >> 6] = inc;
    __syncthreads();
    int64_t base = 0;
    Place p;
    p.total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < (tid >> 6)) base += sum_s[w];
        p.total += sum_s[w];
    }
    p.total = uniform(p.total);
    p.parts = (int)min((int64_t)a.groups, p.total);
    p.r = a.R;
    p.off = 0;
    if (XCD) {
        const int per = (p.parts + 7) >> 3, in = num >> 3;
        num = in < per ? (num & 7) * per + in : a.groups;
    }
    if (num >= p.parts) {
        num = -1;
        return p;
    }
    const int64_t at = border(p, num);
    const int64_t first = base + inc - mine;
    if (at >= first && at < first + mine) {
        int64_t left = at - first;
        int r = r0;
        for (; r < r1; ++r) {
            const int64_t u = head_units<TR>(a, request_of<TR>(a, r)) * a.c.heads;
            if (left < u) break;
            left -= u;
        }
        r_s = r;
        off_s = left;
    }
    __syncthreads();
    p.r = __builtin_amdgcn_readfirstlane(r_s);
    p.off = uniform(off_s);
    return p;
}

struct Item {
    int h, t, u;                 // key head, row tile, unit in the item
    int units;
};
template <int TR>
__device__ __forceinline__ Item item_of(const AttnArgs &a, const Req &rq, int64_t off) {
    const int64_t hu = head_units<TR>(a, rq);
    Item i;
    i.h = (int)(off / hu);
    i.t = 0;
    int64_t rem = off - i.h * hu;
    if (a.mask || !rq.ok) {
        i.units = tile_units<TR>(a, rq, 0);
        i.t = (int)(rem / i.units);
        rem -= (int64_t)i.t * i.units;
    } else {
        while (rem >= (i.units = tile_units<TR>(a, rq, i.t))) {
            rem -= i.units;
            ++i.t;
        }
    }
    i.u = (int)rem;
    return i;
}

// ---------------------------------------------------------------------------
// one wave's step
// ---------------------------------------------------------------------------

template <bool FP8, int D> struct Tile {
    static constexpr int KS = D / 32;              // contraction steps of Q K^T
    static constexpr int DV = D / 16;              // values of V a lane holds per token
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int KV = D * EB / 64;         // 16-byte K loads per 16 tokens
    static constexpr int VW = DV * EB / 4;         // 32-bit words of V per token
    uint4 k[2][KV];
    uint32_t v[8][VW];
    float4 ks[2], vs[2];                           // scales (FP8)
};

// N consecutive 32-bit words (N a multiple of 4, or 1 or 2: aligned to them).
template <int N>
__device__ __forceinline__ void load_words(const char *p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *(const uint32_t *)p;
    } else if constexpr (N == 2) {
        const uint2 x = *(const uint2 *)p;
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *(const uint4 *)(p + 4 * i);
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

__device__ __forceinline__ Half halves_of(const AttnArgs &a, int r, int h, int t, int L) {
    Half x;
    x.bad = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int tt = t + 16 * s < L ? t + 16 * s : t;  // a half behind the end is not used
        int page = a.c.table[(int64_t)r * a.c.max_pages + (tt >> a.c.shift)];
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
    const int c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const char *p = (const char *)a.c.k + (x.row[s] + c) * (D * Tile<FP8, D>::EB) + g * 16;
#pragma unroll
        for (int i = 0; i < Tile<FP8, D>::KV; ++i) t.k[s][i] = *(const uint4 *)(p + i * 64);
        if constexpr (FP8) t.ks[s] = *(const float4 *)(a.c.k_scale + x.row[s] + 4 * g);
    }
}
template <bool FP8, int D>
__device__ __forceinline__ void load_v(const AttnArgs &a, const Half &x, int lane, Tile<FP8, D> &t) {
    typedef Tile<FP8, D> TT;
    const int c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const char *p = (const char *)a.c.v + (x.row[s] + 4 * g) * (D * TT::EB) + c * (TT::VW * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words(p + i * (D * TT::EB), t.v[4 * s + i]);
        if constexpr (FP8) t.vs[s] = *(const float4 *)(a.c.v_scale + x.row[s] + 4 * g);
    }
}

// The A operand of contraction step ks of the 16 tokens of half s.
template <bool FP8, int D>
__device__ __forceinline__ bf16x8_t k_frag(const Tile<FP8, D> &t, int s, int ks) {
    if constexpr (!FP8) {
        return __builtin_bit_cast(bf16x8_t, t.k[s][ks]);
    } else {
        const uint4 w = t.k[s][ks >> 1];
        const uint32_t x = ks & 1 ? w.z : w.x, y = ks & 1 ? w.w : w.y;
        return __builtin_bit_cast(bf16x8_t, make_uint4(e4m3_bf16<false>(x), e4m3_bf16<true>(x),
                                                       e4m3_bf16<false>(y), e4m3_bf16<true>(y)));
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

__device__ __forceinline__ bool odd_word(uint32_t w) {  // a NaN or an infinity in it
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Whether the row of node v (position pos) sees token t < L.
__device__ __forceinline__ bool sees(const AttnArgs &a, int t, int ctx, int n, int v, int pos,
                                     const uint32_t *mrow) {
    if (t < ctx) return !a.window || t > pos - a.window;
    const int u = t - ctx;
    if (u >= n) return false;
    return mrow ? (mrow[u >> 5] >> (u & 31)) & 1u : u <= v && (!a.window || v - u < a.window);
}

// ---------------------------------------------------------------------------
// the attention launch
// ---------------------------------------------------------------------------

template <int D, int RT> constexpr int waves_per_simd() {
    return D * RT <= 128 ? 2 : 1;
}

template <bool FP8, int D, int RT>
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
    const Place at = find_unit<TR, true>(a, grp);
    if (grp < 0) return;
    int64_t left = border(at, grp + 1) - border(at, grp);
    int r = at.r;
    Req rq = request_of<TR>(a, r);
    const Item it = item_of<TR>(a, rq, at.off);
    int h = it.h, t = it.t, u0 = it.u;
    while (true) {
        // ---- one item (r, h, t), its units from u0 on
        const int end = tile_end<TR>(a, rq, t);
        const int units = tile_units<TR>(a, rq, t);
        const int u1 = (int)min((int64_t)units, u0 + left);
        const int t0 = rq.lo + u0 * kUnit, t1 = min(end, rq.lo + u1 * kUnit);
        const bool whole = u0 == 0 && u1 == units;
        // ---- the rows of this lane's column
        bf16x8_t qf[RT][KS];
        int node[RT], pos[RT];
        bool rowbad[RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            const int row = min(t * TR + x * 16 + c, rq.rows - 1);
            node[x] = row / a.G;
            const size_t nd = (size_t)r * a.M + node[x];
            pos[x] = a.positions ? a.positions[nd] : rq.ctx + node[x];
            rowbad[x] = !rq.ok || pos[x] < rq.ctx;
            const uint16_t *qp = a.q + (nd * a.Hq + h * a.G + (row - node[x] * a.G)) * D;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                qf[x][ks] = __builtin_bit_cast(bf16x8_t, *(const uint4 *)(qp + q_chunk<FP8>(ks, g)));
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
        // tokens before `plain` are seen by every row of the tile
        int plain = rq.ctx;
        if (!a.mask) plain += t * TR / a.G + 1;
        if (a.window) plain = 0;
        plain = min(plain, t1);
        int tok = t0 + wave * kStep;
        if (rq.ok && tok < t1) {
            TT kv;
            Half cur = halves_of(a, r, h, tok, end);
            load_k<FP8, D>(a, cur, lane, kv);
            load_v<FP8, D>(a, cur, lane, kv);
            while (true) {
                const int nxt = tok + kUnit;
                const bool more = nxt < t1;
                Half nh = cur;
                if (more) nh = halves_of(a, r, h, nxt, end);
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
                float ksc[8], vsc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ksc[i] = a.scale2;
                    vsc[i] = 1.f;
                }
                if constexpr (FP8) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        ksc[4 * hf] *= kv.ks[hf].x;
                        ksc[4 * hf + 1] *= kv.ks[hf].y;
                        ksc[4 * hf + 2] *= kv.ks[hf].z;
                        ksc[4 * hf + 3] *= kv.ks[hf].w;
                        vsc[4 * hf] = kv.vs[hf].x;
                        vsc[4 * hf + 1] = kv.vs[hf].y;
                        vsc[4 * hf + 2] = kv.vs[hf].z;
                        vsc[4 * hf + 3] = kv.vs[hf].w;
                    }
                }
                if (more) load_k<FP8, D>(a, nh, lane, kv);
                __builtin_amdgcn_sched_barrier(0);
                const bool masked = tok + kStep > plain || cur.bad;
                uint32_t seen[RT];  // bit i: this lane's token i is seen by its row
                uint4 pw[RT];
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    float p[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = s[x][i >> 2][i & 3] * ksc[i];
                    seen[x] = 0xffu;
                    if (masked) {
                        const uint32_t *mrow = a.mask ? a.mask + ((size_t)r * a.M + node[x]) * a.W : nullptr;
                        seen[x] = 0u;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int tt = tok + 16 * (i >> 2) + 4 * g + (i & 3);
                            const bool see = sees(a, tt, rq.ctx, rq.n, node[x], pos[x], mrow);
                            seen[x] |= (uint32_t)see << i;
                            p[i] = !see ? -INFINITY : (cur.bad >> (i >> 2)) & 1 ? NAN : p[i];
                        }
                    }
                    float tm = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])),
                                     fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
                    tm = fmaxf(tm, __shfl_xor(tm, 16, 64));
                    tm = fmaxf(tm, __shfl_xor(tm, 32, 64));
                    if (__any(tm > m[x] + kLazy)) {
                        const float mn = fmaxf(m[x], tm);
                        const float al = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[x] - mn);
                        l[x] *= al;
#pragma unroll
                        for (int j = 0; j < DV; ++j) acc[x][j] *= al;
                        m[x] = mn;
                    }
                    const float ref = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p[i] = __builtin_amdgcn_exp2f(p[i] - ref);
                        l[x] += p[i];
                    }
                    if constexpr (FP8) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            p[i] = !masked || (seen[x] >> i & 1u) ? p[i] * vsc[i] : 0.f;
                    }
                    // weights in bf16 (2^-8 relative, as the output's own rounding)
                    pw[x] = make_uint4(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]),
                                       pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
                }
                uint32_t odd = 0u;  // bit i: token i of this lane holds a NaN or an infinity
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool live = tok + 16 * (i >> 2) + 4 * g + (i & 3) < t1;
#pragma unroll
                        for (int w = 0; w < TT::VW; ++w) kv.v[i][w] = live ? kv.v[i][w] : 0u;
                        bool o = false;
#pragma unroll
                        for (int w = 0; w < DV / 2; ++w) o |= odd_word(v_word<FP8, D>(kv, i, w));
                        odd |= (uint32_t)o << i;
                    }
                }
                if (__any(odd != 0u)) {
                    // weight 0 times such a value is not 0: rows that do not
                    // see the token must not meet it.  These tokens leave the
                    // product and are added one by one where they are seen.
                    uint32_t all = odd;  // over the 16 lanes that hold a token's row
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) all |= __shfl_xor(all, o, 64);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int w = 0; w < TT::VW; ++w) kv.v[i][w] = all >> i & 1u ? 0u : kv.v[i][w];
#pragma unroll 1
                    for (int q = 0; q < 32; ++q) {
                        const int tg = q >> 3, ti = q & 7;  // lane group and index of the token
                        if (!(__shfl((int)all, tg * 16, 64) >> ti & 1)) continue;
                        const int64_t row = (ti & 4 ? cur.row[1] : cur.row[0]) + 4 * tg + (ti & 3);
#pragma unroll
                        for (int x = 0; x < RT; ++x) {
                            const uint32_t lo = ti & 4 ? (ti & 2 ? pw[x].w : pw[x].z)
                                                       : (ti & 2 ? pw[x].y : pw[x].x);
                            const float mine = ti & 1 ? bf16_hi(lo) : bf16_lo(lo);
                            const float pv = __shfl(mine, tg * 16 + c, 64);
                            const bool see = __shfl((int)seen[x], tg * 16 + c, 64) >> ti & 1;
#pragma unroll
                            for (int j = 0; j < DV; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int64_t e = row * D + DV * (4 * g + i) + j;
                                    float val;
                                    if constexpr (FP8) val = bf16_lo(e4m3_bf16<false>(((const uint8_t *)a.c.v)[e]));
                                    else val = bf16_lo(((const uint16_t *)a.c.v)[e]);
                                    if (see) acc[x][j][i] += pv * val;
                                }
                        }
                    }
                }
                // ---- product
#pragma unroll
                for (int w = 0; w < DV / 2; ++w) {
                    uint32_t b[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[i] = v_word<FP8, D>(kv, i, w);
                    uint4 f0, f1;
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
                if (cur.bad && lane == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
                if (!more) break;
                load_v<FP8, D>(a, nh, lane, kv);
                __builtin_amdgcn_sched_barrier(0);
                cur = nh;
                tok = nxt;
            }
        }
        // ---- join the four waves, 16 rows at a time
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            l[x] += __shfl_xor(l[x], 16, 64);
            l[x] += __shfl_xor(l[x], 32, 64);
            if (rowbad[x]) l[x] = NAN;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < DV; j += 4)
                    *(float4 *)&o_s[wave][c][DV * (4 * g + i) + j] =
                        make_float4(acc[x][j][i], acc[x][j + 1][i], acc[x][j + 2][i], acc[x][j + 3][i]);
            if (g == 0) {
                m_s[wave][c] = m[x];
                l_s[wave][c] = l[x];
            }
            __syncthreads();
            const int jr = tid >> 4, e0 = (tid & 15) * DV;  // this thread's row and values
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
                    if (sum == 0.f) {  // nothing seen: o is 0
                        sum = 1.f;
                        mm = -INFINITY;
                    }
                    const float inv = 1.f / sum;
                    uint16_t *op = a.out + orow * D + e0;
#pragma unroll
                    for (int j = 0; j < DV; j += 4)
                        *(uint2 *)(op + j) = make_uint2(pack_bf16(o[j] * inv, o[j + 1] * inv),
                                                        pack_bf16(o[j + 2] * inv, o[j + 3] * inv));
                    if ((tid & 15) == 0) {
                        if (a.lse) a.lse[orow] = (mm + log2f(sum)) * (float)kLn2;
                        if (!rq.ok || (a.positions && a.positions[(size_t)r * a.M + nd] < rq.ctx))
                            atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
                    }
                } else {
                    float *pp = a.part + (size_t)(2 * grp + (u0 == 0)) * a.part_stride;
                    float *po = pp + (size_t)(x * 16 + jr) * D + e0;
#pragma unroll
                    for (int j = 0; j < DV; j += 4) *(float4 *)(po + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    if ((tid & 15) == 0) {
                        pp[TR * D + x * 16 + jr] = mm;
                        pp[TR * D + TR + x * 16 + jr] = sum;
                    }
                }
            }
        }
        // ---- the next item
        left -= u1 - u0;
        if (left <= 0) return;
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

// Joins the parts of the item that the border between groups b - 1 and b cuts
// first (workgroup x = b - 1), in token order; one wave per row, its lanes
// D / 64 values each.
template <int D, int TR>
__global__ void __launch_bounds__(kBlock) attn_join_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    int b = blockIdx.x + 1;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Place at = find_unit<TR, false>(a, b);
    if (b < 0) return;
    const Req rq = request_of<TR>(a, at.r);
    const Item it = item_of<TR>(a, rq, at.off);
    const int64_t first = border(at, b) - it.u, last = first + it.units;  // the item's units
    if (it.u == 0 || border(at, b - 1) > first) return;  // not cut, or cut by an earlier border
    int e = b;                                           // the last range with units of the item
    while (e + 1 < at.parts && border(at, e + 1) < last) ++e;
    const int h = it.h, t = it.t;
    const int lr = blockIdx.y * kWaves + wave, row = t * TR + lr;
    if (row >= rq.rows) return;
    const int f = b - 1, n = e - f + 1;
    auto slot = [&](int i) -> const float * {
        return a.part + (size_t)(2 * (f + i) + (i == 0)) * a.part_stride;
    };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 64) M = fmaxf(M, slot(i)[TR * D + lr]);
    M = wave_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float sum = 0.f, o[E];
    for (int q = 0; q < E; ++q) o[q] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 64) {
        float w = 0.f, l = 0.f;
        if (i0 + lane < n) {
            const float *p = slot(i0 + lane);
            w = __builtin_amdgcn_exp2f(p[TR * D + lr] - ref);
            l = p[TR * D + TR + lr];
        }
        sum += wave_sum_f(w * l);
        const int cnt = min(64, n - i0);
        for (int i = 0; i < cnt; i += 8) {  // eight loads in flight
            float x[8][E];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                load_part(slot(i0 + min(i + k, cnt - 1)) + (size_t)lr * D + lane * E, x[k]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wi = i + k < cnt ? readlane_f(w, i + k) : 0.f;
                if (i + k < cnt) {
#pragma unroll
                    for (int q = 0; q < E; ++q) o[q] += wi * x[k][q];
                }
            }
        }
    }
    const int nd = row / a.G;
    const size_t node = (size_t)at.r * a.M + nd;
    const size_t orow = node * a.Hq + h * a.G + (row - nd * a.G);
    if (sum == 0.f) {  // nothing seen: o is 0
        sum = 1.f;
        M = -INFINITY;
    }
    const float inv = 1.f / sum;
    uint16_t *op = a.out + orow * D + lane * E;
    if constexpr (E == 1) op[0] = (uint16_t)pack_bf16(o[0] * inv, 0.f);
    else if constexpr (E == 2) *(uint32_t *)op = pack_bf16(o[0] * inv, o[1] * inv);
    else *(uint2 *)op = make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    if (lane == 0) {
        if (a.lse) a.lse[orow] = (M + log2f(sum)) * (float)kLn2;
        if (a.positions && a.positions[node] < rq.ctx)
            atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
    }
}

// Row tiles of 16, 32 or 64 rows: the smallest that takes all rows of the
// largest request; 32 at D = 256, whose accumulators fill the registers.
inline int row_tiles(int64_t rows, int D) {
    return rows <= 16 ? 1 : rows <= 32 || D == 256 ? 2 : 4;
}
inline int groups_of(int RT, int D) { return D * RT <= 128 ? kMaxGroups : kMaxGroups / 2; }

template <bool FP8, int D, int RT>
static void launch_attn(AttnArgs a, hipStream_t st) {
    a.groups = groups_of(RT, D);
    a.part_stride = 16 * RT * (D + 2);
    hipLaunchKernelGGL((attn_kernel<FP8, D, RT>), dim3(a.groups), dim3(kBlock), 0, st, a);
    hipLaunchKernelGGL((attn_join_kernel<D, 16 * RT>), dim3(a.groups - 1, 16 * RT / kWaves),
                       dim3(kBlock), 0, st, a);
}
template <bool FP8>
static void launch_attn(const AttnArgs &a, int D, int RT, hipStream_t st) {
    if (D == 64) {
        if (RT == 1) launch_attn<FP8, 64, 1>(a, st);
        else if (RT == 2) launch_attn<FP8, 64, 2>(a, st);
        else launch_attn<FP8, 64, 4>(a, st);
    } else if (D == 128) {
        if (RT == 1) launch_attn<FP8, 128, 1>(a, st);
        else if (RT == 2) launch_attn<FP8, 128, 2>(a, st);
        else launch_attn<FP8, 128, 4>(a, st);
    } else {
        if (RT == 1) launch_attn<FP8, 256, 1>(a, st);
        else launch_attn<FP8, 256, 2>(a, st);
    }
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_tree_attention_workspace_bytes(int R, int M, int Hq, int Hkv, int D) {
    if (R < 0 || M < 1 || M > SPEC_TREE_MAX_NODES || Hkv < 1 || Hq < 1 || Hq % Hkv ||
        Hq / Hkv > 64 || (D != 64 && D != 128 && D != 256))
        return 0;
    const int RT = row_tiles((int64_t)M * (Hq / Hkv), D);
    return sizeof(Control) + (size_t)2 * groups_of(RT, D) * 16 * RT * (D + 2) * sizeof(float);
}

int spec_tree_attention(const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                        int cache_dtype, const float *k_scale, const float *v_scale,
                        int num_pages, int page_size, const int32_t *page_table, int max_pages,
                        const int32_t *ctx_len, const int32_t *n_nodes, const uint32_t *mask,
                        const int32_t *positions, float scale, int window, int R, int M, int Hq,
                        int Hkv, int D, void *out, float *out_lse, void *workspace,
                        size_t workspace_bytes, void *stream) {
    if (R < 0 || M < 1 || Hq < 1 || window < 0 || !isfinite(scale)) return SPEC_EINVAL;
    if (q_dtype != SPEC_BF16) return SPEC_EDTYPE;
    const int bad = check_pages(k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                                page_size, page_table, max_pages, Hkv, D);
    if (bad) return bad;
    if (Hq % Hkv) return SPEC_EINVAL;
    const size_t need = spec_tree_attention_workspace_bytes(R, M, Hq, Hkv, D);
    if (!need || R > 65535) return SPEC_EUNSUPPORTED;
    if (R == 0) return SPEC_OK;
    if (!q || !ctx_len || !n_nodes || !out) return SPEC_EINVAL;
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
    a.scale2 = (float)(scale * kLog2e);
    a.R = R;
    a.window = window;
    a.M = M;
    a.W = (M + 31) / 32;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.out = (uint16_t *)out;
    a.lse = out_lse;
    a.ctl = (Control *)workspace;
    a.part = (float *)((char *)workspace + sizeof(Control));
    const int RT = row_tiles((int64_t)M * a.G, D);
    if (cache_dtype == SPEC_E4M3) launch_attn<true>(a, D, RT, (hipStream_t)stream);
    else launch_attn<false>(a, D, RT, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
