// cache.hip -- writing, reading and moving rows of the paged key/value cache
// on gfx950.
//
// A head row of D values belongs to D / 8 lanes, 8 values each, so a wave
// holds 512 / D rows and every sum or maximum over a row stays inside it.
#include <math.h>

#include <type_traits>

#include "cache.h"

namespace sv {

// ---------------------------------------------------------------------------
// spec_qkv_write
// ---------------------------------------------------------------------------

struct WriteArgs {
    const void *q, *k, *v;       // token rows, ld_* elements apart
    int64_t ld_q, ld_k, ld_v;
    const void *q_weight, *k_weight;
    float eps;
    const float2 *rope;          // [max_pos][half] (cos, sin)
    int max_pos, half, interleaved;
    const int32_t *positions, *ctx_len, *n_nodes;
    Pages c;
    int M, Hq;
    uint16_t *out_q;
    Control *ctl;
};

__device__ __forceinline__ u32x4_t bf16x8(const float (&x)[8]) {
    return u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                   pack_bf16(x[6], x[7])};
}

// Sum and maximum over the D / 8 lanes of a row, by lane moves.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
    v += dpp_f<kDppSwap1>(v);
    v += dpp_f<kDppSwap2>(v);
    v += dpp_f<kDppHalfMirror>(v);
    if constexpr (LPR >= 16) v += dpp_f<kDppMirror>(v);
    if constexpr (LPR == 32) {
        uint32_t lo, hi;
        lane_pair<16>(__float_as_uint(v), lo, hi);
        v = __uint_as_float(lo) + __uint_as_float(hi);
    }
    return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, dpp_f<kDppSwap1>(v));
    v = fmaxf(v, dpp_f<kDppSwap2>(v));
    v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
    if constexpr (LPR >= 16) v = fmaxf(v, dpp_f<kDppMirror>(v));
    if constexpr (LPR == 32) {
        uint32_t lo, hi;
        lane_pair<16>(__float_as_uint(v), lo, hi);
        v = fmaxf(__uint_as_float(lo), __uint_as_float(hi));
    }
    return v;
}

// The two groups of four values a lane holds, from elements a and b on.  The
// two halves of a rotation are half elements apart: a lane that turns takes
// four of each, so that both values of a pair are its own; the other lanes,
// and all of them for interleaved pairs, take eight in a row.
struct Place {
    int a, b;
    bool in;                     // the lane's values turn
};
__device__ __forceinline__ Place place_of(const WriteArgs &w, int l) {
    Place p;
    const int split = w.interleaved ? 0 : w.half / 4;  // lanes that hold both halves
    p.a = l < split ? 4 * l : 2 * (w.interleaved ? 0 : w.half) + 8 * (l - split);
    p.b = l < split ? w.half + 4 * l : p.a + 4;
    p.in = w.interleaved ? p.a < 2 * w.half : l < split;
    return p;
}

// Four values as they lie in memory.
template <typename T> struct Raw4 {
    uint32_t w[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw4<T> load4(const T *p) {
    Raw4<T> r;
    if constexpr (sizeof(T) == 2) {
        const u32x2_t x = *(const u32x2_t *)p;
        r.w[0] = x[0];
        r.w[1] = x[1];
    } else {
        const u32x4_t x = *(const u32x4_t *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = x[i];
    }
    return r;
}
template <typename T>
__device__ __forceinline__ float value(const Raw4<T> &r, int i) {
    if constexpr (sizeof(T) == 2) return i & 1 ? bf16_hi(r.w[i >> 1]) : bf16_lo(r.w[i >> 1]);
    else return __uint_as_float(r.w[i]);
}

// One workgroup per token: its lanes keep the same values of every head row,
// so the rotation and the weights are read once; ROWS head rows a thread are
// asked for before the first is used.  Few tokens: ROWS = 1 and workgroups
// (y) share a token's rows.  Several tokens a workgroup with the next one's
// rows in flight was slower (150 us against 125 for 16 k tokens of 48 rows:
// the registers cost more waves than the waits).
// Bound by HBM: the projections read, q and the cache written; 16 k tokens of
// 48 rows to e4m3 pages take 74 us, 5.0 TB/s of 365 MB (a large copy: 4.74).
template <typename T, bool FP8, int D, int ROWS>
__global__ void __launch_bounds__(kBlock) qkv_write_kernel(WriteArgs a) {
    constexpr int LPR = D / 8, RPB = kBlock / LPR;
    const int token = blockIdx.x, r = token / a.M, v = token - r * a.M;
    const int tid = threadIdx.x, l = tid & (LPR - 1);
    const int n = a.n_nodes[r], ctx = a.ctx_len[r];
    const bool sane = n >= 0 && n <= a.M && in_table(ctx, n, a.c.max_pages, a.c.shift);
    if (sane && v >= n) return;
    const int Hkv = a.c.heads, rows = a.Hq + 2 * Hkv;
    const int first = blockIdx.y * RPB + tid / LPR, step = gridDim.y * RPB;
    if (!sane) {
        const uint32_t nan2 = pack_bf16(NAN, NAN);
        for (int row = first; row < a.Hq; row += step)
            *(u32x4_t *)(a.out_q + ((size_t)token * a.Hq + row) * D + 8 * l) = u32x4_t{nan2, nan2, nan2, nan2};
        if (first == 0 && l == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        return;
    }
    const Place at = place_of(a, l);
    // the token's place in the cache and its angles
    const int t = ctx + v;
    const int page = a.c.table[(size_t)r * a.c.max_pages + (t >> a.c.shift)];
    const bool good = page >= 0 && page < a.c.num_pages;
    const int pos = a.half && a.positions ? a.positions[token] : t;
    const bool there = !a.half || (pos >= 0 && pos < a.max_pos);
    if ((!good || !there) && first == 0 && l == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
    f32x4_t cs[2] = {};          // (cos, sin) of the lane's four pairs
    if (at.in) {
        const f32x4_t *p = (const f32x4_t *)(a.rope + (size_t)(there ? pos : 0) * a.half +
                                             (a.interleaved ? at.a / 2 : at.a));
        cs[0] = p[0];
        cs[1] = p[1];
    }
    Raw4<T> qw[2], kw[2];
    if (a.q_weight) {
        qw[0] = load4((const T *)a.q_weight + at.a);
        qw[1] = load4((const T *)a.q_weight + at.b);
    }
    if (a.k_weight) {
        kw[0] = load4((const T *)a.k_weight + at.a);
        kw[1] = load4((const T *)a.k_weight + at.b);
    }
    for (int row0 = first; row0 < rows; row0 += ROWS * step) {
        Raw4<T> raw[ROWS][2];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int row = row0 + i * step;
            if (row < rows) {
                const T *src = row < a.Hq ? (const T *)a.q + (int64_t)token * a.ld_q + row * D
                             : row < a.Hq + Hkv ? (const T *)a.k + (int64_t)token * a.ld_k + (row - a.Hq) * D
                                                : (const T *)a.v + (int64_t)token * a.ld_v + (row - a.Hq - Hkv) * D;
                raw[i][0] = load4(src + at.a);
                raw[i][1] = load4(src + at.b);
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int row = row0 + i * step;
            if (row >= rows) break;
            const int kind = row < a.Hq ? 0 : row < a.Hq + Hkv ? 1 : 2;  // q, k, v
            const int head = row - (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + Hkv);
            float x[8];          // values a .. a + 3, then b .. b + 3
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = value(raw[i][q >> 2], q & 3);
            if (kind < 2) {
                if (kind == 0 ? a.q_weight != nullptr : a.k_weight != nullptr) {
                    float ss = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) ss = fmaf(x[q], x[q], ss);
                    const float inv = 1.0f / sqrtf(row_sum<LPR>(ss) * (1.0f / D) + a.eps);
                    if (kind == 0) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) x[q] = x[q] * inv * value(qw[q >> 2], q & 3);
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) x[q] = x[q] * inv * value(kw[q >> 2], q & 3);
                    }
                }
                if (at.in) {
                    float y[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float c = cs[q >> 1][2 * (q & 1)], s = cs[q >> 1][2 * (q & 1) + 1];
                        const float p0 = a.interleaved ? x[2 * q] : x[q], p1 = a.interleaved ? x[2 * q + 1] : x[4 + q];
                        const float y0 = p0 * c - p1 * s, y1 = p1 * c + p0 * s;
                        y[2 * q] = y0;
                        y[2 * q + 1] = y1;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) x[q] = a.interleaved ? y[q] : q < 4 ? y[2 * q] : y[2 * (q - 4) + 1];
                }
                if (!there) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) x[q] = NAN;
                }
            }
            if (kind == 0) {
                const u32x4_t w = bf16x8(x);
                uint16_t *o = a.out_q + ((size_t)token * a.Hq + head) * D;
                *(u32x2_t *)(o + at.a) = u32x2_t{w[0], w[1]};
                *(u32x2_t *)(o + at.b) = u32x2_t{w[2], w[3]};
                continue;
            }
            if (!good) continue;
            const size_t slot = ((size_t)page * Hkv + head) * a.c.size + (t & (a.c.size - 1));
            if constexpr (!FP8) {
                const u32x4_t w = bf16x8(x);
                uint16_t *o = (uint16_t *)(kind == 1 ? a.c.k : a.c.v) + slot * D;
                *(u32x2_t *)(o + at.a) = u32x2_t{w[0], w[1]};
                *(u32x2_t *)(o + at.b) = u32x2_t{w[2], w[3]};
            } else {
                float m = 0.f;
                int bad = 0;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    m = fmaxf(m, fabsf(x[q]));
                    bad |= !(fabsf(x[q]) <= 3.40282347e38f);
                }
                m = row_max<LPR>(bad ? INFINITY : m);
                const bool fin = m <= 3.40282347e38f;
                const float s = fin ? fmaxf(m / kE4m3Max, kMinScale) : 1.0f;
                // x / s: the product with the reciprocal and one correction
                const float inv = 1.0f / s;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float d = x[q] * inv;
                    x[q] = fin ? fmaf(fmaf(-d, s, x[q]), inv, d) : 0.f;
                }
                uint8_t *o = (uint8_t *)(kind == 1 ? a.c.k : a.c.v) + slot * D;
                *(uint32_t *)(o + at.a) = pack_e4m3(x[0], x[1], x[2], x[3]);
                *(uint32_t *)(o + at.b) = pack_e4m3(x[4], x[5], x[6], x[7]);
                if (l == 0) (kind == 1 ? a.c.k_scale : a.c.v_scale)[slot] = fin ? s : NAN;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// spec_kv_read
// ---------------------------------------------------------------------------

struct ReadArgs {
    Pages c;
    const int32_t *start, *len;
    int L;
    void *out_k, *out_v;
    Control *ctl;
};

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        *(u32x4_t *)p = bf16x8(x);
    } else {
        *(f32x4_t *)p = f32x4_t{x[0], x[1], x[2], x[3]};
        *(f32x4_t *)(p + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
    }
}

constexpr int kReadTokens = 4;

// One workgroup per kReadTokens tokens of a request (y); a thread takes 8
// values of a head row of each, all loads before the first store.
// Bound by HBM: pages read, rows written; 32 users of 4 k tokens from e4m3
// pages take 121 us, 5.1 TB/s of 614 MB (one token a workgroup: 147 us).
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kBlock) kv_read_kernel(ReadArgs a) {
    const int r = blockIdx.y, i0 = blockIdx.x * kReadTokens;
    const int n = a.len[r], st = a.start[r];
    const bool sane = n >= 0 && n <= a.L && in_table(st, n, a.c.max_pages, a.c.shift);
    const int end = sane ? n : a.L;  // rows of this request that are written
    if (i0 >= end) return;
    const int Hkv = a.c.heads;
    int64_t slot[kReadTokens];       // of head 0; -1: a bad page or request
    bool bad = false;
#pragma unroll
    for (int q = 0; q < kReadTokens; ++q) {
        const int t = st + min(i0 + q, end - 1);
        const int page = sane ? a.c.table[(size_t)r * a.c.max_pages + (t >> a.c.shift)] : -1;
        const bool good = page >= 0 && page < a.c.num_pages;
        slot[q] = good ? (int64_t)page * Hkv * a.c.size + (t & (a.c.size - 1)) : -1;
        bad |= !good;
    }
    if (bad && threadIdx.x == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
    const int half = Hkv * (D / 8);
    for (int j = threadIdx.x; j < 2 * half; j += kBlock) {
        const bool isv = j >= half;
        const int jj = isv ? j - half : j, head = jj / (D / 8), e = (jj % (D / 8)) * 8;
        T *dst = (T *)(isv ? a.out_v : a.out_k) + (((size_t)r * a.L + i0) * Hkv + head) * D + e;
        const char *pages = (const char *)(isv ? a.c.v : a.c.k);
        const float *scales = isv ? a.c.v_scale : a.c.k_scale;
        typedef typename std::conditional<FP8, u32x2_t, u32x4_t>::type raw_t;
        raw_t w[kReadTokens];
        float s[kReadTokens];
#pragma unroll
        for (int q = 0; q < kReadTokens; ++q) {
            const int64_t at = max(slot[q], (int64_t)0) + (int64_t)head * a.c.size;  // slot 0 is there
            w[q] = *(const raw_t *)(pages + (at * D + e) * (FP8 ? 1 : 2));
            if constexpr (FP8) s[q] = scales[at];
        }
#pragma unroll
        for (int q = 0; q < kReadTokens; ++q) {
            if (i0 + q >= end) break;
            float x[8];
            if constexpr (!FP8) {
                const uint32_t b[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = bf16_lo(b[i]);
                    x[2 * i + 1] = bf16_hi(b[i]);
                }
            } else {
                const uint32_t b[4] = {e4m3_bf16<false>(w[q].x), e4m3_bf16<true>(w[q].x),
                                       e4m3_bf16<false>(w[q].y), e4m3_bf16<true>(w[q].y)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = bf16_lo(b[i]) * s[q];
                    x[2 * i + 1] = bf16_hi(b[i]) * s[q];
                }
            }
            if (slot[q] < 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = NAN;
            }
            store8(dst + (size_t)q * Hkv * D, x);
        }
    }
}

// ---------------------------------------------------------------------------
// spec_kv_commit
// ---------------------------------------------------------------------------

struct CommitArgs {
    Pages c;
    const int32_t *ctx_len, *accepted, *path;
    int M, row_bytes;            // bytes of one head row
    int32_t *out_ctx;
    Control *ctl;
};

// One workgroup per request.  Every column (16 bytes of one head row of K or
// V, or one scale) belongs to one thread, which moves its rows eight at a time
// in ascending order, reading the eight before it writes them: the path rises
// from path[i] >= i + 1 on, so a later row's source path[j] >= j + 1 lies
// behind every slot i + 1 <= j written for earlier ones.  Bound by four
// dependent memory round trips: 256 users, 5.3 us.
__global__ void __launch_bounds__(kBlock) kv_commit_kernel(CommitArgs a) {
    __shared__ int64_t from_s[SPEC_TREE_MAX_NODES], to_s[SPEC_TREE_MAX_NODES];
    const int r = blockIdx.x, tid = threadIdx.x;
    const int A = a.accepted[r], ctx = a.ctx_len[r];
    if (A == -1) {
        if (tid == 0 && a.out_ctx) a.out_ctx[r] = ctx;
        return;
    }
    const int32_t *path = a.path + (size_t)r * a.M;
    bool ok = A >= 0 && A < a.M && in_table(ctx, 1 + (A >= 0 ? A : 0), a.c.max_pages, a.c.shift);
    const int nA = ok ? A : 0;
    for (int i = tid; i < nA; i += kBlock) {
        const int u = path[i], prev = i ? path[i - 1] : 0;
        ok = ok && u > prev && u < a.M && in_table(ctx, u + 1, a.c.max_pages, a.c.shift);
        if (ok) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int t = ctx + (s ? 1 + i : u);
                const int page = a.c.table[(size_t)r * a.c.max_pages + (t >> a.c.shift)];
                ok = ok && page >= 0 && page < a.c.num_pages;
                const int64_t slot = (int64_t)page * a.c.heads * a.c.size + (t & (a.c.size - 1));
                (s ? to_s : from_s)[i] = slot;
            }
        }
    }
    ok = __syncthreads_and(ok);
    if (tid == 0) {
        if (a.out_ctx) a.out_ctx[r] = ok ? ctx + 1 + A : -1;
        if (!ok) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
    }
    if (!ok) return;
    const int cols = a.row_bytes / 16, all = 2 * a.c.heads * cols;
    for (int j = tid; j < all; j += kBlock) {
        const int head = j / cols % a.c.heads, col = j % cols;
        char *base = (char *)(j >= a.c.heads * cols ? a.c.v : a.c.k) +
                     (int64_t)head * a.c.size * a.row_bytes + col * 16;
        for (int i0 = 0; i0 < nA; i0 += 8) {
            u32x4_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < nA) w[i] = *(const u32x4_t *)(base + from_s[i0 + i] * a.row_bytes);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < nA) *(u32x4_t *)(base + to_s[i0 + i] * a.row_bytes) = w[i];
        }
    }
    if (a.c.k_scale) {
        for (int j = tid; j < 2 * a.c.heads; j += kBlock) {
            float *base = (j >= a.c.heads ? a.c.v_scale : a.c.k_scale) +
                          (int64_t)(j % a.c.heads) * a.c.size;
            for (int i0 = 0; i0 < nA; i0 += 8) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < nA) w[i] = base[from_s[i0 + i]];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < nA) base[to_s[i0 + i]] = w[i];
            }
        }
    }
}

// Few tokens: one head row a thread, so that latency is a row's (64 tokens of
// 48 rows: 4.0 us against 4.8); from two workgroups to a compute unit on, a
// workgroup per token and four rows a thread (512 tokens 5.9 us against 6.2,
// 16 k tokens 77 against 121; all of 48 rows of 128).
template <typename T, bool FP8, int D>
static void launch_write(const WriteArgs &a, int64_t tokens, int rows, hipStream_t st) {
    constexpr int RPB = kBlock / (D / 8);
    const int y = (rows + RPB - 1) / RPB;
    if (tokens < 512)
        hipLaunchKernelGGL((qkv_write_kernel<T, FP8, D, 1>), dim3((unsigned)tokens, (unsigned)y),
                           dim3(kBlock), 0, st, a);
    else
        hipLaunchKernelGGL((qkv_write_kernel<T, FP8, D, 4>), dim3((unsigned)tokens), dim3(kBlock), 0,
                           st, a);
}
template <typename T, bool FP8>
static void launch_write(const WriteArgs &a, int D, int64_t tokens, int rows, hipStream_t st) {
    if (D == 64) launch_write<T, FP8, 64>(a, tokens, rows, st);
    else if (D == 128) launch_write<T, FP8, 128>(a, tokens, rows, st);
    else launch_write<T, FP8, 256>(a, tokens, rows, st);
}

template <typename T, bool FP8>
static void launch_read(const ReadArgs &a, int D, dim3 grid, hipStream_t st) {
    if (D == 64) hipLaunchKernelGGL((kv_read_kernel<T, FP8, 64>), grid, dim3(kBlock), 0, st, a);
    else if (D == 128) hipLaunchKernelGGL((kv_read_kernel<T, FP8, 128>), grid, dim3(kBlock), 0, st, a);
    else hipLaunchKernelGGL((kv_read_kernel<T, FP8, 256>), grid, dim3(kBlock), 0, st, a);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_cache_workspace_bytes(void) { return sizeof(Control); }

int spec_qkv_write(const void *q, const void *k, const void *v, int dtype, int64_t ld_q,
                   int64_t ld_k, int64_t ld_v, const void *q_weight, const void *k_weight,
                   float eps, const float *rope, int max_pos, int rot_dim, int interleaved,
                   const int32_t *positions, const int32_t *ctx_len, const int32_t *n_nodes,
                   const int32_t *page_table, int max_pages, int R, int M, int Hq, int Hkv, int D,
                   void *k_cache, void *v_cache, int cache_dtype, float *k_scale, float *v_scale,
                   int num_pages, int page_size, void *out_q, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (R < 0 || M < 0 || Hq < 0 || rot_dim < 0 || max_pos < 0 || !(eps >= 0.0f))
        return SPEC_EINVAL;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EDTYPE;
    const int bad = check_pages(k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                                page_size, max_pages, Hkv, D);
    if (bad) return bad;
    if (rot_dim > D || rot_dim % 16) return SPEC_EUNSUPPORTED;
    if (rot_dim > 0 && max_pos < 1) return SPEC_EINVAL;
    const int64_t tokens = (int64_t)R * M;
    if (tokens > kMaxBlocks) return SPEC_EUNSUPPORTED;
    if (Hq % Hkv) return SPEC_EINVAL;
    if (tokens == 0) return SPEC_OK;  // (an empty q may well be null)
    if ((q != nullptr) != (Hq > 0)) return SPEC_EINVAL;
    if (!k || !v || !ctx_len || !n_nodes || (max_pages > 0 && !page_table) || (q && !out_q) || (rot_dim > 0) != (rope != nullptr))
        return SPEC_EINVAL;
    const int64_t per = dtype == SPEC_BF16 ? 8 : 4;  // elements of 16 bytes
    if ((q && (ld_q < (int64_t)Hq * D || ld_q % per)) || ld_k < (int64_t)Hkv * D || ld_k % per ||
        ld_v < (int64_t)Hkv * D || ld_v % per)
        return SPEC_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_weight | (uintptr_t)k_weight |
         (uintptr_t)rope | (uintptr_t)out_q) & 15u)
        return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, sizeof(Control))) return SPEC_EWORKSPACE;
    WriteArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.rope = (const float2 *)rope;
    a.max_pos = max_pos;
    a.half = rot_dim / 2;
    a.interleaved = interleaved != 0;
    a.positions = positions;
    a.ctx_len = ctx_len;
    a.n_nodes = n_nodes;
    a.c = make_pages(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, page_table,
                     max_pages, Hkv);
    a.M = M;
    a.Hq = Hq;
    a.out_q = (uint16_t *)out_q;
    a.ctl = (Control *)workspace;
    const int rpb = kBlock / (D / 8), rows = Hq + 2 * Hkv;
    if ((rows + rpb - 1) / rpb > 65535) return SPEC_EUNSUPPORTED;
    hipStream_t st = (hipStream_t)stream;
    const bool fp8 = cache_dtype == SPEC_E4M3;
    if (dtype == SPEC_BF16) {
        if (fp8) launch_write<uint16_t, true>(a, D, tokens, rows, st);
        else launch_write<uint16_t, false>(a, D, tokens, rows, st);
    } else {
        if (fp8) launch_write<float, true>(a, D, tokens, rows, st);
        else launch_write<float, false>(a, D, tokens, rows, st);
    }
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_kv_read(const void *k_cache, const void *v_cache, int cache_dtype, const float *k_scale,
                 const float *v_scale, int num_pages, int page_size, const int32_t *page_table,
                 int max_pages, const int32_t *start, const int32_t *len, int R, int max_len,
                 int Hkv, int D, void *out_k, void *out_v, int out_dtype, void *workspace,
                 size_t workspace_bytes, void *stream) {
    if (R < 0 || max_len < 0) return SPEC_EINVAL;
    const int bad = check_pages(k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                                page_size, max_pages, Hkv, D);
    if (bad) return bad;
    if (out_dtype != SPEC_BF16 && out_dtype != SPEC_F32) return SPEC_EDTYPE;
    if (R > 65535 || max_len > kReadTokens * kMaxBlocks) return SPEC_EUNSUPPORTED;
    if (R == 0 || max_len == 0) return SPEC_OK;
    if (!start || !len || !out_k || !out_v || (max_pages > 0 && !page_table)) return SPEC_EINVAL;
    if (((uintptr_t)out_k | (uintptr_t)out_v) & 15u) return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, sizeof(Control))) return SPEC_EWORKSPACE;
    ReadArgs a{};
    a.c = make_pages(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, page_table,
                     max_pages, Hkv);
    a.start = start;
    a.len = len;
    a.L = max_len;
    a.out_k = out_k;
    a.out_v = out_v;
    a.ctl = (Control *)workspace;
    const dim3 grid((unsigned)((max_len + kReadTokens - 1) / kReadTokens), (unsigned)R);
    hipStream_t st = (hipStream_t)stream;
    const bool fp8 = cache_dtype == SPEC_E4M3;
    if (out_dtype == SPEC_BF16) {
        if (fp8) launch_read<uint16_t, true>(a, D, grid, st);
        else launch_read<uint16_t, false>(a, D, grid, st);
    } else {
        if (fp8) launch_read<float, true>(a, D, grid, st);
        else launch_read<float, false>(a, D, grid, st);
    }
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_kv_commit(void *k_cache, void *v_cache, int cache_dtype, float *k_scale, float *v_scale,
                   int num_pages, int page_size, const int32_t *page_table, int max_pages,
                   const int32_t *ctx_len, const int32_t *accepted, const int32_t *path, int R,
                   int M, int Hkv, int D, int32_t *out_ctx_len, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (R < 0 || M < 1) return SPEC_EINVAL;
    const int bad = check_pages(k_cache, v_cache, cache_dtype, k_scale, v_scale, num_pages,
                                page_size, max_pages, Hkv, D);
    if (bad) return bad;
    if (M > SPEC_TREE_MAX_NODES || R > kMaxBlocks) return SPEC_EUNSUPPORTED;
    if (R == 0) return SPEC_OK;
    if (!ctx_len || !accepted || !path || (max_pages > 0 && !page_table)) return SPEC_EINVAL;
    if (out_ctx_len == ctx_len || out_ctx_len == accepted || out_ctx_len == path) return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, sizeof(Control))) return SPEC_EWORKSPACE;
    CommitArgs a{};
    a.c = make_pages(k_cache, v_cache, cache_dtype == SPEC_E4M3 ? k_scale : nullptr,
                     cache_dtype == SPEC_E4M3 ? v_scale : nullptr, num_pages, page_size,
                     page_table, max_pages, Hkv);
    a.ctx_len = ctx_len;
    a.accepted = accepted;
    a.path = path;
    a.M = M;
    a.row_bytes = D * (cache_dtype == SPEC_E4M3 ? 1 : 2);
    a.out_ctx = out_ctx_len;
    a.ctl = (Control *)workspace;
    hipLaunchKernelGGL(kv_commit_kernel, dim3((unsigned)R), dim3(kBlock), 0, (hipStream_t)stream,
                       a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
