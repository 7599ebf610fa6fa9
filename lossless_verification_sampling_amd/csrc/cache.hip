// cache.hip -- writing, reading and moving rows of the paged key/value cache
// on gfx950.
//
// A head row of D values belongs to D / 8 lanes, 8 values (16 bytes of bf16)
// each, so a wave holds 512 / D rows and every sum, maximum or exchange over a
// row stays inside it.
#include <math.h>

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

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        VecLoad<T, 8>::run(p, 0, x);
    } else {
        VecLoad<T, 4>::run(p, 0, x);
        VecLoad<T, 4>::run(p, 4, x + 4);
    }
}

__device__ __forceinline__ uint4 bf16x8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

// Sum and maximum over the D / 8 lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

// One workgroup per token (x) and group of 2048 / D head rows (y).
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kBlock) qkv_write_kernel(WriteArgs a) {
    constexpr int LPR = D / 8, RPB = kBlock / LPR;
    const int token = blockIdx.x, r = token / a.M, v = token - r * a.M;
    const int tid = threadIdx.x, l = tid & (LPR - 1), e = l * 8;
    const int n = a.n_nodes[r], ctx = a.ctx_len[r];
    const bool sane = n >= 0 && n <= a.M && in_table(ctx, n, a.c.max_pages, a.c.shift);
    if (sane && v >= n) return;
    const int Hkv = a.c.heads, rows = a.Hq + 2 * Hkv;
    const int row = blockIdx.y * RPB + tid / LPR;
    if (row >= rows) return;
    if (!sane) {
        if (row < a.Hq) {
            const float nan8[8] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
            *(uint4 *)(a.out_q + ((size_t)token * a.Hq + row) * D + e) = bf16x8(nan8);
        }
        if (row == 0 && l == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        return;
    }
    const int kind = row < a.Hq ? 0 : row < a.Hq + Hkv ? 1 : 2;  // q, k, v
    const int head = kind == 0 ? row : kind == 1 ? row - a.Hq : row - a.Hq - Hkv;
    const T *src = kind == 0 ? (const T *)a.q + (int64_t)token * a.ld_q
                 : kind == 1 ? (const T *)a.k + (int64_t)token * a.ld_k
                             : (const T *)a.v + (int64_t)token * a.ld_v;
    float x[8];
    load8(src + head * D + e, x);
    if (kind < 2) {
        const T *w = (const T *)(kind == 0 ? a.q_weight : a.k_weight);
        if (w) {
            float wt[8], ss = 0.f;
            load8(w + e, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            ss = row_sum<LPR>(ss);
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wt[i];
        }
        if (a.half) {
            const int pos = a.positions ? a.positions[token] : ctx + v;
            const bool there = pos >= 0 && pos < a.max_pos;
            const float2 *cs = a.rope + (size_t)(there ? pos : 0) * a.half;
            if (a.interleaved) {
                if (e < 2 * a.half) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = cs[e / 2 + i];
                        const float p = x[2 * i], q = x[2 * i + 1];
                        x[2 * i] = p * t.x - q * t.y;
                        x[2 * i + 1] = q * t.x + p * t.y;
                    }
                }
            } else {
                // the partner of lane l < half / 8 is lane l + half / 8
                const int hl = a.half / 8;
                const int lo = l < hl, in = l < 2 * hl;
                const int from = (tid & 63) + (in ? (lo ? hl : -hl) : 0);
                const int i0 = lo ? e : e - a.half;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float other = __shfl(x[i], from, 64);
                    if (in) {
                        const float2 t = cs[i0 + i];
                        x[i] = lo ? x[i] * t.x - other * t.y : x[i] * t.x + other * t.y;
                    }
                }
            }
            if (!there) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = NAN;
                if (l == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
            }
        }
    }
    if (kind == 0) {
        *(uint4 *)(a.out_q + ((size_t)token * a.Hq + head) * D + e) = bf16x8(x);
        return;
    }
    const int t = ctx + v;
    const int page = a.c.table[(size_t)r * a.c.max_pages + (t >> a.c.shift)];
    const bool good = page >= 0 && page < a.c.num_pages;
    if (!good) {
        if (l == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
        return;
    }
    const size_t slot = ((size_t)page * Hkv + head) * a.c.size + (t & (a.c.size - 1));
    if constexpr (!FP8) {
        *(uint4 *)((uint16_t *)(kind == 1 ? a.c.k : a.c.v) + slot * D + e) = bf16x8(x);
    } else {
        float m = 0.f;
        int bad = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m = fmaxf(m, fabsf(x[i]));
            bad |= !(fabsf(x[i]) <= 3.40282347e38f);
        }
        m = row_max<LPR>(bad ? INFINITY : m);
        const bool fin = m <= 3.40282347e38f;
        const float s = fin ? fmaxf(m / kE4m3Max, kMinScale) : NAN;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fin ? x[i] / s : 0.f;
        uint2 w;
        w.x = pack_e4m3(x[0], x[1], x[2], x[3]);
        w.y = pack_e4m3(x[4], x[5], x[6], x[7]);
        *(uint2 *)((uint8_t *)(kind == 1 ? a.c.k : a.c.v) + slot * D + e) = w;
        if (l == 0) (kind == 1 ? a.c.k_scale : a.c.v_scale)[slot] = s;
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
        *(uint4 *)p = bf16x8(x);
    } else {
        *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
        *(float4 *)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// One workgroup per token of a request (y); thread: 8 values of a head row.
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kBlock) kv_read_kernel(ReadArgs a) {
    const int r = blockIdx.y, i = blockIdx.x;
    const int n = a.len[r], st = a.start[r];
    const bool sane = n >= 0 && n <= a.L && in_table(st, n, a.c.max_pages, a.c.shift);
    if (sane && i >= n) return;
    int page = -1;
    const int t = st + i;
    if (sane) {
        page = a.c.table[(size_t)r * a.c.max_pages + (t >> a.c.shift)];
        if (page < 0 || page >= a.c.num_pages) page = -1;
    }
    if (page < 0 && threadIdx.x == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
    const int Hkv = a.c.heads;
    for (int j = threadIdx.x; j < 2 * Hkv * (D / 8); j += kBlock) {
        const int half = Hkv * (D / 8);
        const bool isv = j >= half;
        const int jj = isv ? j - half : j, head = jj / (D / 8), e = (jj % (D / 8)) * 8;
        T *dst = (T *)(isv ? a.out_v : a.out_k) + (((size_t)r * a.L + i) * Hkv + head) * D + e;
        float x[8] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
        if (page >= 0) {
            const size_t slot = ((size_t)page * Hkv + head) * a.c.size + (t & (a.c.size - 1));
            if constexpr (!FP8) {
                VecLoad<uint16_t, 8>::run((const uint16_t *)(isv ? a.c.v : a.c.k) + slot * D, e, x);
            } else {
                const uint2 w = *(const uint2 *)((const uint8_t *)(isv ? a.c.v : a.c.k) + slot * D + e);
                const float s = (isv ? a.c.v_scale : a.c.k_scale)[slot];
                const uint32_t b[4] = {e4m3_bf16<false>(w.x), e4m3_bf16<true>(w.x),
                                       e4m3_bf16<false>(w.y), e4m3_bf16<true>(w.y)};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[2 * q] = bf16_lo(b[q]) * s;
                    x[2 * q + 1] = bf16_hi(b[q]) * s;
                }
            }
        }
        store8(dst, x);
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
// V, or one scale) belongs to one thread, which moves its rows in ascending
// order: path[i] > i, and the path rises, so a row is read before any move
// writes to it.
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
        char *base = (char *)(j >= a.c.heads * cols ? a.c.v : a.c.k) + col * 16;
        for (int i = 0; i < nA; ++i) {
            const int64_t hs = (int64_t)head * a.c.size;
            const uint4 w = *(const uint4 *)(base + (from_s[i] + hs) * a.row_bytes);
            *(uint4 *)(base + (to_s[i] + hs) * a.row_bytes) = w;
        }
    }
    if (a.c.k_scale) {
        for (int j = tid; j < 2 * a.c.heads; j += kBlock) {
            float *base = (j >= a.c.heads ? a.c.v_scale : a.c.k_scale) +
                          (int64_t)(j % a.c.heads) * a.c.size;
            for (int i = 0; i < nA; ++i) base[to_s[i]] = base[from_s[i]];
        }
    }
}

template <typename T, bool FP8>
static void launch_write(const WriteArgs &a, int D, dim3 grid, hipStream_t st) {
    if (D == 64) hipLaunchKernelGGL((qkv_write_kernel<T, FP8, 64>), grid, dim3(kBlock), 0, st, a);
    else if (D == 128) hipLaunchKernelGGL((qkv_write_kernel<T, FP8, 128>), grid, dim3(kBlock), 0, st, a);
    else hipLaunchKernelGGL((qkv_write_kernel<T, FP8, 256>), grid, dim3(kBlock), 0, st, a);
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
                                page_size, page_table, max_pages, Hkv, D);
    if (bad) return bad;
    if (rot_dim > D || rot_dim % 16) return SPEC_EUNSUPPORTED;
    const int64_t tokens = (int64_t)R * M;
    if (tokens > 0x7fffffff) return SPEC_EUNSUPPORTED;
    if (q ? Hq < 1 || Hq % Hkv : Hq != 0) return SPEC_EINVAL;
    if (tokens == 0) return SPEC_OK;
    if (!k || !v || !ctx_len || !n_nodes || (q && !out_q) || (rot_dim > 0) != (rope != nullptr))
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
    const dim3 grid((unsigned)tokens, (unsigned)((rows + rpb - 1) / rpb));
    hipStream_t st = (hipStream_t)stream;
    const bool fp8 = cache_dtype == SPEC_E4M3;
    if (dtype == SPEC_BF16) {
        if (fp8) launch_write<uint16_t, true>(a, D, grid, st);
        else launch_write<uint16_t, false>(a, D, grid, st);
    } else {
        if (fp8) launch_write<float, true>(a, D, grid, st);
        else launch_write<float, false>(a, D, grid, st);
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
                                page_size, page_table, max_pages, Hkv, D);
    if (bad) return bad;
    if (out_dtype != SPEC_BF16 && out_dtype != SPEC_F32) return SPEC_EDTYPE;
    if (R > 65535) return SPEC_EUNSUPPORTED;
    if (R == 0 || max_len == 0) return SPEC_OK;
    if (!start || !len || !out_k || !out_v) return SPEC_EINVAL;
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
    const dim3 grid((unsigned)max_len, (unsigned)R);
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
                                page_size, page_table, max_pages, Hkv, D);
    if (bad) return bad;
    if (M > SPEC_TREE_MAX_NODES) return SPEC_EUNSUPPORTED;
    if (R == 0) return SPEC_OK;
    if (!ctx_len || !accepted || !path || out_ctx_len == ctx_len) return SPEC_EINVAL;
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
