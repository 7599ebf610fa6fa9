// tree_attn.hip -- attention of drafted tokens over the paged cache on gfx950.
//
// Row (v, h) of request r: s_j = scale q . k_j over the tokens j the node sees,
// o = sum_j e^{s_j} v_j / sum_j e^{s_j}, in one pass over the tokens with the
// running maximum m, sum l and product o: a token with s > m rescales l and o
// by e^{m - s}.
#include <math.h>

#include "cache.h"

namespace sv {

struct AttnArgs {
    const uint16_t *q;           // [R][M][Hq][D] bf16
    Pages c;
    const int32_t *ctx_len, *n_nodes;
    const uint32_t *mask;        // [R][M][W], null: chain
    const int32_t *positions;    // [R][M], null: ctx + v
    float scale;
    int window, M, W, Hq, G;
    uint16_t *out;
    float *lse;
    Control *ctl;
};

// One workgroup per row: wave w takes tokens w, w + 4, ..., its lanes D / 64
// values each.
template <bool FP8, int D>
__global__ void __launch_bounds__(kBlock) attn_row_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    __shared__ float wm[kWaves], wl[kWaves], wo[kWaves][D];
    const int h = blockIdx.x, v = blockIdx.y, r = blockIdx.z;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = a.n_nodes[r], ctx = a.ctx_len[r];
    bool ok = n >= 0 && n <= a.M && in_table(ctx, n, a.c.max_pages, a.c.shift);
    if (ok && v >= n) return;
    const size_t node = (size_t)r * a.M + v, row = node * a.Hq + h;
    const int pos = a.positions ? a.positions[node] : ctx + v;
    ok = ok && pos >= 0;
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int i = 0; i < E; ++i) {
        q[i] = bf16_lo(a.q[row * D + lane * E + i]);
        o[i] = 0.f;
    }
    const int g = h / a.G, L = ok ? ctx + n : 0;
    for (int t = wave; t < L; t += kWaves) {
        bool see;
        if (t < ctx) {
            see = !a.window || t > pos - a.window;
        } else {
            const int u = t - ctx;
            see = a.mask ? (a.mask[node * a.W + (u >> 5)] >> (u & 31)) & 1u
                         : u <= v && (!a.window || v - u < a.window);
        }
        if (!see) continue;
        const int page = a.c.table[(size_t)r * a.c.max_pages + (t >> a.c.shift)];
        if (page < 0 || page >= a.c.num_pages) {
            ok = false;
            break;
        }
        const size_t slot = ((size_t)page * a.c.heads + g) * a.c.size + (t & (a.c.size - 1));
        float s = 0.f, x[E];
        for (int i = 0; i < E; ++i) {
            const size_t e = slot * D + lane * E + i;
            float k;
            if constexpr (FP8) {
                k = bf16_lo(e4m3_bf16<false>(((const uint8_t *)a.c.k)[e]));
                x[i] = bf16_lo(e4m3_bf16<false>(((const uint8_t *)a.c.v)[e])) * a.c.v_scale[slot];
            } else {
                k = bf16_lo(((const uint16_t *)a.c.k)[e]);
                x[i] = bf16_lo(((const uint16_t *)a.c.v)[e]);
            }
            s = fmaf(q[i], k, s);
        }
        s = wave_sum_f(s) * a.scale;
        if constexpr (FP8) s *= a.c.k_scale[slot];
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float al = expf(m - ref), p = expf(s - ref);
        l = l * al + p;
        for (int i = 0; i < E; ++i) o[i] = o[i] * al + p * x[i];
        m = mn;
    }
    if (lane == 0) {
        wm[wave] = m;
        wl[wave] = l;
    }
    for (int i = 0; i < E; ++i) wo[wave][lane * E + i] = o[i];
    ok = __syncthreads_and(ok);
    if (!ok && threadIdx.x == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
    float M = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
    if (M == -INFINITY) M = 0.f;
    float sum = 0.f, w[kWaves];
    for (int i = 0; i < kWaves; ++i) {
        w[i] = expf(wm[i] - M);
        sum += w[i] * wl[i];
    }
    for (int e = threadIdx.x; e < D; e += kBlock) {
        float x = 0.f;
        for (int i = 0; i < kWaves; ++i) x += w[i] * wo[i][e];
        x = !ok ? NAN : sum == 0.f ? 0.f : x / sum;
        a.out[row * D + e] = (uint16_t)pack_bf16(x, 0.f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = !ok ? NAN : M + logf(sum);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_tree_attention_workspace_bytes(int R, int M, int Hq, int Hkv, int D) {
    if (R < 0 || M < 1 || M > SPEC_TREE_MAX_NODES || Hkv < 1 || Hq < 1 || Hq % Hkv ||
        Hq / Hkv > 64 || (D != 64 && D != 128 && D != 256))
        return 0;
    return sizeof(Control);
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
    a.scale = scale;
    a.window = window;
    a.M = M;
    a.W = (M + 31) / 32;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.out = (uint16_t *)out;
    a.lse = out_lse;
    a.ctl = (Control *)workspace;
    const dim3 grid((unsigned)Hq, (unsigned)M, (unsigned)R);
    hipStream_t st = (hipStream_t)stream;
    if (cache_dtype == SPEC_E4M3) {
        if (D == 64) hipLaunchKernelGGL((attn_row_kernel<true, 64>), grid, dim3(kBlock), 0, st, a);
        else if (D == 128) hipLaunchKernelGGL((attn_row_kernel<true, 128>), grid, dim3(kBlock), 0, st, a);
        else hipLaunchKernelGGL((attn_row_kernel<true, 256>), grid, dim3(kBlock), 0, st, a);
    } else {
        if (D == 64) hipLaunchKernelGGL((attn_row_kernel<false, 64>), grid, dim3(kBlock), 0, st, a);
        else if (D == 128) hipLaunchKernelGGL((attn_row_kernel<false, 128>), grid, dim3(kBlock), 0, st, a);
        else hipLaunchKernelGGL((attn_row_kernel<false, 256>), grid, dim3(kBlock), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
