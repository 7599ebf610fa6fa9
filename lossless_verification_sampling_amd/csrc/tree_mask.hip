// tree_mask.hip -- positions and ancestor bits of drafted trees on gfx950.
//
// Node v (parent p(v) < v) stands at position ctx + depth(v) and sees the
// nodes on its path to the root: bit u of row v is set iff u is v or one of
// its ancestors.  Indices fall strictly along the path, so one walk meets the
// row's words from the highest to the lowest and ends by itself.
#include "cache.h"

namespace sv {

constexpr int kMaskNodes = 128;  // nodes (threads) per workgroup

struct MaskArgs {
    const int32_t *parent;   // [R][M]
    const int32_t *n_nodes;  // [R]
    const int32_t *ctx_len;  // [R]
    int M, W, window;
    int32_t *pos;            // [R][M]
    uint32_t *mask;          // [R][M][W]
    Control *ctl;
};

// One workgroup takes kMaskNodes nodes of one request: the request's parents
// go to shared memory (checked on the way), each thread walks up from its
// node and collects its row in shared memory, and the rows leave in order.
// Bound by the walk's chain of shared-memory reads (one per level) for deep
// trees and by the mask's bytes for many flat ones: 256 trees of 1024 nodes
// take 11.4 us (36 MB, 3.1 TB/s), one of 9 nodes 2.0.
__global__ void __launch_bounds__(kMaskNodes) tree_mask_kernel(MaskArgs a) {
    __shared__ int16_t par[SPEC_TREE_MAX_NODES];
    __shared__ uint32_t rows[kMaskNodes * (SPEC_TREE_MAX_NODES / 32 + 1)];
    const int r = blockIdx.y, v0 = blockIdx.x * kMaskNodes, tid = threadIdx.x;
    const size_t rb = (size_t)r * a.M;
    const int n = a.n_nodes[r], ctx = a.ctx_len[r];
    bool ok = n >= 0 && n <= a.M && ctx >= 0 && ctx <= 0x7fffffff - a.M;
    const int nn = ok ? n : 0;
    for (int v = tid; v < nn; v += kMaskNodes) {
        const int p = v ? a.parent[rb + v] : -1;
        if (v) ok = ok && p >= 0 && p < v;
        par[v] = (int16_t)p;
    }
    const int ld = a.W + 1;  // padded: rows start in different banks
    for (int w = 0; w < a.W; ++w) rows[tid * ld + w] = 0u;
    ok = __syncthreads_and(ok);
    const int v = v0 + tid;
    int pos = -1;
    if (ok && v < nn) {
        int d = 0, w = v >> 5;
        uint32_t bits = 0u;
        for (int u = v; u >= 0; u = par[u], ++d) {
            if (a.window && d >= a.window) continue;
            if ((u >> 5) != w) {
                rows[tid * ld + w] = bits;
                bits = 0u;
                w = u >> 5;
            }
            bits |= 1u << (u & 31);
        }
        rows[tid * ld + w] = bits;
        pos = ctx + d - 1;
    }
    if (v < a.M) a.pos[rb + v] = pos;
    __syncthreads();
    const int cnt = min(kMaskNodes, a.M - v0) * a.W;
    uint32_t *out = a.mask + (rb + v0) * a.W;
    const int down = kMaskNodes / a.W, right = kMaskNodes - down * a.W;
    int row = tid / a.W, col = tid - row * a.W;
    for (int i = tid; i < cnt; i += kMaskNodes) {
        out[i] = rows[row * ld + col];
        row += down;
        col += right;
        if (col >= a.W) {
            col -= a.W;
            ++row;
        }
    }
    if (!ok && tid == 0) atomic_or_u32(&a.ctl->status, SPEC_DEV_BAD_REQUEST);
}

}  // namespace sv

using namespace sv;

extern "C" {

int spec_tree_mask(const int32_t *parent, const int32_t *n_nodes, const int32_t *ctx_len, int R,
                   int M, int window, int32_t *out_positions, uint32_t *out_mask, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (R < 0 || M < 1 || window < 0) return SPEC_EINVAL;
    if (M > SPEC_TREE_MAX_NODES || R > 65535) return SPEC_EUNSUPPORTED;
    if (R == 0) return SPEC_OK;
    if (!parent || !n_nodes || !ctx_len || !out_positions || !out_mask) return SPEC_EINVAL;
    if (bad_workspace(workspace, workspace_bytes, sizeof(Control))) return SPEC_EWORKSPACE;
    MaskArgs a{};
    a.parent = parent;
    a.n_nodes = n_nodes;
    a.ctx_len = ctx_len;
    a.M = M;
    a.W = (M + 31) / 32;
    a.window = window;
    a.pos = out_positions;
    a.mask = out_mask;
    a.ctl = (Control *)workspace;
    hipLaunchKernelGGL(tree_mask_kernel, dim3((M + kMaskNodes - 1) / kMaskNodes, (unsigned)R),
                       dim3(kMaskNodes), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
