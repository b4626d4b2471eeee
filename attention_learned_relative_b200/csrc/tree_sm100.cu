// tree_sm100.cu -- attention of drafted token trees over a paged bf16 key/value cache,
// with the learned relative-position bias.
//
// Sequence b has ctx_b prefix rows and a tree of n_b drafted nodes whose keys and values
// are cache rows ctx_b + t.  Node t sits at position ctx_b + depth_t, so with
// rel_j = j - ctx_b for a prefix row j and rel = depth_s for a node s, its distance to a
// key is depth_t - rel; it sees prefix rows, and the nodes its mask names, at distances
// 0 <= dist (< window), and its logits carry r * w[h, dist] for dist < R.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace relbias {

namespace {

constexpr int kTreeWarps = 4;

// One block per (head, node, sequence); its warps take keys in turn, a key's d elements
// spread over a warp's lanes, each warp with its own running max, sum and output.
template <int D>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_attn_kernel(const TreeAttnParams p) {
    constexpr int E = D / 32;
    __shared__ float sm[kTreeWarps], sl[kTreeWarps], so[kTreeWarps][D];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = p.max_pages * p.page_size;
    int ctx = __ldg(p.ctx_lens + b), n = __ldg(p.tree_lens + b);
    if (ctx < 0 || ctx > min(p.max_ctx, cap) || n < 0 || n > p.T || n > cap - ctx) {
        atomicOr(&g_status, kStatusBadLength);
        ctx = min(max(ctx, 0), min(p.max_ctx, cap));
        n = min(max(n, 0), min(p.T, cap - ctx));
    }
    if (t >= n) return;
    const size_t node = static_cast<size_t>(b) * p.T + t;
    int dep = __ldg(p.depth + node);
    if (dep < 0 || dep >= p.T) {
        atomicOr(&g_status, kStatusBadTree);
        dep = min(max(dep, 0), p.T - 1);
    }
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[(node * p.Hq + h) * D + lane * E + e]);
        acc[e] = 0.0f;
    }
    const float rs = __ldg(p.r + node * p.Hq + h) * p.inv_scale;
    float c1 = p.scale_log2;
    const int pos = ctx + dep;
    const int seen = p.window > 0 ? min(pos + 1, p.window) : pos + 1;
    if (p.temp_n0 > 1 && seen > p.temp_n0) c1 *= logf(static_cast<float>(seen)) * p.inv_log_n0;
    float m = -INFINITY, l = 0.0f;
    const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    for (int j = first + warp; j < ctx + n; j += kTreeWarps) {
        int dist = pos - j;
        if (j >= ctx) {
            const int s = j - ctx;
            if (!((__ldg(p.mask + node * p.words + (s >> 5)) >> (s & 31)) & 1)) continue;
            dist = dep - min(max(__ldg(p.depth + static_cast<size_t>(b) * p.T + s), 0), p.T - 1);
        }
        if (dist < 0 || (p.window > 0 && dist >= p.window)) continue;
        const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + j / p.page_size);
        const bool ok = page >= 0 && page < p.num_pages;
        if (!ok) atomicOr(&g_status, kStatusBadLength);
        const size_t row = ((static_cast<size_t>(ok ? page : 0) * p.page_size + j % p.page_size) * p.Hkv + h / p.G) * D;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], ok ? __bfloat162float(p.k_pages[row + lane * E + e]) : 0.0f, s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (dist < p.R) s = fmaf(rs, __ldg(p.w + static_cast<size_t>(h) * p.R + dist), s);
        s *= c1;
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.0f : exp2f(m - mn), pr = s == -INFINITY ? 0.0f : exp2f(s - mn);
        l = fmaf(l, a, pr);
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = fmaf(acc[e], a, pr * (ok ? __bfloat162float(p.v_pages[row + lane * E + e]) : 0.0f));
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    __syncthreads();
    float M = -INFINITY, L = 0.0f;
    for (int x = 0; x < kTreeWarps; ++x) M = fmaxf(M, sm[x]);
    for (int x = 0; x < kTreeWarps; ++x) L += sm[x] == -INFINITY ? 0.0f : sl[x] * exp2f(sm[x] - M);
    if (threadIdx.x < D) {
        float v = 0.0f;
        for (int x = 0; x < kTreeWarps; ++x) v += sm[x] == -INFINITY ? 0.0f : so[x][threadIdx.x] * exp2f(sm[x] - M);
        p.o[(node * p.Hq + h) * D + threadIdx.x] = __float2bfloat16(L > 0.0f ? v / L : 0.0f);
    }
    if (p.lse != nullptr && threadIdx.x == 0)
        p.lse[(static_cast<size_t>(b) * p.Hq + h) * p.T + t] = L > 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_tree_attn(const TreeAttnParams& p, int d, cudaStream_t stream) {
    const dim3 grid(p.Hq, p.T, p.B);
    if (d == 128)
        tree_attn_kernel<128><<<grid, kTreeWarps * 32, 0, stream>>>(p);
    else
        tree_attn_kernel<64><<<grid, kTreeWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace relbias
