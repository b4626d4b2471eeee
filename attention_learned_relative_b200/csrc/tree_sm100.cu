// tree_sm100.cu -- attention of drafted token trees over a paged bf16 key/value cache,
// with the learned relative-position bias: a split-KV tcgen05 kernel and a log-sum-exp
// combine.
//
// Sequence b has ctx_b prefix rows and a tree of n_b drafted nodes whose keys and values
// are cache rows ctx_b + t.  Node t sits at position ctx_b + depth_t, so with
// rel_j = j - ctx_b for a prefix row j and rel = depth_s for a node s, its distance to a
// key is depth_t - rel; it sees prefix rows, and the nodes its mask names, at distances
// 0 <= dist (< window), and its logits carry r * w[h, dist] for dist < R.
//
// Rows.  All query heads of a group read the same keys, so the (node, head) pairs of a
// key/value head are packed into 128-row tiles, row = node * G + head (nodes_per_tile =
// 128 / G nodes; TMA writes them in that order as one box of G heads by nodes_per_tile
// tokens).  A work item is (sequence, key/value head, up to two row tiles, a run of
// 128-key tiles).  Its two softmax slots take
//   two row tiles (T * G > 128): a row tile each, both on every key tile, or
//   one row tile: the even and the odd key tiles, merged at the end in tensor memory,
// so K and V of an item cross from HBM to shared memory once in either case and one
// slot's softmax always overlaps the other's products.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax and epilogue of slot 0, slot 1 (one row per thread)
//   warp 8          TMA producer: Q once, K and V per key tile (2-stage rings); a key tile is
//                   128 / box_rows boxes, each inside one page, one lane per box
//   warp 9          TMEM allocator, zeroing of dead V rows, tcgen05.mma issuer
//   warps 10-11     bias stagers: the distances a key tile meets span 128 + T - 1 values, so
//                   they copy that slice of the group's tables to shared memory tile by
//                   tile (any R, and nothing for the tiles beyond R)
// Units u = 0, 1, ... are (key tile, slot) pairs, slot = u & 1; the MMA warp issues QK(u),
// then PV(u - 1).  Products of one thread run in issue order, so QK(u) may overwrite the P
// of unit u - 2, and when S(u) is complete O of its slot holds all earlier units.
// Tensor memory: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D); P (bf16) over S.
//
// Masks.  Tiles that hold tree keys, or that reach past some row's window, are masked (and
// given their bias) by a pass over S in tensor memory before the softmax reads it: one or
// two tiles per sequence and head.  Other tiles add their bias in registers, if any key is
// nearer than R, and are never masked.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "kernels.h"
#include "ptx.cuh"

namespace relbias {

namespace {

constexpr int kTrM = 128, kTrN = 128;      // rows of a row tile, keys of a key tile
constexpr int kTrStages = 2;               // K and V ring depth
constexpr int kTrThreads = 384;
constexpr int kTrSoftmaxRegs = 216, kTrOtherRegs = 72;
constexpr float kTrGrow = 8.0f;            // log2 units: O is rescaled when a row's max grows by more
constexpr int kTrRec = 4;                  // floats of a partial record beyond its output: max, sum, pad

template <int D>
struct TreeLayout {
    static constexpr int kTile = kTrM * D * 2;
    static constexpr int kBox = kTrM * 128;               // 128 rows of 64 columns
    static constexpr int kQ = 0;                          // two row tiles
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kTrStages * kTile;
    static constexpr int kTab = kV + kTrStages * kTile;   // two slices, then two runs of key positions
    // The slots' (max, sum) exchange of one-row-tile items: over the second row tile's place.
    static constexpr int kXch = kQ + kTile;
};

struct TreeBars {
    uint64_t q_full[2];
    uint64_t k_full[kTrStages], k_empty[kTrStages], v_full[kTrStages], v_empty[kTrStages];
    uint64_t s_full[2], p_full[2], o_final[2];
    uint64_t tab_full[2], tab_empty[2];
    uint64_t xch, mma_done;
    uint32_t tmem_base;
    int abort_flag;
};

// Floats of a head's slice of the bias table: 128 + T - 1 distances, in a stride that is 4
// modulo 32, so that eight heads at one depth meet eight different banks.
__host__ __device__ constexpr int tree_tab_stride(int T) { return (kTrN + T - 1 + 31) / 32 * 32 + 4; }

int tree_smem_bytes(int d, int G, int T) {
    const int tiles = d == 64 ? TreeLayout<64>::kTab : TreeLayout<128>::kTab;
    const int need = tiles + 2 * (G * tree_tab_stride(T) + kTrN) * 4 + static_cast<int>(sizeof(TreeBars)) + 1024;
    return std::max(need, 120 * 1024);   // one CTA per SM: each allocates all of tensor memory
}

// A sequence's lengths, clamped into range, and its key tiles.
struct TreeSeq {
    int ctx, n;      // prefix rows, nodes
    int lo, end;     // cache rows some node may see: [lo, end)
    int base, nt;    // first row of the first key tile (a box boundary), number of key tiles
    bool bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeAttnParams& p, int b) {
    TreeSeq s;
    const int cap = p.max_pages * p.page_size, top = min(p.max_ctx, cap);
    s.ctx = __ldg(p.ctx_lens + b);
    s.n = __ldg(p.tree_lens + b);
    s.bad = s.ctx < 0 || s.ctx > top || s.n < 0 || s.n > p.T || s.n > cap - s.ctx;
    if (s.bad) {
        s.ctx = min(max(s.ctx, 0), top);
        s.n = min(max(s.n, 0), min(p.T, cap - s.ctx));
    }
    s.end = s.ctx + s.n;
    s.lo = p.window > 0 ? max(0, s.ctx - p.window + 1) : 0;
    s.base = s.lo / p.box_rows * p.box_rows;
    s.nt = s.n > 0 ? (s.end - s.base + kTrN - 1) / kTrN : 0;
    return s;
}

// Depth of node t, clamped into [0, T).
__device__ __forceinline__ int tree_depth(const TreeAttnParams& p, int b, int t, bool& bad) {
    const int d = __ldg(p.depth + static_cast<size_t>(b) * p.T + t);
    bad = d < 0 || d >= p.T;
    return min(max(d, 0), p.T - 1);
}

template <int D>
__device__ __forceinline__ void tree_issue_qk(bool leader, uint32_t d_tmem, uint32_t q_addr, uint32_t k_addr) {
    const uint32_t idesc = idesc_bf16_f32(kTrM, kTrN, false, false);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk & 3) * 32 + (kk >> 2) * TreeLayout<D>::kBox;
        const uint64_t a = smem_desc_sw128(q_addr + off, 16, 1024), b = smem_desc_sw128(k_addr + off, 16, 1024);
        if (leader) umma_ss(d_tmem, a, b, idesc, kk > 0 ? 1u : 0u);
    }
}

template <int D>
__device__ __forceinline__ void tree_issue_pv(bool leader, uint32_t d_tmem, uint32_t p_tmem, uint32_t v_addr,
                                              bool accumulate) {
    const uint32_t idesc = idesc_bf16_f32(kTrM, D, false, true);
#pragma unroll
    for (int kk = 0; kk < kTrN / 16; ++kk) {
        const uint64_t b = smem_desc_sw128(v_addr + kk * 16 * 128, TreeLayout<D>::kBox, 1024);
        if (leader) umma_ts(d_tmem, p_tmem + kk * 8, b, idesc, (accumulate || kk > 0) ? 1u : 0u);
    }
}

// Zero rows [first, last) of a key tile, by a warp, before the tensor cores read it.
template <int D>
__device__ __forceinline__ void tree_zero_rows(uint8_t* tile, int first, int last, int lane) {
    for (int x = lane; x < (last - first) * (D / 8); x += 32) {
        const int row = first + x / (D / 8), rem = x % (D / 8);
        *reinterpret_cast<uint4*>(tile + (rem >> 3) * TreeLayout<D>::kBox + row * 128 + (rem & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_shared();
    __syncwarp();
}

__device__ __forceinline__ bool tree_all(bool ok) { return __all_sync(0xffffffffu, ok); }

template <int D>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const TreeAttnParams p) {
    using L = TreeLayout<D>;
    // Item: row group fastest (its CTAs share K and V in L2), then key/value head, then split.
    const int b = blockIdx.y;
    const int grp = blockIdx.x % p.groups;
    const int g = blockIdx.x / p.groups % p.Hkv;
    const int split = blockIdx.x / (p.groups * p.Hkv);
    const TreeSeq q = tree_seq(p, b);
    const int npt = kTrM / p.G;                         // nodes of a row tile
    const int tile0 = split * p.tiles_per_split;
    const int ntiles = min(q.nt - tile0, p.tiles_per_split);
    if (q.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, kStatusBadLength);
    if (ntiles <= 0 || 2 * grp * npt >= q.n) return;    // nothing here (the combine skips it)
    const bool two = (2 * grp + 1) * npt < q.n;         // two row tiles, or two halves of the key tiles
    const int units = two ? 2 * ntiles : ntiles;
    const int jbase = q.base + tile0 * kTrN;
    // The first key tile of this run with a slice of the bias table: it holds a prefix key
    // nearer than R to a node of depth 0, or a tree key.  So do all later ones.
    const int first_slice = min(max(0, (q.ctx - max(p.R, 1) + 1 - jbase) / kTrN), ntiles);

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tstride = tree_tab_stride(p.T);
    float* tabs = reinterpret_cast<float*>(smem + L::kTab);
    int* kpos = reinterpret_cast<int*>(tabs + 2 * p.G * tstride);
    TreeBars* bars = reinterpret_cast<TreeBars*>(kpos + 2 * kTrN);
    volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kTrStages; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->q_full[s], 1);
            mbar_init(&bars->s_full[s], 1);
            mbar_init(&bars->p_full[s], 4);
            mbar_init(&bars->o_final[s], 1);
            mbar_init(&bars->tab_full[s], 2);
            mbar_init(&bars->tab_empty[s], two ? 8 : 4);
        }
        mbar_init(&bars->xch, 8);
        mbar_init(&bars->mma_done, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;

    if (warp >= 8) {
        regs_decrease<kTrOtherRegs>();
        if (warp == 8) {
            // ------------------------------------------------------------ TMA producer
            const bool leader = elect_one();
            const int nboxes = kTrN / p.box_rows;
            bool ok = true;
            int nk = 0, nv = 0;   // loads issued: number n goes to stage n % 2, phase n / 2
            if (leader) {
                for (int s = 0; s < (two ? 2 : 1); ++s) {
                    mbar_arrive_expect_tx(&bars->q_full[s], npt * p.G * 128 * (D / 64));
                    for (int bx = 0; bx < D / 64; ++bx)
                        tma_load_4d(smem + L::kQ + s * L::kTile + bx * L::kBox, &tm_q, &bars->q_full[s], bx * 64,
                                    g * p.G, (2 * grp + s) * npt, b);
                }
            }
            // This lane's box of key tile t: its page (-1, which reads zeros, past the
            // sequence's end or for an index outside the pool) and its row in the page.
            auto lookup = [&](int t, int& page, int& prow) {
                page = -1, prow = 0;
                const int row = jbase + t * kTrN + lane * p.box_rows;
                if (t >= ntiles || lane >= nboxes || row >= q.end) return;
                const int blk = row / p.page_size;
                prow = row - blk * p.page_size;
                page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + blk);
                if (page < 0 || page >= p.num_pages) {
                    atomicOr(&g_status, kStatusBadLength);
                    page = -1, prow = 0;
                }
            };
            int page, prow, next_page, next_row;
            lookup(0, next_page, next_row);
            for (int t = 0; t < ntiles; ++t) {
                const int st = t & 1;
                const uint32_t ph = (t >> 1) & 1;
                page = next_page, prow = next_row;
                lookup(t + 1, next_page, next_row);
                for (int kv = 0; kv < 2; ++kv) {
                    uint64_t* full = kv ? &bars->v_full[st] : &bars->k_full[st];
                    if (!(ok = tree_all(mbar_wait(kv ? &bars->v_empty[st] : &bars->k_empty[st], ph ^ 1, abort_flag))))
                        break;
                    if (leader) mbar_arrive_expect_tx(full, L::kTile);
                    __syncwarp();
                    if (lane < nboxes) {
                        uint8_t* dst = smem + (kv ? L::kV : L::kK) + st * L::kTile + lane * p.box_rows * 128;
                        for (int bx = 0; bx < D / 64; ++bx)
                            tma_load_4d(dst + bx * L::kBox, kv ? &tm_v : &tm_k, full, bx * 64, g, prow, page);
                    }
                    __syncwarp();
                    if (kv) ++nv; else ++nk;
                }
                if (!ok) break;
            }
            // Drain, also after an abort: no copy may be in flight when the CTA exits.
            mbar_drain_wait(&bars->q_full[0], 0);
            if (two) mbar_drain_wait(&bars->q_full[1], 0);
            for (int n = max(0, nk - kTrStages); n < nk; ++n) mbar_drain_wait(&bars->k_full[n & 1], (n >> 1) & 1);
            for (int n = max(0, nv - kTrStages); n < nv; ++n) mbar_drain_wait(&bars->v_full[n & 1], (n >> 1) & 1);
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA issuer
            const bool leader = elect_one();
            const uint32_t s_tm[2] = {tmem_base, tmem_base + 128}, o_tm[2] = {tmem_base + 256, tmem_base + 384};
            const uint32_t q_addr = smem_u32(smem + L::kQ), k_addr = smem_u32(smem + L::kK),
                           v_addr = smem_u32(smem + L::kV);
            bool ok = true;
            for (int u = 0; u <= units; ++u) {
                if (u < units) {
                    const int slot = u & 1, t = two ? u >> 1 : u, st = t & 1;
                    const bool opens = !two || slot == 0, closes = !two || slot == 1;
                    if (opens && !(ok = tree_all(mbar_wait(&bars->k_full[st], (t >> 1) & 1, abort_flag)))) break;
                    if (u < (two ? 2 : 1) && !(ok = tree_all(mbar_wait(&bars->q_full[slot], 0, abort_flag)))) break;
                    tc_fence_after();
                    tree_issue_qk<D>(leader, s_tm[slot], q_addr + (two ? slot * L::kTile : 0), k_addr + st * L::kTile);
                    if (leader) umma_commit(&bars->s_full[slot]);
                    if (leader && closes) umma_commit(&bars->k_empty[st]);
                }
                if (u > 0) {
                    const int x = u - 1, slot = x & 1, t = two ? x >> 1 : x, st = t & 1;
                    const bool opens = !two || slot == 0, closes = !two || slot == 1;
                    if (opens) {
                        if (!(ok = tree_all(mbar_wait(&bars->v_full[st], (t >> 1) & 1, abort_flag)))) break;
                        // Rows no node sees by position may hold anything, and a NaN times a
                        // zero weight is NaN: zero them before the first product reads them.
                        const int j0 = jbase + t * kTrN;
                        uint8_t* vt = smem + L::kV + st * L::kTile;
                        if (q.end < j0 + kTrN) tree_zero_rows<D>(vt, q.end - j0, kTrN, lane);
                        if (q.lo > j0) tree_zero_rows<D>(vt, 0, q.lo - j0, lane);
                    }
                    if (!(ok = tree_all(mbar_wait(&bars->p_full[slot], (x >> 1) & 1, abort_flag)))) break;
                    tc_fence_after();
                    tree_issue_pv<D>(leader, o_tm[slot], s_tm[slot], v_addr + st * L::kTile, x >= 2);
                    if (leader && closes) umma_commit(&bars->v_empty[st]);
                    if (leader && x + 2 >= units) umma_commit(&bars->o_final[slot]);
                }
            }
            // Drain: every product issued has finished before tensor memory is released.
            if (leader) umma_commit(&bars->mma_done);
            mbar_drain_wait(&bars->mma_done, 0);
        } else {
            // ------------------------------------------------------------ bias stagers
            const int x0 = threadIdx.x - 320;   // 0..63
            const int width = kTrN + p.T - 1;
            for (int t = first_slice; t < ntiles; ++t) {
                const int n = t - first_slice, buf = n & 1;
                if (!tree_all(mbar_wait(&bars->tab_empty[buf], ((n >> 1) & 1) ^ 1, abort_flag))) break;
                const int j0 = jbase + t * kTrN;
                // The slice starts at the nearest key's distance from depth 0 (0 with tree keys).
                const int dlo = max(q.ctx - j0 - (kTrN - 1), 0);
                float* tab = tabs + buf * p.G * tstride;
                const float* src = p.w + static_cast<size_t>(g) * p.G * p.R + dlo;
                for (int x = x0; x < width; x += 64) {
                    const bool in = dlo + x < p.R;
                    for (int h0 = 0; h0 < p.G; h0 += 8) {   // eight loads in flight
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = in && h0 + e < p.G ? __ldg(src + static_cast<size_t>(h0 + e) * p.R + x) : 0.0f;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (h0 + e < p.G) tab[(h0 + e) * tstride + x] = v[e];
                    }
                }
                if (j0 + kTrN > q.ctx) {
                    // Position of each key less ctx; dead keys are never reached.
                    for (int c = x0; c < kTrN; c += 64) {
                        const int s = j0 + c - q.ctx;
                        bool bad;
                        kpos[buf * kTrN + c] = s < 0 ? s : s < q.n ? tree_depth(p, b, s, bad) : INT_MAX / 2;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->tab_full[buf]);
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax / epilogue
        regs_increase<kTrSoftmaxRegs>();
        const int slot = threadIdx.x >> 7;
        const int ri = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>(ri & ~31) << 16;
        const uint32_t s_tm = tmem_base + lane_off + slot * 128;
        const int hh = ri % p.G, h = g * p.G + hh;
        const int node = ri / p.G;
        const int t_node = (2 * grp + (two ? slot : 0)) * npt + node;
        const bool row_ok = node < npt && t_node < q.n;
        int dep = 0;
        float rs = 0.0f, c1 = p.scale_log2;
        const int* words = p.mask;
        if (row_ok) {
            bool bad;
            dep = tree_depth(p, b, t_node, bad);
            if (bad) atomicOr(&g_status, kStatusBadTree);
            const size_t at = static_cast<size_t>(b) * p.T + t_node;
            rs = __ldg(p.r + at * p.Hq + h) * p.inv_scale;
            words = p.mask + at * p.words;
            // Context-length temperature: a row that sees n > temp_n0 keys (by position) has its
            // logits, content and bias, scaled by ln n / ln temp_n0.
            if (p.temp_n0 > 1) {
                const int seen = p.window > 0 ? min(q.ctx + dep + 1, p.window) : q.ctx + dep + 1;
                if (seen > p.temp_n0) c1 *= logf(static_cast<float>(seen)) * p.inv_log_n0;
            }
        }
        const int wlim = p.window > 0 ? p.window : INT_MAX;
        const uint64_t c1x2 = f2_pack(c1, c1);
        float m_used = -INFINITY;   // running reference max, log2 units
        uint64_t l2 = 0;            // running sum of the weights against it, in two lanes
        bool ok = true;
        int cnt = 0;
        for (int t = two ? 0 : slot; t < ntiles; t += two ? 1 : 2, ++cnt) {
            const int j0 = jbase + t * kTrN;
            const bool slice = t >= first_slice;
            const bool tree = j0 + kTrN > q.ctx;
            const bool edge = tree || q.ctx + q.n - 1 - j0 >= wlim;   // some key may be masked for some row
            const int n = t - first_slice, buf = n & 1;
            const float* tab = tabs + (buf * p.G + hh) * tstride;
            if (!(ok = tree_all(mbar_wait(&bars->s_full[slot], cnt & 1, abort_flag)))) break;
            if (slice && !(ok = tree_all(mbar_wait(&bars->tab_full[buf], (n >> 1) & 1, abort_flag)))) break;
            tc_fence_after();
            if (edge) {
                // Bias and masks of an edge tile, 32 columns at a time, back into S.
                const int dlo = max(q.ctx - j0 - (kTrN - 1), 0);
#pragma unroll 1
                for (int cc = 0; cc < kTrN; cc += 32) {
                    uint32_t vis = 0xffffffffu;   // visibility by mask of the 32 keys
                    const int s0 = j0 + cc - q.ctx;
                    if (s0 + 32 > 0) {
                        // Bits s0 .. s0 + 31 of the row's mask; keys before the tree are set.
                        const int k = s0 >> 5, sh = s0 & 31;
                        const uint32_t lo = k >= 0 && k < p.words ? __ldg(words + k) : k < 0 ? 0xffffffffu : 0u;
                        const uint32_t hi = k + 1 >= 0 && k + 1 < p.words ? __ldg(words + k + 1) : 0u;
                        vis = __funnelshift_r(lo, hi, sh);
                    }
                    uint32_t sr[32];
                    tmem_ld32(s_tm + cc, sr);
                    tmem_ld_wait_regs(sr);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = cc + e;
                        const int dist = dep - (tree ? kpos[buf * kTrN + c] : j0 + c - q.ctx);
                        const bool see = ((vis >> e) & 1u) && static_cast<unsigned>(dist) < static_cast<unsigned>(wlim);
                        float s = __uint_as_float(sr[e]);
                        if (slice) s = fmaf(rs, tab[see ? dist - dlo : 0], s);
                        sr[e] = __float_as_uint(see ? s : -INFINITY);
                    }
                    tmem_st32(s_tm + cc, sr);
                    tmem_st_wait();
                    tmem_regs_keep16(sr);
                    tmem_regs_keep16(sr + 16);
                }
            }
            uint32_t sr[kTrN];
#pragma unroll
            for (int c = 0; c < kTrN; c += 32) tmem_ld32(s_tm + c, sr + c);
            tmem_ld_wait_regs(sr);
#pragma unroll
            for (int c = 32; c < kTrN; c += 32) tmem_regs_fence(sr + c);
            float s[kTrN];
#pragma unroll
            for (int c = 0; c < kTrN; ++c) s[c] = __uint_as_float(sr[c]);
            if (slice && !edge) {
                // Key c lies dep + 127 - c entries into the slice.
                const float* run = tab + dep + (kTrN - 1);
#pragma unroll
                for (int c = 0; c < kTrN; ++c) s[c] = fmaf(rs, run[-c], s[c]);
            }
            if (slice) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->tab_empty[buf]);
            }
            float mc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) mc[e] = fmaxf(s[2 * e], s[2 * e + 1]);
#pragma unroll
            for (int c = 16; c < kTrN; c += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e) mc[e] = fmax3f(mc[e], s[c + 2 * e], s[c + 2 * e + 1]);
            const float mx =
                fmaxf(fmax3f(mc[0], mc[1], mc[2]), fmax3f(fmax3f(mc[3], mc[4], mc[5]), mc[6], mc[7])) * c1;
            if (cnt == 0) {
                m_used = mx;
            } else if (__any_sync(0xffffffffu, mx > m_used + kTrGrow)) {
                // Some row's max grew past the slack (or is its first): what has been summed
                // is scaled to the new reference.
                const float m_new = mx > m_used + kTrGrow ? mx : m_used;
                const float alpha = m_used == -INFINITY ? 0.0f : ex2_approx(m_used - m_new);
                m_used = m_new;
                l2 = f2_mul(l2, f2_pack(alpha, alpha));
                const uint32_t o_tm = tmem_base + lane_off + 256 + slot * 128;
                uint32_t ob[32];
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    tmem_ld32(o_tm + c, ob);
                    tmem_ld_wait_regs(ob);
#pragma unroll
                    for (int e = 0; e < 32; ++e) ob[e] = __float_as_uint(__uint_as_float(ob[e]) * alpha);
                    tmem_st32(o_tm + c, ob);
                    tmem_st_wait();
                    tmem_regs_keep16(ob);
                    tmem_regs_keep16(ob + 16);
                }
            }
            const float mb = m_used == -INFINITY ? 0.0f : m_used;
            const uint64_t nm2 = f2_pack(-mb, -mb);
            uint64_t acc[4] = {0, 0, 0, 0};
            uint32_t pk[kTrN / 2];
#pragma unroll
            for (int c = 0; c < kTrN; c += 2) {
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), c1x2, nm2), x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                acc[(c >> 1) & 3] = f2_add(acc[(c >> 1) & 3], f2_pack(p0, p1));
                // Weights are rounded to bf16 for the tensor cores (2^-8 of each at most, while
                // their sum stays in fp32).
                pk[c / 2] = pack_bf16x2(p0, p1);
            }
            l2 = f2_add(l2, f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])));
            tmem_st32(s_tm, pk);
            tmem_st32(s_tm + 32, pk + 32);
            tmem_st_wait();
#pragma unroll
            for (int c = 0; c < kTrN / 2; c += 16) tmem_regs_keep16(pk + c);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[slot]);
        }

        // Epilogue.  Two row tiles: each slot writes its own rows.  One: both slots hold a part
        // of every row, in the same tensor-memory lanes; they exchange their maxima and sums
        // through shared memory and write half of the columns each.
        float la, lb;
        f2_unpack(l2, la, lb);
        float l = la + lb, m = m_used;
        float a0 = 1.0f, a1 = 0.0f;   // scale of O0 and O1 (or of the slot's own O)
        if (ok && !two) {
            float* xch = reinterpret_cast<float*>(smem + L::kXch);   // [slot][row] {max, sum}
            xch[(slot * kTrM + ri) * 2] = m;
            xch[(slot * kTrM + ri) * 2 + 1] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->xch);
            ok = tree_all(mbar_wait(&bars->xch, 0, abort_flag));
            const float m_other = xch[((slot ^ 1) * kTrM + ri) * 2], l_other = xch[((slot ^ 1) * kTrM + ri) * 2 + 1];
            const float top = fmaxf(m, m_other);
            const float mine = m == -INFINITY ? 0.0f : ex2_approx(m - top);
            const float other = m_other == -INFINITY ? 0.0f : ex2_approx(m_other - top);
            l = l * mine + l_other * other;
            m = top;
            a0 = slot == 0 ? mine : other;
            a1 = slot == 0 ? other : mine;
        }
        if (ok) ok = two || ntiles > 1 ? tree_all(mbar_wait(&bars->o_final[two ? slot : 1], 0, abort_flag)) : true;
        if (ok && !two) ok = tree_all(mbar_wait(&bars->o_final[0], 0, abort_flag));
        if (ok) {
            tc_fence_after();
            const bool direct = p.nsplit == 1;
            if (direct) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                a0 *= inv;
                a1 *= inv;
            }
            const size_t row = (static_cast<size_t>(b) * p.T + t_node) * p.Hq + h;
            float* rec = p.part + (row * p.nsplit + split) * (D + kTrRec);
            const uint32_t o0 = tmem_base + lane_off + 256 + (two ? slot * 128 : 0);
            const int c_lo = two ? 0 : slot * (D / 2), c_hi = two ? D : c_lo + D / 2;
#pragma unroll 1
            for (int c = c_lo; c < c_hi; c += 32) {
                uint32_t x[32];
                float v[32];
                tmem_ld32(o0 + c, x);
                tmem_ld_wait_regs(x);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(x[e]) * a0;
                if (!two && ntiles > 1) {
                    tmem_ld32(tmem_base + lane_off + 384 + c, x);
                    tmem_ld_wait_regs(x);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(x[e]), a1, v[e]);
                }
                if (row_ok) {
                    if (direct) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            st_global_v4(p.o + row * D + c + e, pack_bf16x2(v[e], v[e + 1]),
                                         pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]),
                                         pack_bf16x2(v[e + 6], v[e + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(rec + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
            }
            if (row_ok && (two || slot == 0)) {
                if (!direct) {
                    *reinterpret_cast<float2*>(rec + D) = make_float2(m, l);
                } else if (p.lse != nullptr) {
                    p.lse[(static_cast<size_t>(b) * p.Hq + h) * p.T + t_node] =
                        l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
                }
            }
            tc_fence_before();
        }
    }

    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// One warp per (sequence, node, head): merges the partials of the splits that had keys.
template <int D>
__global__ void __launch_bounds__(128) tree_combine_kernel(const TreeAttnParams p) {
    constexpr int E = D / 32;
    const int b = blockIdx.y, x = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t = x / p.Hq, h = x - t * p.Hq;
    const TreeSeq q = tree_seq(p, b);
    if (t >= q.n) return;
    const int ns = (q.nt + p.tiles_per_split - 1) / p.tiles_per_split;
    const size_t row = (static_cast<size_t>(b) * p.T + t) * p.Hq + h;
    const float* recs = p.part + row * p.nsplit * (D + kTrRec);
    float M = -INFINITY;
    for (int s = lane; s < ns; s += 32) M = fmaxf(M, recs[s * (D + kTrRec) + D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.0f, acc[E] = {};
#pragma unroll 4
    for (int s = 0; s < ns; ++s) {
        const float* rec = recs + s * (D + kTrRec);
        const float2 ml = *reinterpret_cast<const float2*>(rec + D);
        const float a = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - M);
        l = fmaf(ml.y, a, l);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(rec + lane * E + e);
            acc[e] = fmaf(v.x, a, acc[e]);
            acc[e + 1] = fmaf(v.y, a, acc[e + 1]);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t out[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = out[e];
    if (p.lse != nullptr && lane == 0)
        p.lse[(static_cast<size_t>(b) * p.Hq + h) * p.T + t] = l > 0.0f ? (M + log2f(l)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeAttnParams& p,
                        cudaStream_t stream) {
    const int smem = tree_smem_bytes(D, p.G, p.T);
    cudaError_t e =
        cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    tree_attn_kernel<D><<<dim3(p.groups * p.Hkv * p.nsplit, p.B), kTrThreads, smem, stream>>>(tq, tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.nsplit == 1) return e;
    tree_combine_kernel<D><<<dim3((p.T * p.Hq + 3) / 4, p.B), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Key tiles of the longest sequence: a first tile may start up to a box before its first key.
int tree_max_tiles(int T, int max_ctx, int window, int box_rows) {
    const int rows = window > 0 ? std::min(max_ctx, window - 1) : max_ctx;
    return (rows + T + (window > 0 && max_ctx >= window ? box_rows - 1 : 0) + kTrN - 1) / kTrN;
}

// Number of splits of the key tiles.  The CTAs run in waves of one per SM, each for its share
// of the tiles and a fixed part (set-up, first loads, epilogue, combine) worth about three
// tiles; the count with the least time for full-length sequences is taken.
int tree_num_splits(int items, int tiles, int sms) {
    int best = 1;
    long long best_cost = LLONG_MAX;
    for (int ns = 1; ns <= std::min(tiles, 256); ++ns) {
        const long long waves = (static_cast<long long>(items) * ns + sms - 1) / sms;
        const int per = (tiles + ns - 1) / ns;
        const long long cost = waves * (per + 3);
        if (cost < best_cost) best = ns, best_cost = cost;
    }
    return best;
}

size_t tree_workspace_bytes(int B, int T, int Hq, int d, int nsplit) {
    return nsplit == 1 ? 16 : static_cast<size_t>(B) * T * Hq * nsplit * (d + kTrRec) * sizeof(float);
}

cudaError_t launch_tree_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const TreeAttnParams& p, int d, cudaStream_t stream) {
    return d == 128 ? launch_tree<128>(tq, tk, tv, p, stream) : launch_tree<64>(tq, tk, tv, p, stream);
}

}  // namespace relbias
