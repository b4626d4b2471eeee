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
// tokens).  A CTA works on a pair of row tiles.  Its two softmax slots take
//   two row tiles (more than 128 rows left): a row tile each, both on every key tile, or
//   one row tile: the even and the odd key tiles, merged at the end in tensor memory,
// so K and V cross from HBM to shared memory once per pair in either case and one slot's
// softmax always overlaps the other's products.
//
// Schedule.  Sequence lengths are known on the device only, and a batch is ragged.  The
// key tiles of all (sequence, key/value head) segments form one stream, and each CTA takes
// an equal run of it: every CTA works for the same time whatever the lengths, in one wave.
// A run covers the end of one segment, whole segments, and the start of another; whole
// segments are written out directly, the two cut ones as partials (unnormalised output,
// max, sum) that the combine kernel merges.  CTAs of different row pairs run the same
// stream side by side, so a K/V tile comes from HBM once and from L2 for the others.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax and epilogue of slot 0, slot 1 (one row per thread)
//   warp 8          TMA producer: Q per segment, K and V per key tile (2-stage rings); a key
//                   tile is 128 / box_rows boxes, each inside one page, one lane per box
//   warp 9          TMEM allocator, zeroing of dead V rows, tcgen05.mma issuer
//   warps 10-11     bias stagers: the distances a key tile meets span 128 + T - 1 values, so
//                   they copy that slice of the group's tables to shared memory tile by
//                   tile (any R, and nothing for the tiles beyond R)
// Units are (key tile, slot) pairs, alternating between the slots through all segments of
// the run; the MMA warp issues QK(u), then PV(u - 1).  Products of one thread run in issue
// order, so QK(u) may overwrite the P of unit u - 2, and when S(u) is complete O of its slot
// holds all earlier units.
// Tensor memory: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D); P (bf16) over S.
//
// Masks.  Tiles that hold tree keys, or that reach past some row's window, are masked (and
// given their bias) by a pass over S in tensor memory before the softmax reads it: one or
// two tiles per segment.  Other tiles add their bias in registers, if any key is nearer
// than R, and are never masked.
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
constexpr int kTrMinTiles = 1;             // least key tiles of a CTA's run
constexpr int kTrRec = 4;                  // floats of a partial record beyond its output: max, sum, pad

template <int D>
struct TreeLayout {
    static constexpr int kTile = kTrM * D * 2;
    static constexpr int kBox = kTrM * 128;               // 128 rows of 64 columns
    static constexpr int kQ = 0;                          // two row tiles
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kTrStages * kTile;
    // Then the slots' (max, sum) exchange of one-row-tile segments, [parity][slot][row], the
    // bars, one or two runs of key positions, and as many slices of the bias table.
    static constexpr int kXch = kV + kTrStages * kTile;
    static constexpr int kBars = kXch + 2 * 2 * kTrM * 8;
};

struct TreeBars {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kTrStages], k_empty[kTrStages], v_full[kTrStages], v_empty[kTrStages];
    uint64_t s_full[2], p_full[2], o_final[2], o_free;
    uint64_t tab_full[2], tab_empty[2];
    uint64_t xch, mma_done;
    long long part[kTrThreads / 32];   // scratch of the schedule's scan
    long long start_prefix;            // where this CTA's run starts: tiles before its first sequence,
    int start_seq;                     // and that sequence
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kTrBarBytes = (static_cast<int>(sizeof(TreeBars)) + 15) / 16 * 16;

// Floats of a head's slice of the bias table: 128 + T - 1 distances, in a stride that is 4
// modulo 32, so that eight heads at one depth meet eight different banks.
__host__ __device__ constexpr int tree_tab_stride(int T) { return (kTrN + T - 1 + 31) / 32 * 32 + 4; }

int tree_smem_need(int d, int G, int T, int bufs) {
    const int bars = d == 64 ? TreeLayout<64>::kBars : TreeLayout<128>::kBars;
    return bars + kTrBarBytes + bufs * (G * tree_tab_stride(T) + kTrN) * 4 + 1024;
}
// Slices are double-buffered where they fit (all but the largest groups and trees at d 128).
int tree_tab_bufs(int d, int G, int T) { return tree_smem_need(d, G, T, 2) <= 232448 ? 2 : 1; }
int tree_smem_bytes(int d, int G, int T) {
    // One CTA per SM: each allocates all of tensor memory.
    return std::max(tree_smem_need(d, G, T, tree_tab_bufs(d, G, T)), 120 * 1024);
}

// A sequence's lengths, clamped into range, and its key tiles.
struct TreeSeq {
    int ctx, n;      // prefix rows, nodes
    int lo, end;     // cache rows some node may see: [lo, end)
    int base, nt;    // first row of the first key tile (a box boundary), number of key tiles
    bool bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeAttnParams& p, int ctx, int n) {
    TreeSeq s;
    const int cap = p.max_pages * p.page_size, top = min(p.max_ctx, cap);
    s.ctx = ctx;
    s.n = n;
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

// A CTA's part of one (sequence, key/value head) segment.
struct TreeSeg {
    int b, g;
    TreeSeq q;
    int tile0, ntiles;   // its key tiles
    int jbase;           // first row of the first one
    int first_slice;     // first tile with a slice of the bias table; all later ones have one
    bool two;            // two row tiles, or one whose key tiles the slots share
};

// Walks the segments of a CTA's run [pos, stop) of its row pair's tile stream.  Every role
// has its own copy.  The next sequence's lengths are loaded one sequence ahead.
struct TreeWalk {
    long long pos, stop;
    int b, g, off;           // current sequence, its next key/value head, next tile in that segment
    TreeSeq q;
    int next_ctx, next_n;

    __device__ __forceinline__ void fetch(const TreeAttnParams& p) {
        const int x = min(b + 1, p.B - 1);
        next_ctx = __ldg(p.ctx_lens + x);
        next_n = __ldg(p.tree_lens + x);
    }
    __device__ __forceinline__ void start(const TreeAttnParams& p, int seq, long long prefix, long long at,
                                          long long end) {
        pos = at, stop = end, b = seq;
        q = tree_seq(p, __ldg(p.ctx_lens + b), __ldg(p.tree_lens + b));
        fetch(p);
        const long long rest = at - prefix;
        g = static_cast<int>(rest / q.nt);
        off = static_cast<int>(rest - static_cast<long long>(g) * q.nt);
    }
    __device__ __forceinline__ bool next(const TreeAttnParams& p, int grp, int npt, TreeSeg& s) {
        if (pos >= stop) return false;
        while (g == p.Hkv || 2 * grp * npt >= q.n) {   // the next sequence with rows of this pair
            ++b;
            g = 0;
            q = tree_seq(p, next_ctx, next_n);
            fetch(p);
        }
        s.b = b, s.g = g, s.q = q;
        s.tile0 = off;
        s.ntiles = static_cast<int>(min(static_cast<long long>(q.nt - off), stop - pos));
        s.jbase = q.base + off * kTrN;
        s.two = (2 * grp + 1) * npt < q.n;
        // A tile has a slice if it holds a prefix key nearer than R to a node of depth 0, or a
        // tree key.
        s.first_slice = min(max(0, (q.ctx - max(p.R, 1) + 1 - s.jbase) / kTrN), s.ntiles);
        pos += s.ntiles;
        off = 0;
        ++g;
        return true;
    }
};

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

// A softmax thread's row of a segment.
struct TreeRow {
    bool ok;
    int t, dep;
    float r;
    uint32_t words[kMaxTree / 32];
};

__device__ __forceinline__ TreeRow tree_row(const TreeAttnParams& p, const TreeSeg& s, int tile, int ri, int npt) {
    TreeRow x;
    const int node = ri / p.G, h = s.g * p.G + ri - node * p.G;
    x.t = tile * npt + node;
    x.ok = node < npt && x.t < s.q.n;
    const size_t at = static_cast<size_t>(s.b) * p.T + (x.ok ? x.t : 0);
    x.r = x.ok ? __ldg(p.r + at * p.Hq + h) : 0.0f;
    bool bad;
    x.dep = tree_depth(p, s.b, x.ok ? x.t : 0, bad);
    if (x.ok && bad) atomicOr(&g_status, kStatusBadTree);
#pragma unroll
    for (int k = 0; k < kMaxTree / 32; ++k) x.words[k] = k < p.words ? __ldg(p.mask + at * p.words + k) : 0u;
    return x;
}

// Word k of a row's mask; words before the tree are set, words after it clear.
__device__ __forceinline__ uint32_t tree_word(const TreeRow& x, int k) {
    uint32_t w = k < 0 ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < kMaxTree / 32; ++i) w = k == i ? x.words[i] : w;
    return w;
}

template <int D>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const TreeAttnParams p) {
    using L = TreeLayout<D>;
    const int npt = kTrM / p.G;                         // nodes of a row tile
    const int grp = blockIdx.x % p.groups;              // this CTA's pair of row tiles
    const int run = blockIdx.x / p.groups;              // its run of that pair's tile stream
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TreeBars* bars = reinterpret_cast<TreeBars*>(smem + L::kBars);
    int* kpos = reinterpret_cast<int*>(smem + L::kBars + kTrBarBytes);
    float* tabs = reinterpret_cast<float*>(kpos + p.tab_bufs * kTrN);
    const int tstride = tree_tab_stride(p.T);
    volatile int* abort_flag = &bars->abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->q_full[s], 1);
            mbar_init(&bars->q_empty[s], 1);
            mbar_init(&bars->s_full[s], 1);
            mbar_init(&bars->p_full[s], 4);
            mbar_init(&bars->o_final[s], 1);
            mbar_init(&bars->tab_full[s], 2);
            mbar_init(&bars->tab_empty[s], 8);
        }
        for (int s = 0; s < kTrStages; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 1);
        }
        mbar_init(&bars->o_free, 8);
        mbar_init(&bars->xch, 8);
        mbar_init(&bars->mma_done, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }

    // The stream: total tiles of this row pair's segments, and where this CTA's run starts.
    auto tiles_of = [&](int x) -> long long {
        const TreeSeq q = tree_seq(p, __ldg(p.ctx_lens + x), __ldg(p.tree_lens + x));
        if (q.bad && blockIdx.x == 0) atomicOr(&g_status, kStatusBadLength);
        return 2 * grp * npt < q.n ? static_cast<long long>(q.nt) * p.Hkv : 0;
    };
    long long mine = 0;   // of this thread's sequence in the first chunk of the scan
    long long total = 0;
    for (int x = threadIdx.x; x < p.B; x += kTrThreads) {
        const long long t = tiles_of(x);
        if (x < kTrThreads) mine = t;
        total += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) bars->part[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int x = 0; x < kTrThreads / 32; ++x) total += bars->part[x];
    const long long per = max((total + p.runs - 1) / p.runs, static_cast<long long>(kTrMinTiles));
    const long long pos = run * per, stop = min(total, pos + per);
    if (pos >= stop) {   // nothing here
        if (threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    long long prefix = 0;
    for (int x0 = 0; x0 < p.B; x0 += kTrThreads) {
        if (x0 > 0) mine = x0 + static_cast<int>(threadIdx.x) < p.B ? tiles_of(x0 + threadIdx.x) : 0;
        long long scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += up;
        }
        __syncthreads();   // the sums of the round before have been read
        if (lane == 31) bars->part[warp] = scan;
        __syncthreads();
        long long before = prefix;
        for (int x = 0; x < kTrThreads / 32; ++x) {
            if (x < warp) before += bars->part[x];
            prefix += bars->part[x];
        }
        before += scan - mine;
        if (before <= pos && pos < before + mine) {
            bars->start_seq = x0 + threadIdx.x;
            bars->start_prefix = before;
        }
        if (prefix > pos) break;   // the same in every thread
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    TreeWalk walk;
    walk.start(p, bars->start_seq, bars->start_prefix, pos, stop);
    TreeSeg s;

    if (warp >= 8) {
        regs_decrease<kTrOtherRegs>();
        if (warp == 8) {
            // ------------------------------------------------------------ TMA producer
            const bool leader = elect_one();
            const int nboxes = kTrN / p.box_rows;
            bool ok = true;
            int nkv = 0, nk = 0, nv = 0;   // key tiles; loads issued: number n goes to stage n % 2, phase n / 2
            int nq[2] = {0, 0};            // loads of each Q buffer
            for (int seg = 0; ok && walk.next(p, grp, npt, s); ++seg) {
                // This lane's box of key tile t: its page (-1, which reads zeros, past the
                // sequence's end or for an index outside the pool) and its row in the page.
                auto lookup = [&](int t, int& page, int& prow) {
                    page = -1, prow = 0;
                    const int row = s.jbase + t * kTrN + lane * p.box_rows;
                    if (t >= s.ntiles || lane >= nboxes || row >= s.q.end) return;
                    const int blk = row / p.page_size;
                    prow = row - blk * p.page_size;
                    page = __ldg(p.block_table + static_cast<size_t>(s.b) * p.max_pages + blk);
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(&g_status, kStatusBadLength);
                        page = -1, prow = 0;
                    }
                };
                int page, prow, next_page, next_row;
                lookup(0, next_page, next_row);
                // Two row tiles go to buffers 0 and 1; single ones alternate, so that a segment's
                // queries arrive while the one before is still being read.
                for (int r = 0; r < (s.two ? 2 : 1); ++r) {
                    const int buf = s.two ? r : seg & 1;
                    if (!(ok = tree_all(mbar_wait(&bars->q_empty[buf], (nq[buf] & 1) ^ 1, abort_flag)))) break;
                    if (leader) {
                        mbar_arrive_expect_tx(&bars->q_full[buf], npt * p.G * 128 * (D / 64));
                        for (int bx = 0; bx < D / 64; ++bx)
                            tma_load_4d(smem + L::kQ + buf * L::kTile + bx * L::kBox, &tm_q, &bars->q_full[buf],
                                        bx * 64, s.g * p.G, (2 * grp + r) * npt, s.b);
                    }
                    ++nq[buf];
                }
                for (int t = 0; ok && t < s.ntiles; ++t, ++nkv) {
                    const int st = nkv & 1;
                    const uint32_t ph = (nkv >> 1) & 1;
                    page = next_page, prow = next_row;
                    lookup(t + 1, next_page, next_row);
                    for (int kv = 0; kv < 2; ++kv) {
                        uint64_t* full = kv ? &bars->v_full[st] : &bars->k_full[st];
                        if (!(ok = tree_all(
                                  mbar_wait(kv ? &bars->v_empty[st] : &bars->k_empty[st], ph ^ 1, abort_flag))))
                            break;
                        if (leader) mbar_arrive_expect_tx(full, L::kTile);
                        __syncwarp();
                        if (lane < nboxes) {
                            uint8_t* dst = smem + (kv ? L::kV : L::kK) + st * L::kTile + lane * p.box_rows * 128;
                            for (int bx = 0; bx < D / 64; ++bx)
                                tma_load_4d(dst + bx * L::kBox, kv ? &tm_v : &tm_k, full, bx * 64, s.g, prow, page);
                        }
                        __syncwarp();
                        if (kv) ++nv; else ++nk;
                    }
                }
            }
            // Drain, also after an abort: no copy may be in flight when the CTA exits.
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0) mbar_drain_wait(&bars->q_full[x], (nq[x] - 1) & 1);
            for (int n = max(0, nk - kTrStages); n < nk; ++n) mbar_drain_wait(&bars->k_full[n & 1], (n >> 1) & 1);
            for (int n = max(0, nv - kTrStages); n < nv; ++n) mbar_drain_wait(&bars->v_full[n & 1], (n >> 1) & 1);
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA issuer
            const bool leader = elect_one();
            const uint32_t q_addr = smem_u32(smem + L::kQ), k_addr = smem_u32(smem + L::kK),
                           v_addr = smem_u32(smem + L::kV);
            bool ok = true;
            int nq[2] = {0, 0}, np[2] = {0, 0};   // uses of the Q buffers; P tiles taken from each slot
            int nkv = 0, parity = 0;              // key tiles and units of earlier segments (units modulo 2)
            // The unit whose PV is still to be issued.
            struct {
                bool any, opens, closes, first, accumulate, last;
                int slot, tile, lo, end, j0;
            } pv{};
            // PV of the pending unit; the next unit's QK has been issued.
            auto issue_pv = [&](int seg) -> bool {
                const int st = pv.tile & 1;
                if (pv.opens) {
                    if (!tree_all(mbar_wait(&bars->v_full[st], (pv.tile >> 1) & 1, abort_flag))) return false;
                    // Rows no node sees by position may hold anything, and a NaN times a zero
                    // weight is NaN: zero them before the first product reads them.
                    uint8_t* vt = smem + L::kV + st * L::kTile;
                    if (pv.end < pv.j0 + kTrN) tree_zero_rows<D>(vt, pv.end - pv.j0, kTrN, lane);
                    if (pv.lo > pv.j0) tree_zero_rows<D>(vt, 0, pv.lo - pv.j0, lane);
                }
                if (!tree_all(mbar_wait(&bars->p_full[pv.slot], np[pv.slot] & 1, abort_flag))) return false;
                ++np[pv.slot];
                // A segment's first product overwrites O: all epilogues of the one before are done.
                if (pv.first && seg > 0 && !tree_all(mbar_wait(&bars->o_free, (seg - 1) & 1, abort_flag))) return false;
                tc_fence_after();
                tree_issue_pv<D>(leader, tmem_base + 256 + pv.slot * 128, tmem_base + pv.slot * 128,
                                 v_addr + st * L::kTile, pv.accumulate);
                if (leader && pv.closes) umma_commit(&bars->v_empty[st]);
                if (leader && pv.last) umma_commit(&bars->o_final[pv.slot]);
                return true;
            };
            int seg = 0;
            for (; ok && walk.next(p, grp, npt, s); ++seg) {
                const int units = s.two ? 2 * s.ntiles : s.ntiles;
                for (int u = 0; ok && u < units; ++u) {
                    const int ls = u & 1, slot = ls ^ parity, t = nkv + (s.two ? u >> 1 : u), st = t & 1;
                    const int buf = s.two ? ls : seg & 1;
                    const bool opens = !s.two || ls == 0, closes = !s.two || ls == 1;
                    if (opens && !(ok = tree_all(mbar_wait(&bars->k_full[st], (t >> 1) & 1, abort_flag)))) break;
                    if (u < (s.two ? 2 : 1) && !(ok = tree_all(mbar_wait(&bars->q_full[buf], nq[buf]++ & 1, abort_flag))))
                        break;
                    tc_fence_after();
                    tree_issue_qk<D>(leader, tmem_base + slot * 128, q_addr + buf * L::kTile, k_addr + st * L::kTile);
                    if (leader) umma_commit(&bars->s_full[slot]);
                    if (leader && closes) umma_commit(&bars->k_empty[st]);
                    if (leader && u + (s.two ? 2 : 1) >= units) umma_commit(&bars->q_empty[buf]);
                    if (pv.any && !(ok = issue_pv(pv.first && u == 0 ? seg - 1 : pv.first ? seg : 0))) break;
                    pv = {true, opens, closes, u == 0, u >= 2, u + 2 >= units, slot, t,
                          s.q.lo, s.q.end, s.jbase + (t - nkv) * kTrN};
                }
                nkv += s.ntiles;
                parity ^= units & 1;
            }
            if (ok && pv.any) issue_pv(seg - 1);
            // Drain: every product issued has finished before tensor memory is released.
            if (leader) umma_commit(&bars->mma_done);
            mbar_drain_wait(&bars->mma_done, 0);
        } else {
            // ------------------------------------------------------------ bias stagers
            const int x0 = threadIdx.x - 320;   // 0..63
            const int width = kTrN + p.T - 1;
            int n = 0, cut = 0, cut_b = 0, cut_g = 0;
            bool ok = true;
            while (ok && walk.next(p, grp, npt, s)) {
                const int after = s.q.nt - s.tile0 - s.ntiles;
                if (s.tile0 == 0 && after > 0) {
                    // The segment starts here and goes on in the next runs.
                    cut = 1 + static_cast<int>((after + per - 1) / per);
                    cut_b = s.b, cut_g = s.g;
                }
                for (int t = s.first_slice; t < s.ntiles; ++t, ++n) {
                    const int buf = p.tab_bufs == 2 ? n & 1 : 0, use = p.tab_bufs == 2 ? n >> 1 : n;
                    if (!(ok = tree_all(mbar_wait(&bars->tab_empty[buf], (use & 1) ^ 1, abort_flag)))) break;
                    const int j0 = s.jbase + t * kTrN;
                    // The slice starts at the nearest key's distance from depth 0 (0 with tree keys).
                    const int dlo = max(s.q.ctx - j0 - (kTrN - 1), 0);
                    if (j0 + kTrN > s.q.ctx) {
                        // Position of each key less ctx; dead keys lie far ahead of every node.
                        for (int c = x0; c < kTrN; c += 64) {
                            const int x = j0 + c - s.q.ctx;
                            bool bad;
                            kpos[buf * kTrN + c] = x < 0 ? x : x < s.q.n ? tree_depth(p, s.b, x, bad) : INT_MAX / 2;
                        }
                    }
                    float* tab = tabs + buf * p.G * tstride;
                    const float* src = p.w + static_cast<size_t>(s.g) * p.G * p.R + dlo;
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
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->tab_full[buf]);
                }
            }
            if (x0 == 0) p.cuts[blockIdx.x] = make_int4(cut, cut_b, cut_g, 0);
        }
    } else {
        // ---------------------------------------------------------------- softmax / epilogue
        regs_increase<kTrSoftmaxRegs>();
        const int slot = threadIdx.x >> 7;
        const int ri = threadIdx.x & 127;
        const uint32_t lane_off = static_cast<uint32_t>(ri & ~31) << 16;
        const uint32_t s_tm = tmem_base + lane_off + slot * 128;
        const int hh = ri % p.G;
        const int wlim = p.window > 0 ? p.window : INT_MAX;
        bool ok = true;
        int ns = 0, nslice = 0, parity = 0;    // S tiles of this slot; slices, and units (modulo 2), of earlier segments
        int nf[2] = {0, 0}, nx = 0;            // finals of each slot; exchanges
        bool more = walk.next(p, grp, npt, s);
        TreeRow row = tree_row(p, s, 2 * grp + (s.two ? slot : 0), ri, npt);
        while (ok && more) {
            const int ls = slot ^ parity;      // this slot's part: its row tile, or its half of the key tiles
            const int h = s.g * p.G + hh;
            const float rs = row.r * p.inv_scale;
            float c1 = p.scale_log2;
            // Context-length temperature: a row that sees n > temp_n0 keys (by position) has its
            // logits, content and bias, scaled by ln n / ln temp_n0.
            if (p.temp_n0 > 1) {
                const int seen = min(s.q.ctx + row.dep + 1, wlim);
                if (seen > p.temp_n0) c1 *= logf(static_cast<float>(seen)) * p.inv_log_n0;
            }
            const uint64_t c1x2 = f2_pack(c1, c1);
            float m_used = -INFINITY;   // running reference max, log2 units
            uint64_t l2 = 0;            // running sum of the weights against it, in two lanes
            const int t_first = s.two ? 0 : ls, t_step = s.two ? 1 : 2;
            for (int t = t_first; t < s.ntiles; t += t_step, ++ns) {
                const int j0 = s.jbase + t * kTrN;
                const bool slice = t >= s.first_slice;
                const bool tree = j0 + kTrN > s.q.ctx;
                // Some key may be masked for some row.
                const bool edge = tree || s.q.ctx + s.q.n - 1 - j0 >= wlim;
                const int n = nslice + t - s.first_slice;
                const int buf = p.tab_bufs == 2 ? n & 1 : 0, use = p.tab_bufs == 2 ? n >> 1 : n;
                const float* tab = tabs + (buf * p.G + hh) * tstride;
                if (!(ok = tree_all(mbar_wait(&bars->s_full[slot], ns & 1, abort_flag)))) break;
                if (slice && !(ok = tree_all(mbar_wait(&bars->tab_full[buf], use & 1, abort_flag)))) break;
                tc_fence_after();
                if (edge) {
                    // Bias and masks of an edge tile, 32 columns at a time, back into S.
                    const int dlo = max(s.q.ctx - j0 - (kTrN - 1), 0);
#pragma unroll 1
                    for (int cc = 0; cc < kTrN; cc += 32) {
                        // Bits s0 .. s0 + 31 of the row's mask; keys before the tree are set.
                        const int s0 = j0 + cc - s.q.ctx;
                        uint32_t vis = __funnelshift_r(tree_word(row, s0 >> 5), tree_word(row, (s0 >> 5) + 1), s0 & 31);
                        uint32_t sr[32];
                        tmem_ld32(s_tm + cc, sr);
                        int dist[32];
                        if (tree) {
                            const int4* kp = reinterpret_cast<const int4*>(kpos + buf * kTrN + cc);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int4 k4 = kp[e];
                                dist[4 * e] = row.dep - k4.x, dist[4 * e + 1] = row.dep - k4.y;
                                dist[4 * e + 2] = row.dep - k4.z, dist[4 * e + 3] = row.dep - k4.w;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) dist[e] = row.dep - s0 - e;
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (static_cast<unsigned>(dist[e]) >= static_cast<unsigned>(wlim)) vis &= ~(1u << e);
                        float w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = 0.0f;
                        if (slice) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) w[e] = tab[(vis >> e) & 1u ? dist[e] - dlo : 0];
                        }
                        tmem_ld_wait_regs(sr);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            sr[e] = (vis >> e) & 1u ? __float_as_uint(fmaf(rs, w[e], __uint_as_float(sr[e])))
                                                    : 0xff800000u;
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
                float x[kTrN];
#pragma unroll
                for (int c = 0; c < kTrN; ++c) x[c] = __uint_as_float(sr[c]);
                if (slice && !edge) {
                    // Key c lies dep + 127 - c entries into the slice.
                    const float* w = tab + row.dep + (kTrN - 1);
#pragma unroll
                    for (int c = 0; c < kTrN; ++c) x[c] = fmaf(rs, w[-c], x[c]);
                }
                if (slice) {
                    // Eight arrivals free a slice: one per reading warp, two if only a slot's four read.
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars->tab_empty[buf]);
                        if (!s.two) mbar_arrive(&bars->tab_empty[buf]);
                    }
                }
                float mc[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mc[e] = fmaxf(x[2 * e], x[2 * e + 1]);
#pragma unroll
                for (int c = 16; c < kTrN; c += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mc[e] = fmax3f(mc[e], x[c + 2 * e], x[c + 2 * e + 1]);
                const float mx =
                    fmaxf(fmax3f(mc[0], mc[1], mc[2]), fmax3f(fmax3f(mc[3], mc[4], mc[5]), mc[6], mc[7])) * c1;
                if (t == t_first) {
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
                    f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), c1x2, nm2), x0, x1);
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
            if (!ok) break;

            // The next segment's row is fetched while this one's last products run.
            const TreeSeg cur = s;
            const TreeRow mine = row;
            const int units = cur.two ? 2 * cur.ntiles : cur.ntiles;
            nslice += cur.ntiles - cur.first_slice;
            parity ^= units & 1;
            more = walk.next(p, grp, npt, s);
            if (more) row = tree_row(p, s, 2 * grp + (s.two ? slot ^ parity : 0), ri, npt);

            // Epilogue.  Two row tiles: each slot writes its own rows.  One: both slots hold a
            // part of every row, in the same tensor-memory lanes; they exchange their maxima and
            // sums through shared memory and write half of the columns each.
            float la, lb;
            f2_unpack(l2, la, lb);
            float l = la + lb, m = m_used;
            float a_own = 1.0f, a_other = 0.0f;   // scales of the slots' O
            if (!cur.two) {
                float2* xch = reinterpret_cast<float2*>(smem + L::kXch) + (nx & 1) * 2 * kTrM;
                xch[slot * kTrM + ri] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->xch);
                if (!(ok = tree_all(mbar_wait(&bars->xch, nx & 1, abort_flag)))) break;
                ++nx;
                const float2 y = xch[(slot ^ 1) * kTrM + ri];
                const float top = fmaxf(m, y.x);
                a_own = m == -INFINITY ? 0.0f : ex2_approx(m - top);
                a_other = y.x == -INFINITY ? 0.0f : ex2_approx(y.x - top);
                l = l * a_own + y.y * a_other;
                m = top;
            }
            // Which slots' O hold something, and are waited for.
            const bool own = cur.two || ls == 0 || units > 1, other = !cur.two && (ls == 1 || units > 1);
            if (own && !(ok = tree_all(mbar_wait(&bars->o_final[slot], nf[slot] & 1, abort_flag)))) break;
            if (other && !(ok = tree_all(mbar_wait(&bars->o_final[slot ^ 1], nf[slot ^ 1] & 1, abort_flag)))) break;
            if (cur.two || ls == 0 || units > 1) ++nf[slot];
            if (cur.two || ls == 1 || units > 1) ++nf[slot ^ 1];
            tc_fence_after();
            const bool left = cur.tile0 > 0, right = cur.tile0 + cur.ntiles < cur.q.nt;
            const bool direct = !left && !right;
            if (direct) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                a_own *= inv;
                a_other *= inv;
            }
            const size_t orow = (static_cast<size_t>(cur.b) * p.T + mine.t) * p.Hq + h;
            // A run's first cut segment goes to its partial 0 if it comes from the run before, else to 1.
            float* rec = p.part + (static_cast<size_t>(blockIdx.x * 2 + (left ? 0 : 1)) * p.part_rows +
                                   (cur.two ? ls * kTrM : 0) + ri) * (D + kTrRec);
            const uint32_t o_tm = tmem_base + lane_off + 256;
            const int c_lo = cur.two ? 0 : slot * (D / 2), c_hi = cur.two ? D : c_lo + D / 2;
#pragma unroll 1
            for (int c = c_lo; c < c_hi; c += 32) {
                uint32_t y[32];
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                if (own) {
                    tmem_ld32(o_tm + slot * 128 + c, y);
                    tmem_ld_wait_regs(y);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(y[e]) * a_own;
                }
                if (other) {
                    tmem_ld32(o_tm + (slot ^ 1) * 128 + c, y);
                    tmem_ld_wait_regs(y);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(y[e]), a_other, v[e]);
                }
                if (mine.ok) {
                    if (direct) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            st_global_v4(p.o + orow * D + c + e, pack_bf16x2(v[e], v[e + 1]),
                                         pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]),
                                         pack_bf16x2(v[e + 6], v[e + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(rec + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
            }
            if (mine.ok && (cur.two || slot == 0)) {
                if (!direct) {
                    *reinterpret_cast<float2*>(rec + D) = make_float2(m, l);
                } else if (p.lse != nullptr) {
                    p.lse[(static_cast<size_t>(cur.b) * p.Hq + h) * p.T + mine.t] =
                        l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->o_free);
        }
    }

    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// Merges the partials of the segment that starts in run blockIdx.y and goes on in later
// runs (at most one per run): one warp per row.
constexpr int kTrCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kTrCombineWarps * 32) tree_combine_kernel(const TreeAttnParams p) {
    constexpr int E = D / 32;
    const int4 cut = p.cuts[blockIdx.y];   // {parts, sequence, key/value head, -}
    if (cut.x == 0) return;
    const int lane = threadIdx.x & 31, ri = blockIdx.x * kTrCombineWarps + (threadIdx.x >> 5);
    const int grp = blockIdx.y % p.groups, npt = kTrM / p.G;
    const int node = (ri & (kTrM - 1)) / p.G, hh = (ri & (kTrM - 1)) - node * p.G;
    const int t = (2 * grp + ri / kTrM) * npt + node, h = cut.z * p.G + hh;
    const TreeSeq q = tree_seq(p, __ldg(p.ctx_lens + cut.y), __ldg(p.tree_lens + cut.y));
    if (node >= npt || t >= q.n) return;
    // Part 0 is partial 1 of its run, the others partial 0 of theirs.
    auto rec = [&](int s) {
        return p.part + (static_cast<size_t>((blockIdx.y + s * p.groups) * 2 + (s == 0 ? 1 : 0)) * p.part_rows + ri) *
                            (D + kTrRec);
    };
    float M = -INFINITY;
    for (int s = lane; s < cut.x; s += 32) M = fmaxf(M, rec(s)[D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.0f, acc[E] = {};
#pragma unroll 4
    for (int s = 0; s < cut.x; ++s) {
        const float* x = rec(s);
        const float2 ml = *reinterpret_cast<const float2*>(x + D);
        const float a = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - M);
        l = fmaf(ml.y, a, l);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(x + lane * E + e);
            acc[e] = fmaf(v.x, a, acc[e]);
            acc[e + 1] = fmaf(v.y, a, acc[e + 1]);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + ((static_cast<size_t>(cut.y) * p.T + t) * p.Hq + h) * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse != nullptr && lane == 0)
        p.lse[(static_cast<size_t>(cut.y) * p.Hq + h) * p.T + t] = l > 0.0f ? (M + log2f(l)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, TreeAttnParams p,
                        cudaStream_t stream) {
    const int smem = tree_smem_bytes(D, p.G, p.T);
    p.tab_bufs = tree_tab_bufs(D, p.G, p.T);
    cudaError_t e =
        cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ctas = p.runs * p.groups;
    tree_attn_kernel<D><<<ctas, kTrThreads, smem, stream>>>(tq, tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.cuttable) return e;
    const int rows = p.part_rows > kTrM ? p.part_rows : p.T * p.G;
    tree_combine_kernel<D><<<dim3((rows + kTrCombineWarps - 1) / kTrCombineWarps, ctas), kTrCombineWarps * 32, 0,
                             stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Key tiles of the longest sequence: a windowed one may start up to a box before its first key.
int tree_max_tiles(int T, int max_ctx, int window, int box_rows) {
    const int rows = (window > 0 ? std::min(max_ctx, window - 1 + box_rows - 1) : max_ctx) + T;
    return (rows + kTrN - 1) / kTrN;
}

TreeLaunch tree_launch_plan(int B, int T, int Hkv, int G, int max_ctx, int window, int d, int sms) {
    TreeLaunch x{};
    const int npt = kTrM / G, row_tiles = (T + npt - 1) / npt;
    x.groups = (row_tiles + 1) / 2;
    x.part_rows = row_tiles > 1 ? 2 * kTrM : kTrM;
    const long long tiles = static_cast<long long>(B) * Hkv * tree_max_tiles(T, max_ctx, window, kTrN);
    x.runs = static_cast<int>(std::min<long long>(std::max(1, sms / x.groups), (tiles + kTrMinTiles - 1) / kTrMinTiles));
    const size_t ctas = static_cast<size_t>(x.runs) * x.groups;
    x.cut_bytes = (ctas * sizeof(int4) + 255) / 256 * 256;
    x.bytes = x.cut_bytes + ctas * 2 * x.part_rows * (d + kTrRec) * sizeof(float);
    return x;
}

cudaError_t launch_tree_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const TreeAttnParams& p, int d, cudaStream_t stream) {
    return d == 128 ? launch_tree<128>(tq, tk, tv, p, stream) : launch_tree<64>(tq, tk, tv, p, stream);
}

}  // namespace relbias
