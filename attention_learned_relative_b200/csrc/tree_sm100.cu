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
// an equal run of it: as many key tiles as any other whatever the lengths, in one wave.
// A run covers the end of one segment, whole segments, and the start of another; whole
// segments are written out directly, the two cut ones as partials (unnormalised output,
// max, sum) that the combine kernel merges.  Where segments are many and none can be long
// (tree_whole_segments), a run takes the whole segments that start in it instead: nothing
// is cut, and nothing combined, and a run exceeds its share by less than a segment.  CTAs
// of different row pairs run the same stream side by side, so a K/V tile comes from HBM
// once and from L2 for the others.
//
// Warp roles (640 threads):
//   warps 0-15      softmax and epilogue: slot = warp / 8, and within a slot two threads per
//                   row, 64 key columns each (warps w and w + 4, the same tensor-memory lanes)
//   warp 16         walks the run's segments and publishes them; TMA producer: Q per segment,
//                   K and V per key tile; a key tile is 128 / box_rows boxes, each inside one
//                   page, one lane per box
//   warp 17         TMEM allocator, zeroing of dead V rows, tcgen05.mma issuer
//   warps 18-19     bias stagers: the distances a key tile meets span 128 + T - 1 values, so
//                   they copy that slice of the group's tables to shared memory tile by
//                   tile (any R, and nothing for the tiles beyond R; one bulk copy per head),
//                   and for tiles with tree keys the keys' positions and the nodes' masks,
//                   aligned to the tile
// Units are (key tile, slot) pairs, alternating between the slots through all segments of
// the run; the MMA warp issues QK(u), then PV(u - 1).  Products of one thread run in issue
// order, so QK(u) may overwrite the P of unit u - 2, and when S(u) is complete O of its slot
// holds all earlier units.  A slot's chain QK, softmax, PV, next QK sets the period of the
// loop, not the products' rate, which is why a row's softmax is shared by two threads, and
// why one warp issues all products: with a warp for QK and one for PV the order of the two
// has to go through a barrier, which costs the chain more than the warps gain (131072-row
// case 1020 us against 870-918).  (One
// thread per row, eight softmax warps with 128 columns in registers, was also built: 3%
// faster on 131072-row caches with 64-node trees, 905-919 against 927-952 us, and 12% slower
// on the local layer, 51.2 against 45.7 us, before runs of whole segments.)
// Tensor memory: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D); each half's P (bf16)
// over the first half of its own columns of S.
//
// Softmax.  A thread takes its 64 columns of S twice, 32 at a time: for the maximum (adding
// the bias on the way, and storing the sum back), and, once the row's two halves have met
// and exchanged their maxima, for the weights.  The reference max of a row moves, and O is
// rescaled, only when the max has grown by more than 2^8.
//
// Measured, ten calls in a graph (a few milliseconds), and in brackets trains of fifty, calls or
// replays alike, in which the power cap takes the SM clock from 1965 to 1365-1515 MHz:
// 8 nodes on 1,048,560 rows, 32 heads on 4 of 128, 330-350 us, 0.94-0.99 of the copy rate, HBM-bound
// (360-430, 0.76-0.91); 64 nodes on eight caches of 73,728 to 131,072 rows 804-970 us, 874-1054
// TFLOP/s (950-970), bound by each slot's chain and the issue of its products; 16 nodes on 64
// windows of 512 32 us (start-up and the same chain); 4 nodes on a window of 64 9.5-9.9 us (cold
// loads in turn).
//
// Masks.  Sixteen-column chunks that hold tree keys are masked, and given their bias, by a
// pass over S in tensor memory before the softmax reads it.  Other chunks add their bias in
// registers, if any key is nearer than R, and are masked by one compare per key only in
// tiles that reach past some row's window.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "kernels.h"
#include "ptx.cuh"

namespace relbias {

namespace {

constexpr int kTrM = 128, kTrN = 128;      // rows of a row tile, keys of a key tile
constexpr int kTrThreads = 640, kTrSoftmaxWarps = 16;
// 640 threads launch with 96 registers each; the split gives the same total.
constexpr int kTrSoftmaxRegs = 104, kTrOtherRegs = 64;
constexpr float kTrGrow = 8.0f;            // log2 units: O is rescaled when a row's max grows by more
constexpr int kTrRec = 4;                  // floats of a partial record beyond its output: max, sum, pad
constexpr int kTrMaxStages = 4;            // of K, and of V
constexpr int kTrCutTiles = 4;             // what cutting segments costs, in key tiles
constexpr int kTrWholeTiles = 12;          // the longest segment that is never cut, in key tiles
constexpr int kTrSegs = 4;                 // published segments

template <int D>
struct TreeLayout {
    static constexpr int kTile = kTrM * D * 2;
    static constexpr int kBox = kTrM * 128;   // 128 rows of 64 columns
};

// A CTA's part of one (sequence, key/value head) segment.
struct TreeSeg {
    int b, g;
    int ctx, n, lo, end;   // as in TreeSeq
    int nt;                // key tiles of the whole segment
    int tile0, ntiles;     // this part's (ntiles 0: the run is over)
    int jbase;             // first row of the first one
    int first_slice;       // first tile with a slice of the bias table; all later ones have one
    int two;               // 1: two row tiles, 0: one whose key tiles the slots share
    int per;               // key tiles of a run
};

// Shared memory besides the tiles and slices.
struct TreeShared {
    float2 xch[2][4][kTrM];         // (max, sum) of each row from each slot and half, by segment parity
    float maxima[2][2][2][kTrM];    // [slot][tile parity][half]: a tile's row maxima
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kTrMaxStages], k_empty[kTrMaxStages], v_full[kTrMaxStages], v_empty[kTrMaxStages];
    uint64_t s_full[2], p_full[2], o_final[2], o_free;
    uint64_t pair[8];               // the two warps of a slot's 32 rows meet
    uint64_t tab_full[2], tab_empty[2];
    uint64_t seg_full[kTrSegs], seg_empty[kTrSegs];
    uint64_t xch_bar, mma_done;
    TreeSeg segs[kTrSegs];
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kTrSharedBytes = (static_cast<int>(sizeof(TreeShared)) + 15) / 16 * 16;

// Floats of a head's slice of the bias table: 128 + T - 1 distances and up to 3 before them (a
// slice starts on a 16-byte boundary of its table row), in a stride that is 4 modulo 32, so
// that eight heads at one depth meet eight different banks.
__host__ __device__ constexpr int tree_tab_stride(int T) { return (kTrN + T - 1 + 31) / 32 * 32 + 4; }

// A buffer of the stagers: masks of up to 128 nodes, four words each; key positions; a slice
// per head.
__host__ __device__ constexpr int tree_buf_bytes(int G, int T) {
    return kMaxTree * 16 + kTrN * 4 + G * tree_tab_stride(T) * 4;
}

// Stages and buffers that fit: [2 Q tiles][K ring][V ring][shared][stager buffers].
struct TreeSmem {
    int nk, nv, bufs, bytes;
};
TreeSmem tree_smem(int d, int G, int T) {
    const int tile = kTrM * d * 2, most = 232448 - 1024 - kTrSharedBytes;
    TreeSmem x{2, 2, 2, 0};
    if (6 * tile + 2 * tree_buf_bytes(G, T) > most) x.bufs = 1;
    if (10 * tile + x.bufs * tree_buf_bytes(G, T) <= most) x.nk = x.nv = 4;   // d 64
    // One CTA per SM: each allocates all of tensor memory.
    x.bytes = std::max((2 + x.nk + x.nv) * tile + kTrSharedBytes + x.bufs * tree_buf_bytes(G, T) + 1024, 120 * 1024);
    return x;
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
    s.base = s.lo & -p.box_rows;   // a power of two
    s.nt = s.n > 0 ? (s.end - s.base + kTrN - 1) / kTrN : 0;
    return s;
}

// Walks the segments of a CTA's run [pos, stop) of its row pair's tile stream.  The next
// sequence's lengths are loaded one sequence ahead.  (The host checks that a stream has
// fewer than 2^31 tiles.)
struct TreeWalk {
    int pos, stop, per;      // per: tiles of a run
    int b, g, off;           // current sequence, its next key/value head, next tile in that segment
    TreeSeq q;
    int next_ctx, next_n;

    __device__ __forceinline__ void fetch(const TreeAttnParams& p) {
        const int x = min(b + 1, p.B - 1);
        next_ctx = __ldg(p.ctx_lens + x);
        next_n = __ldg(p.tree_lens + x);
    }
    // Finds the start of run number `run`, by a whole warp: the stream's length, then the
    // sequence that holds the run's first tile.  head: the lengths of sequence `lane`.
    __device__ __forceinline__ void start(const TreeAttnParams& p, int grp, int npt, int run, int lane, int2 head) {
        auto tiles_of = [&](int x, TreeSeq& s) {
            s = x < 32 ? tree_seq(p, head.x, head.y) : tree_seq(p, __ldg(p.ctx_lens + x), __ldg(p.tree_lens + x));
            if (s.bad && grp == 0 && run == 0) atomicOr(&g_status, kStatusBadLength);
            return 2 * grp * npt < s.n ? s.nt * p.Hkv : 0;
        };
        int total = 0, mine = 0;   // mine: of this lane's sequence among the first 32
        TreeSeq s{};
        for (int x = lane; x < p.B; x += 32) {
            TreeSeq y;
            const int t = tiles_of(x, y);
            if (x < 32) mine = t, s = y;
            total += t;
        }
        total = __reduce_add_sync(0xffffffffu, total);
        per = max((total + p.runs - 1) / p.runs, 1);
        const long long at = static_cast<long long>(run) * per;
        pos = static_cast<int>(min(at, static_cast<long long>(total)));
        stop = min(total - pos, per) + pos;
        if (pos >= stop) return;
        for (int x0 = 0, prefix = 0;; x0 += 32) {
            if (x0 > 0) mine = x0 + lane < p.B ? tiles_of(x0 + lane, s) : 0;
            int scan = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, scan, o);
                if (lane >= o) scan += up;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, pos < prefix + scan);
            if (hit == 0) {
                prefix += __shfl_sync(0xffffffffu, scan, 31);
                continue;
            }
            const int w = __ffs(hit) - 1;   // the sequence that holds the run's first tile
            b = x0 + w;
            const int rest = pos - prefix - __shfl_sync(0xffffffffu, scan - mine, w);
            q.ctx = __shfl_sync(0xffffffffu, s.ctx, w);
            q.n = __shfl_sync(0xffffffffu, s.n, w);
            fetch(p);
            q = tree_seq(p, q.ctx, q.n);
            g = rest / q.nt;
            off = rest - g * q.nt;
            if (p.whole && off > 0) {   // its segment belongs to the run before
                pos += q.nt - off;
                off = 0;
                ++g;
            }
            return;
        }
    }
    __device__ __forceinline__ TreeSeg next(const TreeAttnParams& p, int grp, int npt) {
        TreeSeg s{};
        if (pos >= stop) return s;
        while (g == p.Hkv || 2 * grp * npt >= q.n) {   // the next sequence with rows of this pair
            ++b;
            g = 0;
            q = tree_seq(p, next_ctx, next_n);
            fetch(p);
        }
        s.b = b, s.g = g, s.ctx = q.ctx, s.n = q.n, s.lo = q.lo, s.end = q.end, s.nt = q.nt;
        s.tile0 = off;
        s.ntiles = p.whole ? q.nt : min(q.nt - off, stop - pos);
        s.jbase = q.base + off * kTrN;
        s.two = (2 * grp + 1) * npt < q.n;
        // A tile has a slice if it holds a prefix key nearer than R to a node of depth 0, or a
        // tree key.
        s.first_slice = min(max(0, (q.ctx - max(p.R, 1) + 1 - s.jbase) / kTrN), s.ntiles);
        s.per = per;
        pos += s.ntiles;
        off = 0;
        ++g;
        return s;
    }
};

// Depth of node t, clamped into [0, T).
__device__ __forceinline__ int tree_depth(const TreeAttnParams& p, int b, int t, bool& bad) {
    const int d = __ldg(p.depth + static_cast<size_t>(b) * p.T + t);
    bad = d < 0 || d >= p.T;
    return min(max(d, 0), p.T - 1);
}

// The products of one unit, by one thread.  Only the address part of a descriptor (its low
// 14 bits, in 16-byte steps) changes from step to step.
template <int D>
__device__ __forceinline__ void tree_issue_qk(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc) {
    const uint32_t idesc = idesc_bf16_f32(kTrM, kTrN, false, false);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = ((kk & 3) * 32 + (kk >> 2) * TreeLayout<D>::kBox) >> 4;
        umma_ss(d_tmem, q_desc + off, k_desc + off, idesc, kk > 0 ? 1u : 0u);
    }
}

template <int D>
__device__ __forceinline__ void tree_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t v_desc, bool accumulate) {
    const uint32_t idesc = idesc_bf16_f32(kTrM, D, false, true);
#pragma unroll
    for (int kk = 0; kk < kTrN / 16; ++kk)
        // P of keys 0-63 and 64-127: 32 columns each, 64 apart.
        umma_ts(d_tmem, p_tmem + (kk & 3) * 8 + (kk >> 2) * 64, v_desc + ((kk * 16 * 128) >> 4), idesc,
                (accumulate || kk > 0) ? 1u : 0u);
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

// A run of 16-byte units from global to shared memory, signalled on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// Four bytes from global to shared memory, asynchronously, and the wait for a thread's own.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Piece (lane & 3) of rows (lane & ~3) + e, e < 4, from four pieces of each lane's own row.
__device__ __forceinline__ void tree_transpose4(uint4 (&u)[4], int lane) {
    auto trade = [&](uint32_t& lo, uint32_t& hi, int m) {   // lo: index bit m clear, hi: set
        const uint32_t y = __shfl_xor_sync(0xffffffffu, (lane & m) ? lo : hi, m);
        if (lane & m) lo = y; else hi = y;
    };
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!(k & m)) {
                trade(u[k].x, u[k | m].x, m);
                trade(u[k].y, u[k | m].y, m);
                trade(u[k].z, u[k | m].z, m);
                trade(u[k].w, u[k | m].w, m);
            }
}

// Log-sum-exp of a row from its reference max (log2 units) and the sum against it.  A row
// that sees nothing has a sum of 0.  A NaN or +inf logit leaves the max as it was, or at
// +inf, but makes the sum NaN, and the log-sum-exp with it.
__device__ __forceinline__ float tree_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ bool tree_all(bool ok) { return __all_sync(0xffffffffu, ok); }

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
    uint8_t* q_tiles = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* k_ring = q_tiles + 2 * L::kTile;
    uint8_t* v_ring = k_ring + p.nk * L::kTile;
    TreeShared* sh = reinterpret_cast<TreeShared*>(v_ring + p.nv * L::kTile);
    uint8_t* bufs = reinterpret_cast<uint8_t*>(sh) + kTrSharedBytes;
    const int tstride = tree_tab_stride(p.T), buf_bytes = tree_buf_bytes(p.G, p.T);
    volatile int* abort_flag = &sh->abort_flag;

    // The schedule's first loads are under way while the bars are set up.
    int2 head = make_int2(0, 0);
    if (warp == 16 && lane < p.B) head = make_int2(__ldg(p.ctx_lens + lane), __ldg(p.tree_lens + lane));
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->q_full[s], 1);
            mbar_init(&sh->q_empty[s], 1);
            mbar_init(&sh->s_full[s], 1);
            mbar_init(&sh->p_full[s], 8);
            mbar_init(&sh->o_final[s], 1);
            mbar_init(&sh->tab_full[s], 2);
            mbar_init(&sh->tab_empty[s], kTrSoftmaxWarps);
        }
        for (int s = 0; s < kTrMaxStages; ++s) {
            mbar_init(&sh->k_full[s], 1);
            mbar_init(&sh->k_empty[s], 1);
            mbar_init(&sh->v_full[s], 1);
            mbar_init(&sh->v_empty[s], 1);
        }
        for (int s = 0; s < 8; ++s) mbar_init(&sh->pair[s], 2);
        for (int s = 0; s < kTrSegs; ++s) {
            mbar_init(&sh->seg_full[s], 1);
            mbar_init(&sh->seg_empty[s], kTrSoftmaxWarps + 3);
        }
        mbar_init(&sh->o_free, kTrSoftmaxWarps);
        mbar_init(&sh->xch_bar, kTrSoftmaxWarps);
        mbar_init(&sh->mma_done, 1);
        sh->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(&sh->tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    if (warp == 16 && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }

    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sh->tmem_base;

    // Consumers of the published segments: wait for number i, and give it back.
    auto seg_wait = [&](int i) { return tree_all(mbar_wait(&sh->seg_full[i % kTrSegs], (i / kTrSegs) & 1, abort_flag)); };
    auto seg_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->seg_empty[i % kTrSegs]);
    };

    if (warp >= kTrSoftmaxWarps) {
        regs_decrease<kTrOtherRegs>();
        if (warp == 16) {
            // ------------------------------------------------------------ schedule and TMA producer
            const bool leader = elect_one();
            const int nboxes = kTrN / p.box_rows;
            TreeWalk walk;
            walk.start(p, grp, npt, run, lane, head);
            bool ok = true;
            int nk = 0, nv = 0, ks = 0, vs = 0, kph = 1, vph = 1;   // loads issued; next stages and their phases
            int nq[2] = {0, 0};                                     // loads of each Q buffer
            // A key tile's V is loaded after the next tile's K, the order in which they are used.
            int v_page = 0, v_row = 0, v_head = -1;
            auto load = [&](bool is_v, int page, int prow, int head) -> bool {
                uint64_t* full = is_v ? &sh->v_full[vs] : &sh->k_full[ks];
                if (!tree_all(mbar_wait(is_v ? &sh->v_empty[vs] : &sh->k_empty[ks], is_v ? vph : kph, abort_flag)))
                    return false;
                if (leader) mbar_arrive_expect_tx(full, L::kTile);
                __syncwarp();
                if (lane < nboxes) {
                    uint8_t* dst = (is_v ? v_ring + vs * L::kTile : k_ring + ks * L::kTile) + lane * p.box_rows * 128;
                    for (int bx = 0; bx < D / 64; ++bx)
                        tma_load_4d(dst + bx * L::kBox, is_v ? &tm_v : &tm_k, full, bx * 64, head, prow, page);
                }
                __syncwarp();
                if (is_v) {
                    ++nv;
                    if (++vs == p.nv) vs = 0, vph ^= 1;
                } else {
                    ++nk;
                    if (++ks == p.nk) ks = 0, kph ^= 1;
                }
                return true;
            };
            for (int i = 0; ok; ++i) {
                const TreeSeg s = walk.next(p, grp, npt);
                if (!(ok = tree_all(mbar_wait(&sh->seg_empty[i % kTrSegs], ((i / kTrSegs) & 1) ^ 1, abort_flag)))) break;
                if (lane == 0) {
                    sh->segs[i % kTrSegs] = s;
                    mbar_arrive(&sh->seg_full[i % kTrSegs]);
                }
                __syncwarp();
                if (s.ntiles == 0) break;
                // This lane's box of key tile t: its page (-1, which reads zeros, past the
                // sequence's end or for an index outside the pool) and its row in the page.
                auto lookup = [&](int t, int& page, int& prow) {
                    page = -1, prow = 0;
                    const int row = s.jbase + t * kTrN + lane * p.box_rows;
                    if (t >= s.ntiles || lane >= nboxes || row >= s.end) return;
                    const int blk = static_cast<int>(static_cast<uint64_t>(row) * p.page_mul >> p.page_shift);
                    prow = row - blk * p.page_size;
                    page = __ldg(p.block_table + static_cast<size_t>(s.b) * p.max_pages + blk);
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(&g_status, kStatusBadLength);
                        page = -1, prow = 0;
                    }
                };
                int page, prow, next_page, next_row;
                lookup(0, next_page, next_row);
                // Two row tiles go to buffers 0 and 1; single ones alternate, so that a segment's queries
                // arrive while the one before is still being read.
                for (int r = 0; r < (s.two ? 2 : 1); ++r) {
                    const int buf = s.two ? r : i & 1;
                    if (!(ok = tree_all(mbar_wait(&sh->q_empty[buf], (nq[buf] & 1) ^ 1, abort_flag)))) break;
                    if (leader) {
                        mbar_arrive_expect_tx(&sh->q_full[buf], npt * p.G * 128 * (D / 64));
                        for (int bx = 0; bx < D / 64; ++bx)
                            tma_load_4d(q_tiles + buf * L::kTile + bx * L::kBox, &tm_q, &sh->q_full[buf], bx * 64,
                                        s.g * p.G, (2 * grp + r) * npt, s.b);
                    }
                    ++nq[buf];
                }
                for (int t = 0; ok && t < s.ntiles; ++t) {
                    page = next_page, prow = next_row;
                    lookup(t + 1, next_page, next_row);
                    if (!(ok = load(false, page, prow, s.g))) break;
                    if (v_head >= 0 && !(ok = load(true, v_page, v_row, v_head))) break;
                    v_page = page, v_row = prow, v_head = s.g;
                }
            }
            if (ok && v_head >= 0) load(true, v_page, v_row, v_head);
            // Drain, also after an abort: no copy may be in flight when the CTA exits.
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0) mbar_drain_wait(&sh->q_full[x], (nq[x] - 1) & 1);
            for (int n = max(0, nk - p.nk); n < nk; ++n) mbar_drain_wait(&sh->k_full[n % p.nk], (n / p.nk) & 1);
            for (int n = max(0, nv - p.nv); n < nv; ++n) mbar_drain_wait(&sh->v_full[n % p.nv], (n / p.nv) & 1);
        } else if (warp == 17) {
            // ------------------------------------------------------------ MMA issuer
            // The whole warp runs the loop and waits; one thread issues.  Between two batches of
            // products this warp's own work is what the tensor cores wait for, so it is short: no
            // arrays, phases as bits.
            const bool leader = elect_one();
            const uint64_t q_desc = smem_desc_sw128(smem_u32(q_tiles), 16, 1024),
                           k_desc = smem_desc_sw128(smem_u32(k_ring), 16, 1024),
                           v_desc = smem_desc_sw128(smem_u32(v_ring), L::kBox, 1024);
            constexpr uint32_t kStep = L::kTile >> 4;
            bool ok = true;
            uint32_t q_phase = 0, p_phase = 0;   // by Q buffer, by slot
            uint32_t ks = 0, k_phase = 0, vs = 0, v_phase = 0, parity = 0;
            // The unit whose PV is still to be issued (pv_slot 2: none), its tile's live rows, and
            // whether it opens and closes its V stage and its segment's products.
            uint32_t pv_slot = 2, pv_seg = 0;
            int pv_lo = 0, pv_end = 0;
            bool pv_opens = false, pv_closes = false, pv_adds = false, pv_last = false;
            // PV of the pending unit; the next unit's QK has been issued.
            auto issue_pv = [&]() -> bool {
                if (pv_opens) {
                    if (!tree_all(mbar_wait(&sh->v_full[vs], v_phase, abort_flag))) return false;
                    // Rows no node sees by position may hold anything, and a NaN times a zero
                    // weight is NaN: zero them before the first product reads them.
                    if (pv_end < kTrN) tree_zero_rows<D>(v_ring + vs * L::kTile, pv_end, kTrN, lane);
                    if (pv_lo > 0) tree_zero_rows<D>(v_ring + vs * L::kTile, 0, pv_lo, lane);
                    // A segment's first product overwrites O: all epilogues of the one before are done.
                    if (pv_seg > 0 && !tree_all(mbar_wait(&sh->o_free, (pv_seg - 1) & 1, abort_flag))) return false;
                }
                if (!tree_all(mbar_wait(&sh->p_full[pv_slot], (p_phase >> pv_slot) & 1, abort_flag))) return false;
                p_phase ^= 1u << pv_slot;
                tc_fence_after();
                if (leader) {
                    tree_issue_pv<D>(tmem_base + 256 + pv_slot * 128, tmem_base + pv_slot * 128, v_desc + vs * kStep,
                                     pv_adds);
                    if (pv_closes) umma_commit(&sh->v_empty[vs]);
                    if (pv_last) umma_commit(&sh->o_final[pv_slot]);
                }
                __syncwarp();
                if (pv_closes && ++vs == static_cast<uint32_t>(p.nv)) vs = 0, v_phase ^= 1;
                return true;
            };
            for (int i = 0; ok; ++i) {
                if (!(ok = seg_wait(i))) break;
                const TreeSeg& s = sh->segs[i % kTrSegs];
                const int ntiles = s.ntiles, two = s.two, units = two ? 2 * ntiles : ntiles;
                int lo = s.lo - s.jbase, end = s.end - s.jbase;   // live rows, from the current tile's first
                seg_done(i);
                if (ntiles == 0) break;
                for (int u = 0; u < units; ++u) {
                    const uint32_t ls = u & 1, slot = ls ^ parity;
                    const uint32_t buf = two ? ls : i & 1;
                    const bool opens = !two || ls == 0, closes = !two || ls == 1;
                    if (opens && !(ok = tree_all(mbar_wait(&sh->k_full[ks], k_phase, abort_flag)))) break;
                    if (u <= two) {   // the unit reads its row tile for the first time
                        if (!(ok = tree_all(mbar_wait(&sh->q_full[buf], (q_phase >> buf) & 1, abort_flag)))) break;
                        q_phase ^= 1u << buf;
                    }
                    tc_fence_after();
                    if (leader) {
                        tree_issue_qk<D>(tmem_base + slot * 128, q_desc + buf * kStep, k_desc + ks * kStep);
                        umma_commit(&sh->s_full[slot]);
                        if (closes) umma_commit(&sh->k_empty[ks]);
                        if (u + 1 + two >= units) umma_commit(&sh->q_empty[buf]);
                    }
                    __syncwarp();
                    if (closes && ++ks == static_cast<uint32_t>(p.nk)) ks = 0, k_phase ^= 1;
                    if (pv_slot < 2 && !(ok = issue_pv())) break;
                    pv_slot = slot, pv_seg = u == 0 ? i : 0, pv_lo = lo, pv_end = end;
                    pv_opens = opens, pv_closes = closes, pv_adds = u >= 2, pv_last = u + 2 >= units;
                    if (closes) lo -= kTrN, end -= kTrN;
                }
                parity ^= units & 1;
            }
            if (ok && pv_slot < 2) issue_pv();
            // Drain: every product issued has finished before tensor memory is released.
            if (leader) umma_commit(&sh->mma_done);
            mbar_drain_wait(&sh->mma_done, 0);
        } else {
            // ------------------------------------------------------------ stagers
            const int x0 = threadIdx.x - (kTrSoftmaxWarps + 2) * 32;   // 0..63
            const int width = kTrN + p.T - 1 + 3;
            int n = 0;
            int4 cut = make_int4(0, 0, 0, 0);
            bool ok = true;
            for (int i = 0; ok; ++i) {
                if (!(ok = seg_wait(i))) break;
                const TreeSeg s = sh->segs[i % kTrSegs];
                seg_done(i);
                if (s.ntiles == 0) break;
                const int after = s.nt - s.tile0 - s.ntiles;
                if (s.tile0 == 0 && after > 0) {   // never, where runs take whole segments
                    // The segment starts here and goes on in the next runs.
                    cut = make_int4(1 + (after + s.per - 1) / s.per, s.b, s.g, s.n);
                }
                for (int t = s.first_slice; t < s.ntiles; ++t, ++n) {
                    // Slice n signals on bars n % 2, phase n / 2, so that a slot meets one pair of bars in a
                    // segment, every phase of them, with one buffer as with two.  The buffer is free
                    // when slice n - 2, or with one buffer slice n - 1, has been read.
                    const int buf = n & 1, last = n - p.tab_bufs;
                    if (last >= 0 &&
                        !(ok = tree_all(mbar_wait(&sh->tab_empty[last & 1], (last >> 1) & 1, abort_flag))))
                        break;
                    uint32_t* vis = reinterpret_cast<uint32_t*>(bufs + (p.tab_bufs == 2 ? buf : 0) * buf_bytes);
                    int* kpos = reinterpret_cast<int*>(vis + kMaxTree * 4);
                    float* tab = reinterpret_cast<float*>(kpos + kTrN);
                    const int j0 = s.jbase + t * kTrN;
                    // The slice starts at the nearest key's distance from depth 0 (0 with tree keys),
                    // rounded down to a 16-byte boundary.  Where the table ends in it, zeros follow.
                    const int dlo = max(s.ctx - j0 - (kTrN - 1), 0) & ~3;
                    const int in = min(max(p.R - dlo, 0), (width + 3) & ~3);
                    const float* src = p.w + static_cast<size_t>(s.g) * p.G * p.R + dlo;
                    if (p.w_bulk) {
                        // Every row starts on a 16-byte boundary and `in` is a multiple of 4.
                        if (warp == kTrSoftmaxWarps + 2) {
                            if (lane == 0 && in > 0) mbar_expect_tx(&sh->tab_full[buf], p.G * in * 4);
                            __syncwarp();
                            if (in > 0 && lane < p.G)
                                bulk_load(tab + lane * tstride, src + static_cast<size_t>(lane) * p.R, in * 4,
                                          &sh->tab_full[buf]);
                        }
                    } else {
                        for (int h = 0; h < p.G; ++h)
                            for (int x = x0; x < min(in, width); x += 64)
                                cp_async4(tab + h * tstride + x, src + static_cast<size_t>(h) * p.R + x);
                    }
                    if (in < width) {
                        for (int h = 0; h < p.G; ++h)
                            for (int x = in + x0; x < width; x += 64) tab[h * tstride + x] = 0.0f;
                        fence_proxy_async_shared();   // before later bulk copies into the same place
                    }
                    if (j0 + kTrN > s.ctx) {
                        // Position of each key less ctx; dead keys are in no mask.
                        for (int c = x0; c < kTrN; c += 64) {
                            const int x = j0 + c - s.ctx;
                            bool bad;
                            kpos[c] = x < 0 ? x : x < s.n ? tree_depth(p, s.b, x, bad) : 0;
                        }
                        // Which keys each node of this row pair may see: all of the prefix, and by mask.
                        const int first = 2 * grp * npt, nodes = min(2 * npt, s.n - first);
                        for (int x = x0; x < 4 * nodes; x += 64) {
                            const int bit = j0 + (x & 3) * 32 - s.ctx;   // the tree node of the word's bit 0
                            const int* words = p.mask + (static_cast<size_t>(s.b) * p.T + first + (x >> 2)) * p.words;
                            auto word = [&](int k) -> uint32_t {
                                uint32_t w = k < 0 ? 0xffffffffu : k < p.words ? __ldg(words + k) : 0u;
                                if (k >= 0 && s.n - 32 * k < 32) w = s.n > 32 * k ? w & ((1u << (s.n - 32 * k)) - 1u) : 0u;
                                return w;
                            };
                            vis[x] = __funnelshift_r(word(bit >> 5), word((bit >> 5) + 1), bit & 31);
                        }
                    }
                    if (!p.w_bulk) cp_async_wait_all();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->tab_full[buf]);
                }
            }
            if (x0 == 0) p.cuts[blockIdx.x] = cut;
            // Drain the bulk copies.  After an abort the second warp may be a slice behind the first,
            // which issues them: it arrives in its place.
            if (!ok && lane == 0 && warp == kTrSoftmaxWarps + 3)
                for (int x = 0; x < 2; ++x) mbar_arrive(&sh->tab_full[x]);
            if (p.w_bulk && warp == kTrSoftmaxWarps + 2)
                for (int x = max(0, n - 2); x < n; ++x) mbar_drain_wait(&sh->tab_full[x & 1], (x >> 1) & 1);
        }
    } else {
        // ---------------------------------------------------------------- softmax / epilogue
        regs_increase<kTrSoftmaxRegs>();
        const int slot = warp >> 3, half = (warp >> 2) & 1;
        const int ri = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t s_tm = tmem_base + lane_off + slot * 128 + half * 64;   // this thread's 64 columns of S
        uint64_t* pair = &sh->pair[slot * 4 + (warp & 3)];
        const int node = ri / p.G, hh = ri - node * p.G;
        const int wlim = p.window > 0 ? p.window : INT_MAX;
        bool ok = true;
        int ns = 0, nslice = 0, parity = 0;    // S tiles of this slot; slices, and units (modulo 2), of earlier segments
        int nf[2] = {0, 0};                    // finals of each slot
        // This thread's row of a segment: loaded one segment ahead.
        struct {
            int t, dep;
            bool ok;
            float r;
        } row{};
        auto load_row = [&](const TreeSeg& s, int part) {
            row.t = (2 * grp + (s.two ? part : 0)) * npt + node;
            row.ok = node < npt && row.t < s.n;
            const size_t at = static_cast<size_t>(s.b) * p.T + (row.ok ? row.t : 0);
            row.dep = __ldg(p.depth + at);
            // Without a table r has no say, whatever it holds (tiles with tree keys multiply it by 0).
            row.r = row.ok && p.R > 0 ? __ldg(p.r + at * p.Hq + s.g * p.G + hh) : 0.0f;
        };
        if ((ok = seg_wait(0)) && sh->segs[0].ntiles > 0) load_row(sh->segs[0], slot);
        for (int i = 0; ok; ++i) {
            const TreeSeg& s = sh->segs[i % kTrSegs];
            const int ntiles = s.ntiles;
            if (ntiles == 0) break;
            const int two = s.two, ctx = s.ctx, nodes = s.n, first_slice = s.first_slice, jbase = s.jbase;
            const int ls = slot ^ parity;      // this slot's part: its row tile, or its half of the key tiles
            const int t_node = row.t;
            const bool row_ok = row.ok;
            if (row_ok && (row.dep < 0 || row.dep >= p.T)) atomicOr(&g_status, kStatusBadTree);
            const int dep = min(max(row.dep, 0), p.T - 1);
            const float rs = row.r * p.inv_scale;
            float c1 = p.scale_log2;
            // Context-length temperature: a row that sees n > temp_n0 keys (by position) has its
            // logits, content and bias, scaled by ln n / ln temp_n0.
            if (p.temp_n0 > 1) {
                const int seen = min(ctx + dep + 1, wlim);
                if (seen > p.temp_n0) c1 *= logf(static_cast<float>(seen)) * p.inv_log_n0;
            }
            const uint64_t c1x2 = f2_pack(c1, c1);
            float m_used = -INFINITY;   // running reference max, log2 units
            uint64_t l2 = 0;            // running sum of this half's weights against it, in two lanes
            bool first = true;
            for (int t = two ? 0 : ls; t < ntiles; t += two ? 1 : 2, ++ns) {
                const int j0 = jbase + t * kTrN;
                const bool slice = t >= first_slice;
                const int n = nslice + t - first_slice;
                const int buf = n & 1;
                const uint32_t* vis = reinterpret_cast<const uint32_t*>(bufs + (p.tab_bufs == 2 ? buf : 0) * buf_bytes);
                const int* kpos = reinterpret_cast<const int*>(vis + kMaxTree * 4);
                const float* tab = reinterpret_cast<const float*>(kpos + kTrN) + hh * tstride;
                if (!(ok = tree_all(mbar_wait(&sh->s_full[slot], ns & 1, abort_flag)))) break;
                if (slice && !(ok = tree_all(mbar_wait(&sh->tab_full[buf], (n >> 1) & 1, abort_flag)))) break;
                tc_fence_after();
                const int own0 = ctx - j0 - half * 64;         // this half's first column with a tree key
                const int dlo = max(ctx - j0 - (kTrN - 1), 0) & ~3;   // the slice's first distance
                if (own0 < 64) {
                    // Bias and masks of the chunks with tree keys, back into S.
                    const uint32_t* mine_vis = vis + (row_ok ? (t_node - 2 * grp * npt) * 4 : 0) + half * 2;
#pragma unroll 1
                    for (int cc = max(own0, 0) & ~15; cc < 64; cc += 16) {
                        if (cc >= own0 + nodes) {   // past the tree: nothing to look up
                            uint32_t none[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) none[e] = 0xff800000u;
                            tmem_st16(s_tm + cc, none);
                            tmem_st_wait();
                            tmem_regs_keep16(none);
                            continue;
                        }
                        uint32_t see = mine_vis[cc >> 5] >> (cc & 16);
                        uint32_t sr[16];
                        tmem_ld16(s_tm + cc, sr);
                        const int4* kp = reinterpret_cast<const int4*>(kpos + half * 64 + cc);
                        float w[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int4 k4 = kp[e];
                            const int ks[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                            for (int f = 0; f < 4; ++f) {
                                const int dist = dep - ks[f];
                                if (static_cast<unsigned>(dist) >= static_cast<unsigned>(wlim)) see &= ~(1u << (4 * e + f));
                                w[4 * e + f] = tab[min(max(dist - dlo, 0), kTrN + p.T + 1)];
                            }
                        }
                        tmem_ld_wait_regs16(sr);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            sr[e] = (see >> e) & 1u ? __float_as_uint(fmaf(rs, w[e], __uint_as_float(sr[e])))
                                                    : 0xff800000u;
                        tmem_st16(s_tm + cc, sr);
                        tmem_st_wait();
                        tmem_regs_keep16(sr);
                    }
                }
                // The maximum, with the bias of the other chunks, and one compare per key where some
                // row's window starts inside the tile (first column inside it: wcol).
                const int wcol = wlim == INT_MAX ? INT_MIN : own0 + dep - wlim + 1;
                const bool cuts_in = __any_sync(0xffffffffu, wcol > 0);
                float mc[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int cc = 0; cc < 64; cc += 32) {
                    uint32_t x[32];
                    tmem_ld32(s_tm + cc, x);
                    tmem_ld_wait_regs(x);
                    if ((slice || cuts_in) && cc + 16 <= own0) {
                        const float* w = tab + dep + own0 - dlo - cc;   // a prefix key's distance is dep + ctx less its row
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            if (cc + h + 16 <= own0) {
                                if (slice) {
#pragma unroll
                                    for (int c = h; c < h + 16; ++c)
                                        x[c] = __float_as_uint(fmaf(rs, w[-c], __uint_as_float(x[c])));
                                }
                                if (cuts_in) {
#pragma unroll
                                    for (int c = h; c < h + 16; ++c) x[c] = cc + c < wcol ? 0xff800000u : x[c];
                                }
                            }
                        }
                        tmem_st32(s_tm + cc, x);
                        tmem_st_wait();
                        tmem_regs_keep16(x);
                        tmem_regs_keep16(x + 16);
                    }
#pragma unroll
                    for (int c = 0; c < 32; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mc[e] = fmax3f(mc[e], __uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
                }
                const float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
                sh->maxima[slot][ns & 1][half][ri] = mx;
                __syncwarp();
                if (lane == 0) mbar_arrive(pair);
                if (!(ok = tree_all(mbar_wait(pair, ns & 1, abort_flag)))) break;
                const float top = fmaxf(mx, sh->maxima[slot][ns & 1][half ^ 1][ri]) * c1;
                if (first) {
                    m_used = top;
                    first = false;
                } else if (__any_sync(0xffffffffu, top > m_used + kTrGrow)) {
                    // Some row's max grew past the slack (or is its first): what has been summed is
                    // scaled to the new reference, each half of the row's threads its half of O.
                    const bool grow = top > m_used + kTrGrow;
                    const float alpha = !grow ? 1.0f : m_used == -INFINITY ? 0.0f : ex2_approx(m_used - top);
                    m_used = grow ? top : m_used;
                    l2 = f2_mul(l2, f2_pack(alpha, alpha));
                    const uint32_t o_tm = tmem_base + lane_off + 256 + slot * 128 + half * (D / 2);
                    uint32_t ob[32];
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 32) {
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
                uint64_t acc[2] = {0, 0};
#pragma unroll 1
                for (int cc = 0; cc < 64; cc += 32) {
                    uint32_t x[32], pk[16];
                    tmem_ld32(s_tm + cc, x);
                    tmem_ld_wait_regs(x);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float p0, p1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), c1x2, nm2), p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        acc[(c >> 1) & 1] = f2_add(acc[(c >> 1) & 1], f2_pack(p0, p1));
                        // Weights are rounded to bf16 for the tensor cores (2^-8 of each at most,
                        // while their sum stays in fp32).
                        pk[c / 2] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(s_tm + cc / 2, pk);   // over columns of S that have been read
                    tmem_st_wait();
                    tmem_regs_keep16(pk);
                }
                l2 = f2_add(l2, f2_add(acc[0], acc[1]));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh->p_full[slot]);
                    // Sixteen arrivals free a slice: one per reading warp, two if only a slot's eight read.
                    if (slice) {
                        mbar_arrive(&sh->tab_empty[buf]);
                        if (!two) mbar_arrive(&sh->tab_empty[buf]);
                    }
                }
            }
            if (!ok) break;

            // Epilogue.  The threads exchange their maxima and sums: the two halves of a row have
            // one max and two sums; with one row tile the slots' parts of a row, in the same
            // tensor-memory lanes, also have two maxima.  Each thread then writes a half (two row
            // tiles) or a quarter of its row's columns.
            const int units = two ? 2 * ntiles : ntiles;
            // The next segment's row is on its way meanwhile.
            if (!(ok = seg_wait(i + 1))) break;
            if (sh->segs[(i + 1) % kTrSegs].ntiles > 0)
                load_row(sh->segs[(i + 1) % kTrSegs], slot ^ parity ^ (units & 1));
            float la, lb;
            f2_unpack(l2, la, lb);
            float2* xch = sh->xch[i & 1][0];
            xch[(slot * 2 + half) * kTrM + ri] = make_float2(m_used, la + lb);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->xch_bar);
            if (!(ok = tree_all(mbar_wait(&sh->xch_bar, i & 1, abort_flag)))) break;
            float m = m_used;
            float l = xch[slot * 2 * kTrM + ri].y + xch[(slot * 2 + 1) * kTrM + ri].y;
            float a_own = 1.0f, a_other = 0.0f;   // scales of the slots' O
            if (!two) {
                const float mo = xch[(slot ^ 1) * 2 * kTrM + ri].x;
                const float lo = xch[(slot ^ 1) * 2 * kTrM + ri].y + xch[((slot ^ 1) * 2 + 1) * kTrM + ri].y;
                const float top = fmaxf(m, mo);
                a_own = m == -INFINITY ? 0.0f : ex2_approx(m - top);
                a_other = mo == -INFINITY ? 0.0f : ex2_approx(mo - top);
                l = l * a_own + lo * a_other;
                m = top;
            }
            const bool left = s.tile0 > 0, direct = !left && ntiles == s.nt;
            if (direct) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                a_own *= inv;
                a_other *= inv;
            }
            const int h = s.g * p.G + hh;
            // Output rows: of the sequence's first node and head 0, and this thread's from there.
            const size_t obase = static_cast<size_t>(s.b) * p.T * p.Hq;
            const int orow = t_node * p.Hq + h;
            const unsigned ok_rows = __ballot_sync(0xffffffffu, row_ok);
            // A run's first cut segment goes to its partial 0 if it comes from the run before, else to 1.
            float* rec = p.part + (static_cast<size_t>(blockIdx.x * 2 + (left ? 0 : 1)) * p.part_rows +
                                   (two ? ls * kTrM : 0) + ri) * (D + kTrRec);
            const uint32_t o_tm = tmem_base + lane_off + 256;
            const int part = two ? half : slot * 2 + half, width = two ? D / 2 : D / 4;
            if (row_ok && part == 0) {
                if (!direct) {
                    *reinterpret_cast<float2*>(rec + D) = make_float2(m, l);
                } else if (p.lse != nullptr) {
                    p.lse[(static_cast<size_t>(s.b) * p.Hq + h) * p.T + t_node] = tree_lse(m, l);
                }
            }
            // Which slots' O hold something, and are waited for.
            const bool own = two || ls == 0 || units > 1, other = !two && (ls == 1 || units > 1);
            if (own && !(ok = tree_all(mbar_wait(&sh->o_final[slot], nf[slot] & 1, abort_flag)))) break;
            if (other && !(ok = tree_all(mbar_wait(&sh->o_final[slot ^ 1], nf[slot ^ 1] & 1, abort_flag)))) break;
            if (own) ++nf[slot];
            if (two || ls == 1 || units > 1) ++nf[slot ^ 1];
            tc_fence_after();
#pragma unroll 1
            for (int c = part * width; c < (part + 1) * width; c += 32) {
                // 32 columns; of a one-row-tile segment at d 64 a thread has 16, and takes its
                // neighbour's along unwritten.
                const int cols = min(width, 32);
                uint32_t y[32], z[32];
                tmem_ld32(o_tm + slot * 128 + c, y);
                tmem_ld32(o_tm + (slot ^ 1) * 128 + c, z);
                tmem_ld_wait_regs(y);
                tmem_regs_fence(z);
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    v[e] = own ? __uint_as_float(y[e]) * a_own : 0.0f;
                    v[e] = other ? fmaf(__uint_as_float(z[e]), a_other, v[e]) : v[e];
                }
                // A thread holds 32 columns of its row; groups of four lanes trade 16-byte pieces, so
                // that a store writes 64 bytes of each of eight rows and not 16 of 32 (the lines that a
                // store touches are its cost: 3.5k -> 1.3k cycles per segment).
                if (direct) {
                    uint4 u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        u[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                                          pack_bf16x2(v[8 * e + 4], v[8 * e + 5]),
                                          pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
                    tree_transpose4(u, lane);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int from = (lane & ~3) + e, at = __shfl_sync(0xffffffffu, orow, from);
                        if (((ok_rows >> from) & 1u) && (lane & 3) * 8 < cols)
                            st_global_v4(p.o + (obase + at) * D + c + (lane & 3) * 8, u[e].x, u[e].y, u[e].z, u[e].w);
                    }
                } else {
#pragma unroll
                    for (int x2 = 0; x2 < 2; ++x2) {
                        uint4 u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float* f = v + 16 * x2 + 4 * e;
                            u[e] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                              __float_as_uint(f[3]));
                        }
                        tree_transpose4(u, lane);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int from = (lane & ~3) + e;
                            if (((ok_rows >> from) & 1u) && 16 * x2 < cols)
                                *reinterpret_cast<uint4*>(rec + (from - lane) * (D + kTrRec) + c + 16 * x2 +
                                                          (lane & 3) * 4) = u[e];
                        }
                    }
                }
            }
            nslice += ntiles - first_slice;
            parity ^= units & 1;
            tc_fence_before();
            seg_done(i);
            if (lane == 0) mbar_arrive(&sh->o_free);
        }
    }

    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// Merges the partials of the segment that starts in run blockIdx.y and goes on in later
// runs (at most one per run): one warp per row.  Bounded by three dependent loads (the cut,
// the maxima and sums, the outputs); those of the first parts are issued together.
constexpr int kTrCombineWarps = 4, kTrCombineAhead = 4;

template <int D>
__global__ void __launch_bounds__(kTrCombineWarps * 32) tree_combine_kernel(const TreeAttnParams p) {
    constexpr int E = D / 32;
    grid_dependency_wait();
    const int4 cut = p.cuts[blockIdx.y];   // {parts, sequence, key/value head, nodes}
    if (cut.x == 0) return;
    const int lane = threadIdx.x & 31, ri = blockIdx.x * kTrCombineWarps + (threadIdx.x >> 5);
    const int grp = blockIdx.y % p.groups, npt = kTrM / p.G;
    const int node = (ri & (kTrM - 1)) / p.G, hh = (ri & (kTrM - 1)) - node * p.G;
    const int t = (2 * grp + ri / kTrM) * npt + node, h = cut.z * p.G + hh;
    if (node >= npt || t >= cut.w) return;
    // Part 0 is partial 1 of its run, the others partial 0 of theirs.
    auto rec = [&](int s) {
        return p.part + (static_cast<size_t>((blockIdx.y + s * p.groups) * 2 + (s == 0 ? 1 : 0)) * p.part_rows + ri) *
                            (D + kTrRec);
    };
    float2 ahead[kTrCombineAhead][E / 2];
#pragma unroll
    for (int s = 0; s < kTrCombineAhead; ++s)
#pragma unroll
        for (int e = 0; e < E; e += 2)
            ahead[s][e / 2] = s < cut.x ? *reinterpret_cast<const float2*>(rec(s) + lane * E + e) : make_float2(0.f, 0.f);
    // Lane x holds the max and sum of parts x, x + 32, ... merged.  A part whose logits are all
    // NaN has a max of -inf and a sum of NaN, which the total keeps.
    float m = -INFINITY, l = 0.0f, m_own = -INFINITY;
    for (int s = lane; s < cut.x; s += 32) {
        const float2 ml = *reinterpret_cast<const float2*>(rec(s) + D);
        const float top = fmaxf(m, ml.x);
        const float a = m == -INFINITY ? 0.0f : ex2_approx(m - top);
        l = l * a + (ml.x == -INFINITY ? ml.y : ml.y * ex2_approx(ml.x - top));
        m = top;
        if (s == lane) m_own = ml.x;
    }
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (m != -INFINITY) l *= ex2_approx(m - M);   // else 0, or NaN
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float w_own = m_own == -INFINITY ? 0.0f : ex2_approx(m_own - M);
    float acc[E] = {};
#pragma unroll
    for (int s = 0; s < kTrCombineAhead; ++s) {
        const float a = __shfl_sync(0xffffffffu, w_own, s);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            acc[e] = fmaf(ahead[s][e / 2].x, a, acc[e]);
            acc[e + 1] = fmaf(ahead[s][e / 2].y, a, acc[e + 1]);
        }
    }
#pragma unroll 4
    for (int s = kTrCombineAhead; s < cut.x; ++s) {
        const float* x = rec(s);
        const float ms = x[D];
        const float a = ms == -INFINITY ? 0.0f : ex2_approx(ms - M);
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
        p.lse[(static_cast<size_t>(cut.y) * p.Hq + h) * p.T + t] = tree_lse(M, l);
}

template <int D>
cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, TreeAttnParams p,
                        cudaStream_t stream) {
    const TreeSmem sm = tree_smem(D, p.G, p.T);
    p.nk = sm.nk, p.nv = sm.nv, p.tab_bufs = sm.bufs;
    cudaError_t e =
        cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm.bytes);
    if (e != cudaSuccess) return e;
    const int ctas = p.runs * p.groups;
    tree_attn_kernel<D><<<ctas, kTrThreads, sm.bytes, stream>>>(tq, tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.whole) return e;   // nothing is cut
    const int rows = p.part_rows > kTrM ? p.part_rows : p.T * p.G;
    // The combine is brought up while the kernel before it runs, and waits for it on the device.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((rows + kTrCombineWarps - 1) / kTrCombineWarps, ctas);
    cfg.blockDim = dim3(kTrCombineWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<D>, p);
}

}  // namespace

// Key tiles of the longest sequence: a windowed one may start up to a box before its first key.
int tree_max_tiles(int T, int max_ctx, int window, int box_rows) {
    const long long prefix = window > 0 ? std::min<long long>(max_ctx, window - 2LL + box_rows) : max_ctx;
    return static_cast<int>((prefix + T + kTrN - 1) / kTrN);
}

TreeLaunch tree_launch_plan(int B, int T, int Hkv, int G, int max_ctx, int window, int d, int sms) {
    TreeLaunch x{};
    const int npt = kTrM / G, row_tiles = (T + npt - 1) / npt;
    x.groups = (row_tiles + 1) / 2;
    x.part_rows = row_tiles > 1 ? 2 * kTrM : kTrM;
    const long long tiles = static_cast<long long>(B) * Hkv * tree_max_tiles(T, max_ctx, window, kTrN);
    x.runs = static_cast<int>(std::min<long long>(std::max(1, sms / x.groups), tiles));
    const size_t ctas = static_cast<size_t>(x.runs) * x.groups;
    x.cut_bytes = (ctas * sizeof(int4) + 255) / 256 * 256;
    x.bytes = x.cut_bytes + ctas * 2 * x.part_rows * (d + kTrRec) * sizeof(float);
    return x;
}

// Whether runs take whole segments.  If all segments are as long as the longest may be,
// whole runs differ from an even share by the rounding of items / runs to whole segments;
// cutting costs partials and the combine kernel, worth about kTrCutTiles tiles.  Lengths are
// known on the device only, though: if one segment is long and the others short, the share
// shrinks and the run that holds the long one does not, so the longest possible segment is
// bounded too.  Cut against whole (us; 16 nodes, 4 key/value heads of 128, 148 runs):
//   longest (tiles)                    6            12           16           32           64
//   37 sequences of that length        23.0  19.5   34.2  30.2   42.1  37.8   69.3  64.7    110  107
//   lengths falling evenly to 0        28.7  24.5   47.2  34.3   53.1  44.5   70.7  54.3   95.1 88.4
//   one, the others of 100 rows        21.3  19.5   20.6  26.1   20.3  30.3   21.7  47.2   28.7 81.4
// and windows of 512 (5-6 tiles): one sequence 13.6 against 17.1, 8 sequences 23.0 against 18.4,
// 64 sequences 45.8 against 32.6.  A bound of 12 tiles makes the loss on the worst of these
// batches the smallest: 27% at 12 (one long segment), 30% at 32 (falling lengths, cut).
bool tree_whole_segments(int B, int Hkv, int runs, int max_tiles) {
    const long long items = static_cast<long long>(B) * Hkv;
    return max_tiles <= kTrWholeTiles &&
           (items + runs - 1) / runs * max_tiles <= (items * max_tiles + runs - 1) / runs + kTrCutTiles;
}

cudaError_t launch_tree_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const TreeAttnParams& p, int d, cudaStream_t stream) {
    return d == 128 ? launch_tree<128>(tq, tk, tv, p, stream) : launch_tree<64>(tq, tk, tv, p, stream);
}

}  // namespace relbias
