// paged_abi.cu -- C entry points of the serving-step operators over a paged cache:
// argument checks and launches of paged_ops.cu and tree_sm100.cu.  Included by
// relbias_attn.cu, whose error reporting and tensor-map helpers it uses.
#include "relbias_attn.h"

namespace relbias {
namespace {

// Checks of a page pool and block table shared by the calls below.
int check_pool(int num_pages, int page_size, int max_pages) {
    if (num_pages < 1 || max_pages < 1 || page_size < 1)
        return fail(RELBIAS_ERR_ARG, "num_pages (%d), max_pages (%d) and page_size (%d) must be >= 1", num_pages,
                    max_pages, page_size);
    if (static_cast<long long>(num_pages) * page_size > INT32_MAX)
        return fail(RELBIAS_ERR_UNSUPPORTED, "num_pages * page_size (%lld) must stay below 2^31",
                    static_cast<long long>(num_pages) * page_size);
    if (static_cast<long long>(max_pages) * page_size > INT32_MAX)
        return fail(RELBIAS_ERR_UNSUPPORTED, "max_pages * page_size (%lld) must stay below 2^31",
                    static_cast<long long>(max_pages) * page_size);
    return RELBIAS_OK;
}

// x / d = x * mul >> shift for 0 <= x < 2^31: with s = ceil(log2 d), mul = ceil(2^(31 + s) / d) is
// above 2^(31 + s) / d by less than 1, so x * mul / 2^(31 + s) is above x / d by less than
// 2^31 / 2^(31 + s) <= 1 / d and does not reach the next whole number.  mul < 2^33.
void invariant_division(int d, uint64_t& mul, int& shift) {
    int s = 0;
    while ((1LL << s) < d) ++s;
    shift = 31 + s;
    mul = ((1ull << shift) + d - 1) / d;
}

template <typename... P>
bool any_null(P... p) {
    return (... || (p == nullptr));
}
template <typename... P>
bool all_aligned4(P... p) {
    return (... && aligned4(p));
}

}  // namespace
}  // namespace relbias

extern "C" int relbias_page_plan(const int* ctx_lens, const int* new_lens, const int* num_blocks, int* num_blocks_out,
                                 int* block_table, int* free_ring, const int* ring_state, int* ring_state_out,
                                 int* granted, int* slots, int B, int T, int page_size, int max_pages, int num_pages,
                                 void* stream) {
    t_err.clear();
    if (B < 0 || T < 0) return fail(RELBIAS_ERR_ARG, "B (%d) and T (%d) must be >= 0", B, T);
    int rc = check_pool(num_pages, page_size, max_pages);
    if (rc != RELBIAS_OK) return rc;
    if (B == INT32_MAX) return fail(RELBIAS_ERR_UNSUPPORTED, "too many requests (%d)", B);
    if (static_cast<long long>(T) > 65535LL * 2048)
        return fail(RELBIAS_ERR_UNSUPPORTED, "T (%d) is past the slot map's limit of 65535 * 2048 rows", T);
    if (any_null(ring_state, ring_state_out, free_ring) ||
        (B > 0 && (any_null(ctx_lens, new_lens, num_blocks, num_blocks_out, block_table, granted) ||
                   (T > 0 && slots == nullptr))))
        return fail(RELBIAS_ERR_ARG, "no pointer argument may be null");
    if (!all_aligned4(ctx_lens, new_lens, num_blocks, num_blocks_out, block_table, free_ring, ring_state,
                      ring_state_out, granted, slots))
        return fail(RELBIAS_ERR_ARG, "all arrays must be 4-byte aligned");
    // Every block reads the inputs of all requests before its own: no output may be one of them.
    for (const void* out : {static_cast<const void*>(ring_state_out), static_cast<const void*>(num_blocks_out),
                            static_cast<const void*>(granted), static_cast<const void*>(slots)})
        for (const void* in : {static_cast<const void*>(ring_state), static_cast<const void*>(num_blocks),
                               static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens)})
            if (out != nullptr && out == in)
                return fail(RELBIAS_ERR_ARG, "num_blocks_out, ring_state_out, granted and slots must not be inputs");
    PagePlanParams p{};
    p.ctx_lens = ctx_lens;
    p.new_lens = new_lens;
    p.num_blocks = num_blocks;
    p.num_blocks_out = num_blocks_out;
    p.block_table = block_table;
    p.free_ring = free_ring;
    p.ring_state = ring_state;
    p.ring_state_out = ring_state_out;
    p.granted = granted;
    p.slots = slots;
    p.B = B;
    p.T = T;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    const cudaError_t e = launch_page_plan(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RELBIAS_OK : cuda_fail(e, "page plan launch");
}

extern "C" int relbias_tree_plan(const int* parents, const int* tree_lens, int* depth, int* mask, int B, int T,
                                 void* stream) {
    t_err.clear();
    if (B < 0 || T < 0) return fail(RELBIAS_ERR_ARG, "B (%d) and T (%d) must be >= 0", B, T);
    if (T > kMaxTree) return fail(RELBIAS_ERR_UNSUPPORTED, "trees have at most %d nodes, got T = %d", kMaxTree, T);
    if (B == 0 || T == 0) return RELBIAS_OK;
    if (any_null(parents, tree_lens, depth, mask)) return fail(RELBIAS_ERR_ARG, "no pointer argument may be null");
    if (!all_aligned4(parents, tree_lens, depth, mask))
        return fail(RELBIAS_ERR_ARG, "all arrays must be 4-byte aligned");
    TreePlanParams p{parents, tree_lens, depth, mask, B, T};
    const cudaError_t e = launch_tree_plan(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RELBIAS_OK : cuda_fail(e, "tree plan launch");
}

extern "C" int relbias_kv_append(const void* q, const void* k, const void* v, const int* slots, const float* q_weight,
                                 const float* k_weight, void* q_out, void* k_pages, void* v_pages, int ntok, int Hq,
                                 int Hkv, int d, long long q_stride, long long k_stride, long long v_stride,
                                 int num_pages, int page_size, float eps, int dtype, void* stream) {
    t_err.clear();
    if (ntok < 0) return fail(RELBIAS_ERR_ARG, "ntok (%d) must be >= 0", ntok);
    if (Hkv < 1 || Hq < 0) return fail(RELBIAS_ERR_ARG, "Hkv (%d) must be >= 1 and Hq (%d) >= 0", Hkv, Hq);
    int rc = check_pool(num_pages, page_size, 1);
    if (rc != RELBIAS_OK) return rc;
    if (dtype != RELBIAS_BF16 && dtype != RELBIAS_FP32) return fail(RELBIAS_ERR_ARG, "unknown dtype %d", dtype);
    if (d != 32 && d != 64 && d != 128 && d != 256)
        return fail(RELBIAS_ERR_UNSUPPORTED, "the cache write supports d in {32, 64, 128, 256}, got %d", d);
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(RELBIAS_ERR_ARG, "eps (%g) must be finite and >= 0", static_cast<double>(eps));
    const bool with_q = q != nullptr;
    if (with_q && Hq < 1) return fail(RELBIAS_ERR_ARG, "q needs Hq >= 1");
    if (ntok == 0) return RELBIAS_OK;
    if (any_null(k, v, slots, k_pages, v_pages) || with_q != (q_out != nullptr))
        return fail(RELBIAS_ERR_ARG, "k, v, slots and the pages must not be null, and q and q_out go together");
    const int esz = dtype == RELBIAS_BF16 ? 2 : 4;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(q) ||
        !aligned16(q_out) || !all_aligned4(slots, q_weight, k_weight))
        return fail(RELBIAS_ERR_ARG, "q, k, v, q_out and the pages must be 16-byte aligned, the other arrays 4-byte");
    const long long kv_row = static_cast<long long>(Hkv) * d, q_row = static_cast<long long>(Hq) * d;
    if (k_stride < kv_row || v_stride < kv_row || (with_q && q_stride < q_row) || k_stride * esz % 16 != 0 ||
        v_stride * esz % 16 != 0 || (with_q && q_stride * esz % 16 != 0))
        return fail(RELBIAS_ERR_ARG, "token strides must cover a token's heads and be multiples of 16 bytes");
    const int heads_q = with_q ? Hq : 0;
    if (static_cast<long long>(ntok) * (heads_q + 2LL * Hkv) > INT32_MAX)
        return fail(RELBIAS_ERR_UNSUPPORTED, "ntok * (Hq + 2 Hkv) must stay below 2^31");
    KvAppendParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.q_out = q_out;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.ntok = ntok;
    p.heads_q = heads_q;
    p.Hkv = Hkv;
    invariant_division(heads_q + 2 * Hkv, p.heads_mul, p.heads_shift);
    p.num_slots = num_pages * page_size;
    p.eps = eps;
    DeviceInfo dev;
    if ((rc = device_info(dev)) != RELBIAS_OK) return rc;
    const cudaError_t e = launch_kv_append(p, dtype == RELBIAS_BF16, d, dev.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RELBIAS_OK : cuda_fail(e, "cache write launch");
}

extern "C" int relbias_kv_compact(void* k_pages, void* v_pages, const int* block_table, const int* ctx_lens,
                                  const int* path, const int* path_lens, int layers, int B, int A, int num_pages,
                                  int page_size, int max_pages, int Hkv, int d, int dtype, void* stream) {
    t_err.clear();
    if (B < 0 || A < 0 || layers < 0)
        return fail(RELBIAS_ERR_ARG, "B (%d), A (%d) and layers (%d) must be >= 0", B, A, layers);
    if (A > kMaxTree) return fail(RELBIAS_ERR_UNSUPPORTED, "paths have at most %d nodes, got A = %d", kMaxTree, A);
    int rc = check_pool(num_pages, page_size, max_pages);
    if (rc != RELBIAS_OK) return rc;
    if (Hkv < 1 || d < 1) return fail(RELBIAS_ERR_ARG, "Hkv (%d) and d (%d) must be >= 1", Hkv, d);
    if (dtype != RELBIAS_BF16 && dtype != RELBIAS_FP32) return fail(RELBIAS_ERR_ARG, "unknown dtype %d", dtype);
    const long long row_bytes = static_cast<long long>(Hkv) * d * (dtype == RELBIAS_BF16 ? 2 : 4);
    if (row_bytes % 16 != 0)
        return fail(RELBIAS_ERR_UNSUPPORTED, "a cache row (%lld bytes) must be a multiple of 16 bytes", row_bytes);
    if (row_bytes / 16 > INT32_MAX) return fail(RELBIAS_ERR_UNSUPPORTED, "a cache row of %lld bytes", row_bytes);
    if (B > 65535 || 2LL * layers > 65535)
        return fail(RELBIAS_ERR_UNSUPPORTED, "at most 65535 requests and 32767 layers, got %d and %d", B, layers);
    if (B == 0 || A == 0 || layers == 0) return RELBIAS_OK;
    if (any_null(k_pages, v_pages) || any_null(block_table, ctx_lens, path, path_lens))
        return fail(RELBIAS_ERR_ARG, "no pointer argument may be null");
    if (!aligned16(k_pages) || !aligned16(v_pages) || !all_aligned4(block_table, ctx_lens, path, path_lens))
        return fail(RELBIAS_ERR_ARG, "the pages must be 16-byte aligned, the other arrays 4-byte");
    KvCompactParams p{};
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.block_table = block_table;
    p.ctx_lens = ctx_lens;
    p.path = path;
    p.path_lens = path_lens;
    p.B = B;
    p.A = A;
    p.layers = layers;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.row_vecs = static_cast<int>(row_bytes / 16);
    const cudaError_t e = launch_kv_compact(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RELBIAS_OK : cuda_fail(e, "cache compaction launch");
}

namespace relbias {
namespace {
int check_tree_shape(int B, int T, int Hq, int Hkv, int max_ctx_len, int d) {
    if (T > kMaxTree) return fail(RELBIAS_ERR_UNSUPPORTED, "trees have at most %d nodes, got T = %d", kMaxTree, T);
    if (max_ctx_len < 0) return fail(RELBIAS_ERR_ARG, "max_ctx_len (%d) must be >= 0", max_ctx_len);
    if (max_ctx_len > 1 << 30) return fail(RELBIAS_ERR_UNSUPPORTED, "max_ctx_len (%d) is past 2^30", max_ctx_len);
    if (d != 64 && d != 128)
        return fail(RELBIAS_ERR_UNSUPPORTED, "the tree attention supports d in {64, 128}, got %d", d);
    if (Hq / Hkv > 16)
        return fail(RELBIAS_ERR_UNSUPPORTED, "the tree attention supports up to 16 query heads per key/value head");
    if (B > 65535) return fail(RELBIAS_ERR_UNSUPPORTED, "at most 65535 sequences, got %d", B);
    if (Hkv > 4096) return fail(RELBIAS_ERR_UNSUPPORTED, "at most 4096 key/value heads, got %d", Hkv);
    return RELBIAS_OK;
}
}  // namespace
}  // namespace relbias

extern "C" size_t relbias_attn_tree_paged_workspace_size(int B, int T, int Hq, int Hkv, int max_ctx_len, int d,
                                                         int window) {
    if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
    if (check_tree_shape(B, T, Hq, Hkv, max_ctx_len, d) != RELBIAS_OK) return 0;
    DeviceInfo dev;
    if (device_info(dev) != RELBIAS_OK) return 0;
    return tree_launch_plan(B, T, Hkv, Hq / Hkv, max_ctx_len, std::max(window, 0), d, dev.sms).bytes;
}

extern "C" int relbias_attn_tree_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                                       const int* ctx_lens, const int* tree_lens, const int* depth, const int* mask,
                                       const float* r, const float* w, void* o, float* lse, int B, int T,
                                       int num_pages, int page_size, int max_pages, int max_ctx_len, int Hq, int Hkv,
                                       int d, int window, int R, float scale, int temp_n0, int dtype, void* workspace,
                                       size_t ws_bytes, void* stream) {
    t_err.clear();
    int rc = check_common(B, T, Hq, Hkv, d, R, scale, w);
    if (rc != RELBIAS_OK) return rc;
    if (dtype != RELBIAS_BF16 && dtype != RELBIAS_FP32) return fail(RELBIAS_ERR_ARG, "unknown dtype %d", dtype);
    if ((rc = check_pool(num_pages, page_size, max_pages)) != RELBIAS_OK) return rc;
    if (page_size % 16 != 0) return fail(RELBIAS_ERR_ARG, "page_size (%d) must be a multiple of 16", page_size);
    if (max_ctx_len < 0 || static_cast<long long>(max_ctx_len) > static_cast<long long>(max_pages) * page_size)
        return fail(RELBIAS_ERR_ARG, "max_ctx_len (%d) must be in [0, max_pages * page_size]", max_ctx_len);
    if (dtype != RELBIAS_BF16) return fail(RELBIAS_ERR_UNSUPPORTED, "the tree attention is bf16 only");
    if (R > 1 << 30) return fail(RELBIAS_ERR_UNSUPPORTED, "R (%d) is past 2^30", R);
    if ((rc = check_tree_shape(B, T, Hq, Hkv, max_ctx_len, d)) != RELBIAS_OK) return rc;
    if (B == 0 || T == 0) return RELBIAS_OK;
    if (any_null(q, k_pages, v_pages, static_cast<const void*>(o), static_cast<const void*>(workspace)) ||
        any_null(block_table, ctx_lens, tree_lens, depth, mask) || r == nullptr)
        return fail(RELBIAS_ERR_ARG, "q, the pages, block_table, ctx_lens, tree_lens, depth, mask, r, o and workspace "
                                     "must not be null");
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned16(workspace))
        return fail(RELBIAS_ERR_ARG, "q, the pages, o and workspace must be 16-byte aligned");
    if (!all_aligned4(block_table, ctx_lens, tree_lens, depth, mask) || !aligned4(r) || !aligned4(lse))
        return fail(RELBIAS_ERR_ARG, "block_table, ctx_lens, tree_lens, depth, mask, r and lse must be 4-byte aligned");
    DeviceInfo dev;
    if ((rc = device_info(dev)) != RELBIAS_OK) return rc;
    if (dev.major != 10 || dev.minor != 0)
        return fail(RELBIAS_ERR_UNSUPPORTED, "the tree attention needs compute capability 10.0 (sm_100a), found %d.%d",
                    dev.major, dev.minor);
    TreeAttnParams p{};
    p.block_table = block_table;
    p.ctx_lens = ctx_lens;
    p.tree_lens = tree_lens;
    p.depth = depth;
    p.mask = mask;
    p.r = r;
    p.w = w;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.words = (T + 31) / 32;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.max_ctx = max_ctx_len;
    p.window = window > 0 ? window : 0;
    p.R = R;
    p.scale_log2 = scale * kLog2e;
    p.inv_scale = 1.0f / scale;
    p.temp_n0 = temp_n0 > 1 ? temp_n0 : 0;
    p.inv_log_n0 = temp_n0 > 1 ? static_cast<float>(1.0 / std::log(static_cast<double>(temp_n0))) : 0.0f;
    p.box_rows = std::min(128, page_size & -page_size);
    invariant_division(page_size, p.page_mul, p.page_shift);
    p.w_bulk = R % 4 == 0 && aligned16(w);
    if (static_cast<long long>(B) * Hkv * tree_max_tiles(T, max_ctx_len, p.window, 128) > INT32_MAX)
        return fail(RELBIAS_ERR_UNSUPPORTED, "too many key tiles (%d sequences, %d heads)", B, Hkv);
    const TreeLaunch plan = tree_launch_plan(B, T, Hkv, p.G, max_ctx_len, p.window, d, dev.sms);
    if (ws_bytes < plan.bytes)
        return fail(RELBIAS_ERR_ARG, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes,
                    plan.bytes);
    p.groups = plan.groups;
    p.runs = plan.runs;
    p.part_rows = plan.part_rows;
    p.max_tiles = tree_max_tiles(T, max_ctx_len, p.window, p.box_rows);
    p.whole = tree_whole_segments(B, Hkv, p.runs, p.max_tiles);
    p.cuts = static_cast<int4*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.cut_bytes);
    CUtensorMap tq, tk, tv;
    if ((rc = make_map(&tq, q, B, T, Hq, d, 128 / p.G, 0, p.G)) != RELBIAS_OK) return rc;
    if ((rc = make_map(&tk, k_pages, num_pages, page_size, Hkv, d, p.box_rows)) != RELBIAS_OK) return rc;
    if ((rc = make_map(&tv, v_pages, num_pages, page_size, Hkv, d, p.box_rows)) != RELBIAS_OK) return rc;
    const cudaError_t e = launch_tree_attn(tq, tk, tv, p, d, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RELBIAS_OK : cuda_fail(e, "tree attention launch");
}
