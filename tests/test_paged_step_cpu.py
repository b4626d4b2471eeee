"""The serving-step operators without a GPU: refusals of the C entry points and of the
binding, and the references' own pins."""
import numpy as np
import pytest
import torch

from attention_learned_relative_b200 import build, ops
from oracle import oracle as O
from paged_ref import mask_words, ref_page_plan, ref_tree_attn, ref_tree_plan

FAKE = 0x10000   # aligned, never dereferenced: every call below fails its checks first
OTHER = 0x20000
ARG, UNSUPPORTED = ops.RELBIAS_ERR_ARG, ops.RELBIAS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.lib()


def _page_plan(lib, **kw):
    a = dict(ctx=FAKE, new=FAKE, held=FAKE, held_out=OTHER, table=FAKE, ring=FAKE, state=FAKE, state_out=OTHER,
             granted=OTHER + 16, slots=OTHER + 32, B=2, T=4, page=16, max_pages=4, num_pages=9)
    a.update(kw)
    return lib.relbias_page_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(page=0), ARG), (dict(max_pages=0), ARG), (dict(num_pages=0), ARG),
    (dict(ctx=None), ARG), (dict(slots=None), ARG), (dict(ring=None), ARG), (dict(state=None), ARG),
    (dict(table=FAKE + 2), ARG), (dict(held_out=FAKE), ARG), (dict(state_out=FAKE), ARG),
    (dict(slots=OTHER, granted=OTHER + 64, new=OTHER + 64), ARG), (dict(slots=OTHER + 64, ctx=OTHER + 64), ARG),
    (dict(num_pages=1 << 28), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED),
    (dict(T=(65535 * 2048) + 1), UNSUPPORTED), (dict(B=(1 << 31) - 1), UNSUPPORTED),
])
def test_page_plan_refuses(lib, kw, code):
    assert _page_plan(lib, **kw) == code
    assert ops.last_error() != ""


def _tree_plan(lib, **kw):
    a = dict(parents=FAKE, lens=FAKE, depth=FAKE, mask=FAKE, B=2, T=4)
    a.update(kw)
    return lib.relbias_tree_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(T=129), UNSUPPORTED), (dict(parents=None), ARG),
    (dict(mask=FAKE + 1), ARG)])
def test_tree_plan_refuses(lib, kw, code):
    assert _tree_plan(lib, **kw) == code


def test_empty_calls_are_no_ops(lib):
    assert _tree_plan(lib, B=0, parents=None) == ops.RELBIAS_OK
    assert _tree_plan(lib, T=0) == ops.RELBIAS_OK
    assert _append(lib, ntok=0, k=None) == ops.RELBIAS_OK
    assert _compact(lib, A=0) == ops.RELBIAS_OK
    assert _compact(lib, B=0, path=None) == ops.RELBIAS_OK
    assert _tree(lib, B=0) == ops.RELBIAS_OK
    assert _tree(lib, T=0, q=None) == ops.RELBIAS_OK


def _append(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, slots=FAKE, qw=FAKE, kw=FAKE, q_out=FAKE, kp=FAKE, vp=FAKE, ntok=4, Hq=8, Hkv=2,
             d=64, qs=512, ks=128, vs=128, num_pages=4, page=16, eps=1e-6, dtype=ops.RELBIAS_BF16)
    a.update(kw)
    return lib.relbias_kv_append(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(ntok=-1), ARG), (dict(Hkv=0), ARG), (dict(Hq=0), ARG), (dict(d=96), UNSUPPORTED), (dict(dtype=3), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(k=None), ARG),
    (dict(q_out=None), ARG), (dict(q=None), ARG), (dict(k=FAKE + 8), ARG), (dict(vp=FAKE + 4), ARG),
    (dict(slots=FAKE + 2), ARG), (dict(ks=64), ARG), (dict(qs=500), ARG), (dict(vs=129), ARG), (dict(page=0), ARG),
    (dict(ntok=1 << 30), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED)])
def test_kv_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code


def _compact(lib, **kw):
    a = dict(kp=FAKE, vp=FAKE, table=FAKE, ctx=FAKE, path=FAKE, lens=FAKE, layers=1, B=2, A=4, num_pages=4, page=16,
             max_pages=2, Hkv=2, d=64, dtype=ops.RELBIAS_BF16)
    a.update(kw)
    return lib.relbias_kv_compact(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), ARG), (dict(A=-1), ARG), (dict(layers=-1), ARG), (dict(A=129), UNSUPPORTED), (dict(d=0), ARG),
    (dict(Hkv=1, d=4), UNSUPPORTED), (dict(dtype=9), ARG), (dict(path=None), ARG), (dict(kp=FAKE + 8), ARG),
    (dict(lens=FAKE + 1), ARG), (dict(B=65536), UNSUPPORTED), (dict(layers=32768), UNSUPPORTED)])
def test_kv_compact_refuses(lib, kw, code):
    assert _compact(lib, **kw) == code


def _tree(lib, **kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, ctx=FAKE, lens=FAKE, depth=FAKE, mask=FAKE, r=FAKE, w=FAKE, o=FAKE,
             lse=None, B=2, T=4, num_pages=8, page=32, max_pages=4, max_ctx=100, Hq=8, Hkv=2, d=128, window=0, R=16,
             scale=0.1, temp_n0=0, dtype=ops.RELBIAS_BF16, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return lib.relbias_attn_tree_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), ARG), (dict(Hq=7), ARG), (dict(R=-1), ARG), (dict(w=None), ARG), (dict(scale=0.0), ARG),
    (dict(dtype=5), ARG), (dict(dtype=ops.RELBIAS_FP32), UNSUPPORTED), (dict(T=129), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(Hq=34), UNSUPPORTED), (dict(page=24), ARG), (dict(max_ctx=129), ARG),
    (dict(max_ctx=-1), ARG), (dict(R=(1 << 30) + 1), UNSUPPORTED),
    (dict(max_ctx=(1 << 30) + 1, max_pages=1 << 26, num_pages=1 << 20), UNSUPPORTED), (dict(q=None), ARG), (dict(mask=None), ARG), (dict(r=None), ARG), (dict(ws=None), ARG), (dict(ws=FAKE + 8), ARG),
    (dict(o=FAKE + 8), ARG), (dict(table=FAKE + 2), ARG), (dict(lse=FAKE + 1), ARG), (dict(B=65536), UNSUPPORTED)])
def test_tree_attention_refuses(lib, kw, code):
    assert _tree(lib, **kw) == code


# ------------------------------------------------------------------------------ the binding


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


def test_binding_refuses_wrong_shapes_and_types():
    with pytest.raises(ValueError):      # lengths of another batch
        ops.page_plan(_i(3), _i(2), _i(3), _i(3, 4), _i(9), _i(2), 16, 4)
    with pytest.raises(ValueError):      # 64-bit lengths
        ops.page_plan(_i(3).long(), _i(3), _i(3), _i(3, 4), _i(9), _i(2), 16, 4)
    with pytest.raises(ValueError):
        ops.tree_plan(_i(2, 8), _i(3))
    with pytest.raises(ValueError):      # mask words of another T
        ops.tree_plan(_i(2, 40), _i(2), mask=_i(2, 40, 1))
    kv, pages = _t(4, 2, 64), _t(3, 16, 2, 64)
    with pytest.raises(ValueError):      # pages of another type
        ops.kv_append(kv, kv, _i(4), pages.bfloat16(), pages.bfloat16())
    with pytest.raises(ValueError):      # pages of other heads
        ops.kv_append(kv, kv, _i(4), _t(3, 16, 1, 64), _t(3, 16, 1, 64))
    with pytest.raises(ValueError):      # a weight of another size
        ops.kv_append(kv, kv, _i(4), pages, pages, k_weight=_t(32))
    with pytest.raises(ValueError):      # a query weight without queries
        ops.kv_append(kv, kv, _i(4), pages, pages, q_weight=_t(64))
    with pytest.raises(ValueError):      # heads that are not dense
        ops.kv_append(_t(4, 64, 2).transpose(1, 2), _t(4, 64, 2).transpose(1, 2), _i(4), pages, pages)
    q, p = _t(2, 4, 8, 64, dtype=torch.bfloat16), _t(6, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # depth of another T
        ops.attn_tree_paged(q, p, p, _i(2, 3), _i(2), _i(2), _i(2, 5), _i(2, 4, 1), _t(2, 4, 8), _t(8, 16), 0, 16, 10)
    with pytest.raises(ValueError):      # r of another shape
        ops.attn_tree_paged(q, p, p, _i(2, 3), _i(2), _i(2), _i(2, 4), _i(2, 4, 1), _t(2, 8, 4), _t(8, 16), 0, 16, 10)
    with pytest.raises(ValueError):      # tensors on the host
        ops.attn_tree_paged(q, p, p, _i(2, 3), _i(2), _i(2), _i(2, 4), _i(2, 4, 1), _t(2, 4, 8), _t(8, 16), 0, 16, 10)
    with pytest.raises(ValueError):
        ops.kv_compact(pages, _t(3, 16, 2, 32), _i(2, 3), _i(2), _i(2, 4), _i(2))
    with pytest.raises(ValueError):
        ops.kv_compact(pages, pages, _i(2, 3), _i(2), _i(2, 4), _i(3))


def test_token_strides_of_projection_slices():
    x = _t(3, 5, 640)
    q, k = x[..., :512].unflatten(2, (8, 64)), x[..., 512:].unflatten(2, (2, 64))
    assert ops._token_stride(q, "q", (3, 5)) == 640 and ops._token_stride(k, "k", (3, 5)) == 640
    assert ops._token_stride(q[:, :1], "q", (3, 1)) == 5 * 640
    assert ops._token_stride(q[:1, :1], "q", (1, 1)) == 512
    with pytest.raises(ValueError):
        ops._token_stride(q[:, :4], "q", (3, 4))        # batches are not evenly spaced any more


# ------------------------------------------------------------------------------ the references


def test_tree_reference_matches_the_oracle_on_each_path():
    """Attention of a node over the prefix and its ancestors is the oracle's decode step on
    the cache that holds the prefix and that path."""
    rng = np.random.default_rng(3)
    ctx, T, Hq, Hkv, d, W, R = 9, 7, 4, 2, 32, 6, 5
    parents = np.array([[-1, 0, 0, 1, 2, 4, -1]])
    depth, anc = ref_tree_plan(parents, [T])
    x = {n: torch.tensor(rng.standard_normal(s), dtype=torch.float32) for n, s in
         dict(q=(T, Hq, d), k=(ctx + T, Hkv, d), v=(ctx + T, Hkv, d), r=(T, Hq), w=(Hq, R)).items()}
    for window in (0, W):
        o, lse, _, _ = ref_tree_attn(x["q"], x["k"], x["v"], ctx, T, depth[0], anc[0], x["r"], x["w"], window, R, 0.2,
                                     temp_n0=4)
        for t in range(T):
            rows = list(range(ctx)) + [ctx + s for s in range(T) if anc[0, t, s]]
            oo, ll = O.attn_decode(x["q"][t][None], x["k"][rows][None], x["v"][rows][None], x["r"][t][None], x["w"],
                                   window, R, 0.2, temp_n0=4)
            assert np.abs(oo[0] - o[t]).max() < 1e-12 and np.abs(ll[0] - lse[t]).max() < 1e-12


def test_page_plan_reference_keeps_every_page_once():
    rng = np.random.default_rng(0)
    page, B, T, P, N = 4, 6, 9, 8, 30
    perm = rng.permutation(N)
    held = np.array([2, 0, 3, 1, 4, 1])
    table, at = np.full((B, P), -1), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    ring = np.roll(np.concatenate([perm[at:], np.full(at, -1)]), 25)
    ctx, new = np.array([5, 0, 0, 3, 9, 2]), np.array([9, 1, 0, 2, 3, 0])
    slots, granted, held2, table2, ring2, state2 = ref_page_plan(ctx, new, held, table, ring, [25, N - at], page, T)
    assert (granted == new).all() and held2.tolist() == [4, 1, 0, 2, 3, 1]
    owned = [table2[b, i] for b in range(B) for i in range(held2[b])]
    free = [ring2[(state2[0] + i) % N] for i in range(state2[1])]
    assert sorted(owned + free) == list(range(N))
    assert mask_words(np.eye(40, dtype=bool)[None])[0, 33].tolist() == [0, 2]
