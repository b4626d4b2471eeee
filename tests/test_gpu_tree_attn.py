"""Attention of drafted trees over a paged cache, against a plain reference in 64 bits.

Rows that no node sees by position (unused pages, rows past the tree and before the window)
hold NaN, so that a stray read shows."""
import math

import numpy as np
import pytest
import torch

from attention_learned_relative_b200 import ops
from paged_ref import assert_tree_close, mask_words, ref_tree_attn, ref_tree_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    ops.device_status(reset=True)
    yield
    assert ops.device_status(reset=True) == 0, "a kernel reported a bad status"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(ctxs, lens, T, Hq, Hkv, d, page, window, R, chain=0.5, seed=0, anc=None, qk=1.0, spare=3):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    B = len(ctxs)
    parents = np.floor(rng.random((B, T)) * np.maximum(np.arange(T), 1)).astype(np.int64)
    parents = np.where(rng.random((B, T)) < chain, np.arange(T) - 1, parents)
    parents[:, 0] = -1
    depth, tree = ref_tree_plan(parents, [T] * B)
    anc = tree if anc is None else anc
    normal = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    need = [-(-(c + n) // page) for c, n in zip(ctxs, lens)]
    P, N = max(1, max(need)), sum(need) + spare
    perm, table, at = rng.permutation(N), np.full((B, P), -7, np.int64), 0
    k_pages = torch.full((N, page, Hkv, d), float("nan"), dtype=torch.bfloat16)
    v_pages = torch.full_like(k_pages, float("nan"))
    ks, vs = [], []
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        rows = ctxs[b] + lens[b]
        k, v = (normal(rows, Hkv, d) * qk).bfloat16(), normal(rows, Hkv, d).bfloat16()
        first = max(0, ctxs[b] - window + 1) if window > 0 else 0
        j = np.arange(first, rows)
        slot = torch.as_tensor(table[b, j // page] * page + j % page)
        k_pages.view(-1, Hkv, d)[slot] = k[first:]
        v_pages.view(-1, Hkv, d)[slot] = v[first:]
        ks.append(k)
        vs.append(v)
    return dict(ctxs=ctxs, lens=lens, window=window, R=R, depth=depth, anc=anc, ks=ks, vs=vs,
                q=(normal(B, T, Hq, d) * qk).bfloat16().cuda(), r=normal(B, T, Hq).cuda(),
                w=(normal(Hq, R) * 0.5).cuda() if R else None, k_pages=k_pages.cuda(), v_pages=v_pages.cuda(),
                table=_i32(table))


def call(x, scale, temp_n0=0, max_ctx=None, **kw):
    B, T, Hq, d = x["q"].shape
    out = torch.full_like(x["q"], 9.0)
    lse = torch.full((B, Hq, T), 9.0, device="cuda")
    ops.attn_tree_paged(x["q"], x["k_pages"], x["v_pages"], x["table"], _i32(x["ctxs"]), _i32(x["lens"]),
                        _i32(x["depth"]), torch.as_tensor(mask_words(x["anc"])).cuda(), x["r"], x["w"], x["window"],
                        x["R"], max(x["ctxs"]) if max_ctx is None else max_ctx, scale=scale, out=out, lse=lse,
                        temp_n0=temp_n0, **kw)
    return out, lse


def check(x, scale=None, temp_n0=0, max_ctx=None, what=""):
    B, T, Hq, d = x["q"].shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = call(x, scale, temp_n0, max_ctx)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (c, n) in enumerate(zip(x["ctxs"], x["lens"])):
        assert (o[b, n:] == 9).all() and (l[b, :, n:] == 9).all(), "rows past the tree were written"
        ref = ref_tree_attn(x["q"][b].double().cpu(), x["ks"][b].double(), x["vs"][b].double(), c, n, x["depth"][b],
                            x["anc"][b], x["r"][b].double().cpu(), x["w"].double().cpu() if x["R"] else None,
                            x["window"], x["R"], scale, temp_n0)
        assert_tree_close(o[b, :n], l[b, :, :n].T, ref, d, "%s sequence %d" % (what, b))
    return out, lse


@pytest.mark.parametrize("ctxs,lens,T,Hq,Hkv,d,page,window,R,temp_n0", [
    ([1], [1], 1, 1, 1, 64, 16, 0, 4, 0),                                  # one key of each kind
    ([0, 0, 5], [1, 4, 0], 4, 8, 2, 64, 16, 0, 16, 0),                     # no prefix; no tree
    ([300, 17, 128], [4, 3, 1], 4, 8, 2, 64, 16, 64, 64, 0),
    ([127, 128, 129, 255], [16, 15, 14, 1], 16, 8, 1, 128, 32, 0, 64, 0),  # the tree around a tile's edge
    ([1000, 90, 511], [33, 32, 31], 33, 8, 1, 128, 48, 0, 300, 0),         # pages that end inside a tile
    ([700, 600], [64, 61], 64, 32, 4, 128, 64, 512, 512, 0),               # the local layer
    ([2000, 100], [128, 127], 128, 8, 1, 64, 256, 0, 1024, 500),           # the largest tree, temperature
    ([333], [20], 20, 6, 1, 128, 16, 3, 7, 0),                             # a window shorter than the tree is deep
    ([333, 2], [20, 20], 20, 16, 1, 64, 96, 1, 1, 0),                      # each node sees itself alone
    ([50, 513], [7, 9], 9, 3, 1, 64, 80, 0, 0, 0),                         # no bias, three heads a group
    ([260], [50], 50, 5, 1, 128, 16, 100, 2048, 10),                       # five heads a group
    ([400, 1], [40, 39], 40, 4, 4, 128, 128, 0, 200, 0),                   # a group of one head
    ([5000, 4999, 3], [8, 8, 8], 8, 32, 2, 128, 16, 0, 5000, 1000),        # bias over the whole prefix
    ([900, 20], [128, 128], 128, 16, 1, 128, 32, 200, 200, 0),
])
def test_tree_attention(ctxs, lens, T, Hq, Hkv, d, page, window, R, temp_n0):
    for chain in (0.0, 0.5, 1.0):
        x = make(ctxs, lens, T, Hq, Hkv, d, page, window, R, chain=chain, seed=sum(ctxs) + T)
        check(x, temp_n0=temp_n0, what="chain %.1f" % chain)


def test_short_sequences_under_a_long_bound():
    """max_ctx_len plans the key splits; shorter sequences leave most of them empty."""
    x = make([40, 3, 1300, 0], [6, 6, 5, 6], 6, 8, 2, 128, 64, 0, 64, seed=5)
    x["table"] = torch.nn.functional.pad(x["table"], (0, 4000), value=-7)
    check(x, max_ctx=200000)


def test_nodes_whose_mask_leaves_nothing():
    """Masks of any kind: empty rows, one node only, later nodes and siblings at the same depth."""
    rng = np.random.default_rng(8)
    B, T = 4, 40
    anc = rng.random((B, T, T)) < 0.3
    anc[:, 5] = False
    anc[0] = False
    x = make([0, 0, 200, 140], [40, 33, 40, 17], T, 8, 2, 64, 16, 0, 30, seed=8, anc=anc)
    _, lse = check(x)
    assert torch.isinf(lse[0]).all()
    x = make([0, 3, 200, 140], [40, 33, 40, 17], T, 8, 2, 128, 16, 5, 30, seed=9, anc=anc)
    check(x)


def test_large_logits():
    """Logits of a few hundred: the running maximum moves by more than any rescaling threshold."""
    x = make([700, 3000], [30, 16], 30, 8, 1, 128, 32, 0, 64, seed=4, qk=4.0)
    check(x, scale=0.5)
    check(x, scale=1e-4)


def test_masked_keys_may_hold_infinities():
    """Keys of nodes off the path may be infinite or NaN: only the values have to be finite."""
    x = make([100], [12], 12, 8, 2, 64, 16, 0, 16, chain=0.0, seed=2)
    leaf = 11   # the last node: only it sees its own key
    slot = 100 + leaf
    x["k_pages"].view(-1, 2, 64)[int(x["table"][0, slot // 16]) * 16 + slot % 16] = float("nan")
    out, lse = call(x, 0.125)
    for t in range(11):
        assert torch.isfinite(out[0, t].float()).all() and torch.isfinite(lse[0, :, t]).all()
    x["lens"], x["ks"], x["vs"] = [11], [x["ks"][0][:111]], [x["vs"][0][:111]]
    x["v_pages"].view(-1, 2, 64)[int(x["table"][0, slot // 16]) * 16 + slot % 16] = float("nan")
    check(x, scale=0.125)   # the row is past the tree now


def test_a_tree_of_one_node_is_the_paged_decode_step():
    ctxs, Hq, Hkv, d, page, R = [1500, 64, 31], 16, 2, 128, 64, 256
    x = make(ctxs, [1, 1, 1], 1, Hq, Hkv, d, page, 0, R, seed=12)
    out, lse = call(x, 0.09, temp_n0=100)
    lse2 = torch.empty(3, Hq, device="cuda")
    o2 = ops.attn_decode_paged(x["q"][:, 0].contiguous(), x["k_pages"], x["v_pages"], x["table"],
                               _i32([c + 1 for c in ctxs]), x["r"][:, 0].contiguous(), x["w"], 0, R, 1501, 0.09,
                               lse=lse2, temp_n0=100)
    # Two kernels, each within one rounding of weights and output of the exact value (|v| <= 5).
    assert (out[:, 0].float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * 2 * 5
    assert (lse[:, :, 0] - lse2).abs().max() <= 1e-3


def test_a_chain_is_the_paged_chunk():
    ctxs, T, Hq, Hkv, d, page, W, R = [640, 65], 70, 8, 2, 128, 64, 300, 128
    x = make(ctxs, [70, 64], T, Hq, Hkv, d, page, W, R, chain=1.0, seed=13)
    pool_k, pool_v = torch.nan_to_num(x["k_pages"]), torch.nan_to_num(x["v_pages"])
    out, lse = call(x, 0.09)
    lse2 = torch.full_like(lse, 9.0)
    o2 = ops.attn_fwd_chunk_paged(x["q"], pool_k, pool_v, x["table"], _i32(ctxs), _i32([70, 64]), x["r"], x["w"], W, R,
                                  0.09, out=torch.full_like(out, 9.0), lse=lse2)
    assert (out.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * 2 * 5
    assert (lse - lse2).abs().max() <= 1e-3


def test_repeatable_and_independent_of_the_batch():
    x = make([900, 200, 31], [16, 9, 16], 16, 32, 4, 128, 32, 0, 128, seed=3)
    a, la = call(x, 0.09)
    b, lb = call(x, 0.09)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_lengths_depths_and_pages_are_reported():
    x = make([100, 64], [8, 8], 8, 8, 2, 64, 16, 0, 16, seed=6)
    good, _ = call(x, 0.125)
    for key, value, status in [("ctxs", [101, 64], 2), ("ctxs", [-1, 64], 2), ("lens", [9, 8], 2), ("lens", [-1, 8], 2)]:
        y = dict(x, **{key: value})
        out, _ = call(y, 0.125, max_ctx=100)
        assert ops.device_status(reset=True) == status
        assert torch.equal(out[1], good[1])
    deep = x["depth"].copy()
    deep[0, 3] = 8
    out, _ = call(dict(x, depth=deep), 0.125)
    assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_TREE
    assert torch.equal(out[1], good[1])
    table = x["table"].clone()
    table[0, 1], table[0, 2] = -1, x["k_pages"].shape[0]
    out, _ = call(dict(x, table=table), 0.125)
    assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_LENGTH
    assert torch.equal(out[1], good[1]) and torch.isfinite(out[0].float()).all()


def test_workspace_and_another_stream():
    x = make([900, 200], [16, 9], 16, 32, 4, 128, 32, 0, 128, seed=7)
    want, lse = call(x, 0.09)
    size = ops.tree_workspace_size(2, 16, 32, 4, 900, 128, 0)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = (x["q"], x["k_pages"], x["v_pages"], x["table"], _i32(x["ctxs"]), _i32(x["lens"]), _i32(x["depth"]),
            torch.as_tensor(mask_words(x["anc"])).cuda(), x["r"], x["w"], 0, 128, 900)
    torch.cuda.synchronize()
    out = torch.full_like(x["q"], 9.0)
    ops.attn_tree_paged(*args, scale=0.09, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ops.RelbiasError):
        ops.attn_tree_paged(*args, scale=0.09, out=out, workspace=ws[:8])


def _ragged(B, T, top, seed):
    rng = np.random.default_rng(seed)
    ctxs = rng.integers(0, top + 1, B)
    lens = rng.integers(0, T + 1, B)
    lens[rng.random(B) < 0.2] = 0
    ctxs[rng.random(B) < 0.2] = 0
    return [int(c) for c in ctxs], [int(n) for n in lens]


@pytest.mark.parametrize("B,T,Hq,Hkv,d,page,window,bound", [
    (70, 20, 16, 1, 64, 16, 0, 0),         # three row tiles a head: CTAs for two pairs of them
    (70, 20, 16, 1, 64, 16, 0, 100000),    # segments are cut: the bound on the prefixes is far above them
    (33, 5, 8, 2, 128, 32, 100, 0),
    (100, 3, 8, 4, 64, 48, 0, 60000),
    (40, 40, 16, 2, 128, 16, 50, 0),       # five row tiles: three pairs, the last of one
    (40, 40, 16, 2, 128, 16, 0, 50000),
])
def test_large_ragged_batches(B, T, Hq, Hkv, d, page, window, bound):
    """More sequences than a warp has lanes, some without a prefix, a tree, or rows of every
    pair of row tiles; runs of whole and of cut segments."""
    ctxs, lens = _ragged(B, T, 400, seed=B + T)
    x = make(ctxs, lens, T, Hq, Hkv, d, page, window, 64, seed=B)
    if bound:
        x["table"] = torch.nn.functional.pad(x["table"], (0, bound // page), value=-7)
    check(x, max_ctx=bound or None, what="ragged")


@pytest.mark.parametrize("ctxs,lens,T,G,window,R", [
    ([700, 1500, 30], [8, 7, 8], 8, 16, 0, 999),       # one row tile, its key tiles shared by the slots
    ([1500, 1200, 900], [8, 8, 8], 8, 14, 700, 1000),
    ([700, 300, 1400], [5, 128, 9], 128, 16, 0, 1024),  # one row tile among sequences with many
])
def test_groups_whose_bias_slices_have_one_buffer(ctxs, lens, T, G, window, R):
    check(make(ctxs, lens, T, G, 1, 128, 16, window, R, seed=G + T))


def test_no_sequence_has_a_node():
    x = make([30, 0, 5000], [0, 0, 0], 8, 8, 2, 64, 16, 0, 16, seed=1)
    check(x)


def test_a_window_of_any_size():
    x = make([700, 40], [9, 16], 16, 8, 2, 128, 16, 0, 64, seed=5)
    want, _ = call(x, 0.09)
    x["window"] = 2 ** 31 - 1
    assert torch.equal(call(x, 0.09)[0], want)


@pytest.mark.parametrize("R", [1, 2, 3, 5, 127, 130, 301])
def test_tables_that_bulk_copies_cannot_take(R):
    """Tables whose rows do not start on 16-byte boundaries, by R or by their address."""
    x = make([300, 77], [9, 16], 16, 8, 2, 128, 16, 0, R, seed=R)
    check(x)
    buf = torch.zeros(8 * R + 1, device="cuda")
    buf[1:] = x["w"].view(-1)
    x["w"] = buf[1:].view(8, R)
    check(x)


def test_a_table_that_starts_off_a_16_byte_boundary():
    x = make([300, 77], [9, 16], 16, 8, 2, 128, 16, 0, 64, seed=3)
    buf = torch.zeros(8 * 64 + 1, device="cuda")
    buf[1:] = x["w"].view(-1)
    x["w"] = buf[1:].view(8, 64)
    check(x)


def test_outputs_and_workspace_stay_in_bounds():
    """Output, log-sum-exp and workspace sit between bands that must survive."""
    x = make([900, 200, 3000], [16, 9, 3], 16, 16, 2, 128, 32, 0, 128, seed=7)
    want, want_lse = call(x, 0.09)
    size = ops.tree_workspace_size(3, 16, 16, 2, 3000, 128, 0)
    band = 4096
    raw = torch.full((size + 2 * band,), 171, dtype=torch.uint8, device="cuda")
    o_raw = torch.full((want.numel() + 2 * band,), 9.0, dtype=torch.bfloat16, device="cuda")
    l_raw = torch.full((want_lse.numel() + 2 * band,), 9.0, device="cuda")
    out = o_raw[band:-band].view_as(want)
    lse = l_raw[band:-band].view_as(want_lse)
    ops.attn_tree_paged(x["q"], x["k_pages"], x["v_pages"], x["table"], _i32(x["ctxs"]), _i32(x["lens"]),
                        _i32(x["depth"]), torch.as_tensor(mask_words(x["anc"])).cuda(), x["r"], x["w"], 0, 128, 3000,
                        scale=0.09, out=out, lse=lse, workspace=raw[band:-band])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (raw[:band] == 171).all() and (raw[-band:] == 171).all()
    assert (o_raw[:band] == 9).all() and (o_raw[-band:] == 9).all()
    assert (l_raw[:band] == 9).all() and (l_raw[-band:] == 9).all()


def test_two_streams_with_a_workspace_each():
    x = make([2000, 700], [16, 9], 16, 16, 2, 128, 32, 0, 128, seed=17)
    y = make([100, 1700], [5, 16], 16, 16, 2, 128, 32, 0, 128, seed=18)
    want = [call(z, 0.09)[0] for z in (x, y)]
    args = [(z["q"], z["k_pages"], z["v_pages"], z["table"], _i32(z["ctxs"]), _i32(z["lens"]), _i32(z["depth"]),
             torch.as_tensor(mask_words(z["anc"])).cuda(), z["r"], z["w"], 0, 128, max(z["ctxs"])) for z in (x, y)]
    outs = [torch.full_like(w, 9.0) for w in want]
    size = ops.tree_workspace_size(2, 16, 16, 2, 2000, 128, 0)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, o, s, b in zip(args, outs, streams, ws):
            ops.attn_tree_paged(*a, scale=0.09, out=o, workspace=b, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_waits_that_run_out_leave_the_next_call_clean():
    """With a limit of a nanosecond ordinary waits give up: the call returns and reports it,
    and the next one under the default limit is right."""
    B, T, Hq, Hkv, d, page, ctx = 4, 16, 32, 4, 128, 256, 65536
    x = make([8] * B, [T] * B, T, Hq, Hkv, d, page, 0, 64, seed=21)
    blocks = ctx // page + 1
    g = torch.Generator(device="cuda").manual_seed(1)
    for n in ("k_pages", "v_pages"):
        x[n] = torch.randn(B * blocks, page, Hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    x["table"] = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)
    x["ctxs"] = [ctx] * B
    want, _ = call(x, 0.09)
    try:
        ops.set_wait_limit_ns(1)
        for _ in range(3):
            call(x, 0.09)
        assert ops.device_status(reset=True) & ops.RELBIAS_STATUS_TIMEOUT
    finally:
        ops.set_wait_limit_ns(0)
    out, _ = call(x, 0.09)
    assert ops.device_status(reset=True) == 0 and torch.equal(out, want)
