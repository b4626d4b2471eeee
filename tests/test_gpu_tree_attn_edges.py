"""Edges of the attention of drafted trees over a paged cache: values that are not finite."""
import numpy as np
import pytest
import torch

from attention_learned_relative_b200 import ops
from test_gpu_tree_attn import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    ops.device_status(reset=True)
    yield
    assert ops.device_status(reset=True) == 0, "a kernel reported a bad status"


def _key(x, b, row):
    """Row `row` of sequence b's keys in the pool: [Hkv, d]."""
    page = x["k_pages"].shape[1]
    return x["k_pages"][int(x["table"][b, row // page]), row % page]


SHAPES = [  # ctxs, lens, T, Hq, Hkv, d, page, window: one row tile, two, cut segments, several pairs of row tiles
    ([20], [9], 9, 4, 2, 64, 16, 0),
    ([200, 77], [16, 12], 16, 16, 1, 128, 32, 50),
    ([3000], [5], 5, 8, 1, 128, 64, 0),
    ([3000], [20], 20, 8, 1, 64, 64, 0),
    ([2000], [70], 70, 16, 1, 128, 48, 0),
]


@pytest.mark.parametrize("ctxs,lens,T,Hq,Hkv,d,page,window", SHAPES)
def test_a_nan_reaches_the_log_sum_exp_of_the_rows_that_see_it(ctxs, lens, T, Hq, Hkv, d, page, window):
    """A NaN query, and a NaN key that a node sees: o and the log-sum-exp of those rows are
    NaN, and -inf is kept for rows that see nothing; all other rows keep their bits."""
    anc = np.tril(np.random.default_rng(T).random((len(ctxs), T, T)) < 0.5) | np.eye(T, dtype=bool)
    x = make(ctxs, lens, T, Hq, Hkv, d, page, window, 32, seed=T, anc=anc)
    good, good_lse = call(x, 0.125)
    t = lens[0] // 2
    x["q"][0, t] = float("nan")
    leaf = lens[0] - 1
    _key(x, 0, ctxs[0] + leaf)[:] = float("nan")
    out, lse = call(x, 0.125)
    for b, n in enumerate(lens):
        for s in range(n):
            dist = x["depth"][b, s] - x["depth"][b, leaf]
            hit = b == 0 and (s == t or (anc[b, s, leaf] and 0 <= dist and (window <= 0 or dist < window)))
            if hit:
                assert torch.isnan(out[b, s].float()).all() and torch.isnan(lse[b, :, s]).all(), (b, s)
            else:
                assert torch.equal(out[b, s], good[b, s]) and torch.equal(lse[b, :, s], good_lse[b, :, s]), (b, s)


@pytest.mark.parametrize("ctxs,lens,T,Hq,Hkv,d,page,window", SHAPES)
@pytest.mark.parametrize("first,last", [(0, 1), (0, 64), (0, 1 << 30)])
def test_nan_keys_of_the_prefix(ctxs, lens, T, Hq, Hkv, d, page, window, first, last):
    """One key, the keys of half a tile, and all keys of the prefix are NaN: every row that
    sees one of them is NaN in both outputs."""
    x = make(ctxs, lens, T, Hq, Hkv, d, page, window, 32, seed=T)
    for b, c in enumerate(ctxs):
        lo = max(0, c - window + 1) if window > 0 else 0
        for row in range(lo + first, min(c, lo + last)):
            _key(x, b, row)[:] = float("nan")
    out, lse = call(x, 0.125)
    for b, (c, n) in enumerate(zip(ctxs, lens)):
        lo = max(0, c - window + 1) if window > 0 else 0
        for s in range(n):
            back = c + int(x["depth"][b, s]) - (min(c, lo + last) - 1)   # distance to the nearest NaN key
            if window <= 0 or back < window:
                assert torch.isnan(out[b, s].float()).all() and torch.isnan(lse[b, :, s]).all(), (b, s)
            else:
                assert torch.isfinite(out[b, s].float()).all() and torch.isfinite(lse[b, :, s]).all(), (b, s)


def test_one_part_of_a_cut_segment_holds_nothing_but_nan():
    """3000 rows of one cache head are a key tile to a CTA: the NaN keys of one tile are all
    that one part sees, and none of the others sees any."""
    x = make([3000], [5], 5, 8, 1, 128, 128, 0, 32, seed=3)
    for row in range(256, 384):
        _key(x, 0, row)[:] = float("nan")
    out, lse = call(x, 0.125)
    assert torch.isnan(out.float()).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("ctxs,lens,T,Hq,Hkv,d,page,window", SHAPES)
def test_infinite_logits(ctxs, lens, T, Hq, Hkv, d, page, window):
    """A key whose logit is +inf makes a row NaN (inf - inf), one whose logit is -inf has no
    weight: here it is the infinite element's sign in the query that tells."""
    x = make(ctxs, lens, T, Hq, Hkv, d, page, window, 32, seed=T + 1)
    row = ctxs[0] - 1
    _key(x, 0, row)[:, 3] = float("inf")
    out, lse = call(x, 0.125)
    for s in range(lens[0]):
        if window > 0 and int(x["depth"][0, s]) + 1 >= window:
            continue
        up = x["q"][0, s, :, 3] > 0
        assert (x["q"][0, s, :, 3] != 0).all()
        assert torch.isnan(out[0, s, up].float()).all() and torch.isnan(lse[0, up, s]).all()
        assert torch.isfinite(out[0, s, ~up].float()).all() and torch.isfinite(lse[0, ~up, s]).all()


def test_without_a_table_r_has_no_say():
    """R = 0: there is no bias, whatever r holds, as in the decode step."""
    for value in (float("nan"), float("inf"), -float("inf")):
        x = make([513, 40], [7, 9], 9, 6, 2, 64, 16, 0, 0, seed=4)
        x["r"].zero_()
        want, want_lse = call(x, 0.125)
        x["r"].fill_(value)
        out, lse = call(x, 0.125)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_a_stream_with_all_arguments_by_keyword():
    side = torch.cuda.Stream()
    parents = torch.tensor([[-1, 0, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([4], dtype=torch.int32, device="cuda")
    want = ops.tree_plan(parents, lens)
    side.wait_stream(torch.cuda.current_stream())
    got = ops.tree_plan(depth=None, mask=None, parents=parents, tree_lens=lens, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
