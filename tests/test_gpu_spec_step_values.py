"""Steps of speculative decoding as a serving loop runs them, each operator's values checked on
what the one before it really wrote: the attention on the queries that kv_append returned and
the rows that stand in the pages, so that its bound is that of a call by itself."""
import numpy as np
import pytest
import torch

from attention_learned_relative_b200 import ops
from paged_ref import assert_tree_close, ref_tree_attn, ref_tree_plan
from test_gpu_spec_step import B, EPS, R, SCALE, W, Hkv, Hq, Loop, T, _cuda, _inputs, d, layers, page

pytestmark = pytest.mark.gpu


def _assert_normed(got, x, w, what):
    """x * w / sqrt(mean x^2 + eps): one rounding to bf16, and (d + 8) 2^-24 for the fp32 sum of
    squares, reciprocal root and products."""
    x = x.astype(np.float64)
    want = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    assert (np.abs(got - want) <= (2.0 ** -8 + (d + 8) * 2.0 ** -24) * np.abs(want) + 2.0 ** -130).all(), what


def _rows(pages, table, n):
    """The first n cache rows of a request, through its block-table row."""
    j = np.arange(n)
    at = table[j // page] * page + j % page
    return pages.view(-1, Hkv, d)[torch.as_tensor(at, device=pages.device)].double().cpu().numpy()


def test_each_operator_of_a_step_on_what_the_one_before_wrote(monkeypatch):
    rng, g = np.random.default_rng(3), torch.Generator().manual_seed(3)
    ops.device_status(reset=True)
    loop = Loop(3)
    seen = []
    attend = ops.attn_tree_paged

    def watched(q, k_pages, v_pages, table, *rest, **kw):
        seen.append([x.clone() for x in (q, k_pages, v_pages, table)])
        return attend(q, k_pages, v_pages, table, *rest, **kw)

    monkeypatch.setattr(ops, "attn_tree_paged", watched)
    w, wq, wk = (x.double().cpu().numpy() for x in (loop.w, loop.wq, loop.wk))
    kept = [[[np.zeros((0, Hkv, d))] * 2 for _ in range(B)] for _ in range(layers)]
    rejected = total = 0
    for i in range(5):
        x = _inputs(rng, g)
        seen.clear()
        outs, lses, granted = loop.step(_cuda(x))
        assert granted.tolist() == x["new"].tolist() and len(seen) == layers
        depth, anc = ref_tree_plan(x["parents"], x["new"])
        for layer in range(layers):
            qn, kp, vp, table = seen[layer]
            qn, table = qn.double().cpu().numpy(), table.cpu().numpy()
            q, k, v = (y.unflatten(-1, (-1, d)).double().numpy()
                       for y in x["qkv"][layer].split([Hq * d, Hkv * d, Hkv * d], -1))
            for b in range(B):
                what = "step %d layer %d request %d" % (i, layer, b)
                n, (k0, v0) = int(x["new"][b]), kept[layer][b]
                ctx = len(k0)
                kk, vv = _rows(kp, table[b], ctx + n), _rows(vp, table[b], ctx + n)
                # The prefix is what the steps before left, bit for bit; new values are moved, keys and queries normed.
                assert np.array_equal(kk[:ctx], k0) and np.array_equal(vv[:ctx], v0), what
                assert np.array_equal(vv[ctx:], v[b, :n]), what
                _assert_normed(kk[ctx:], k[b, :n], wk, what + ": keys")
                _assert_normed(qn[b, :n], q[b, :n], wq, what + ": queries")
                assert (qn[b, n:] == 0).all(), what
                ref = ref_tree_attn(qn[b], kk, vv, ctx, n, depth[b], anc[b], x["r"][layer][b], w[layer],
                                    W if layer == 0 else 0, R, SCALE)
                o = outs[layer][b, :n].double().cpu().numpy()
                lse = lses[layer][b, :, :n].T.double().cpu().numpy()
                assert_tree_close(o, lse, ref, d, what)
                assert (outs[layer][b, n:] == 0).all(), what
                # The bound tells a wrong answer from a right one: zeros, and the values of another head.
                total += 2
                for wrong in (np.zeros_like(o), np.roll(o, Hq // Hkv, axis=1)):
                    try:
                        assert_tree_close(wrong, lse, ref, d, what)
                    except AssertionError:
                        rejected += 1
                keep = x["path"][b, :x["taken"][b]]
                kept[layer][b] = [np.concatenate([y[:ctx], y[ctx + keep]]) for y in (kk, vv)]
    assert rejected == total
    assert loop.ctx.tolist() == [len(kept[0][b][0]) for b in range(B)]
    # Compaction left every layer's accepted rows in place.
    table = loop.table.cpu().numpy()
    for layer in range(layers):
        for b in range(B):
            n = len(kept[layer][b][0])
            assert np.array_equal(_rows(loop.k[layer], table[b], n), kept[layer][b][0])
            assert np.array_equal(_rows(loop.v[layer], table[b], n), kept[layer][b][1])
    assert ops.device_status(reset=True) == 0
