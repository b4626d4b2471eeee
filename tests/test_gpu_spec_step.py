"""Steps of speculative decoding with all the operators together, as a serving loop runs
them, against dense caches kept on the side; then the same step captured into a graph."""
import numpy as np
import pytest
import torch

from attention_learned_relative_b200 import ops
from paged_ref import assert_tree_close, ref_tree_attn, ref_tree_plan

pytestmark = pytest.mark.gpu

B, T, Hq, Hkv, d, page, layers, W, R = 3, 12, 8, 2, 64, 16, 2, 40, 24
P, N, SCALE, EPS, MAX_CTX = 12, 40, 0.125, 1e-6, 150


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Loop:
    """The device state of a serving loop, and one step of it."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.k = torch.full((layers, N, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = torch.full_like(self.k, float("nan"))
        self.table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(N, generator=g).int().cuda()
        self.state, self.held, self.ctx = _i32([0, N]), _i32([0] * B), _i32([0] * B)
        self.wq, self.wk = (1 + 0.2 * torch.randn(2, d, generator=g)).cuda()
        self.w = (0.5 * torch.randn(layers, Hq, R, generator=g)).cuda()

    def step(self, x):
        slots, granted, held, state = ops.page_plan(self.ctx, x["new"], self.held, self.table, self.ring, self.state,
                                                    page, T)
        self.held.copy_(held)
        self.state.copy_(state)
        depth, mask = ops.tree_plan(x["parents"], granted)
        outs, lses = [], []
        for layer in range(layers):
            q, k, v = (y.unflatten(-1, (-1, d)) for y in x["qkv"][layer].split([Hq * d, Hkv * d, Hkv * d], -1))
            qn = ops.kv_append(k, v, slots, self.k[layer], self.v[layer], q=q, q_weight=self.wq, k_weight=self.wk,
                               eps=EPS, q_out=torch.zeros(B, T, Hq, d, dtype=torch.bfloat16, device="cuda"))
            lse = torch.zeros(B, Hq, T, device="cuda")
            outs.append(ops.attn_tree_paged(qn, self.k[layer], self.v[layer], self.table, self.ctx, granted, depth,
                                            mask, x["r"][layer], self.w[layer], W if layer == 0 else 0, R, MAX_CTX,
                                            scale=SCALE, out=torch.zeros_like(qn), lse=lse))
            lses.append(lse)
        ops.kv_compact(self.k, self.v, self.table, self.ctx, x["path"], x["taken"])
        self.ctx.add_(x["taken"])
        return outs, lses, granted


def _inputs(rng, g):
    parents = np.floor(rng.random((B, T)) * np.maximum(np.arange(T), 1)).astype(np.int64)
    parents[:, 0] = -1
    new = rng.integers(1, T + 1, B)
    path, taken = np.zeros((B, T), np.int64), np.zeros(B, np.int64)
    for b in range(B):
        chain, x = [], int(rng.integers(0, new[b]))
        while x >= 0:
            chain.insert(0, x)
            x = int(parents[b, x])
        path[b, :len(chain)], taken[b] = chain, len(chain)
    qkv = torch.randn(layers, B, T, (Hq + 2 * Hkv) * d, generator=g).bfloat16()
    r = torch.randn(layers, B, T, Hq, generator=g)
    return dict(parents=parents, new=new, path=path, taken=taken, qkv=qkv, r=r)


def _cuda(x):
    return {n: y.cuda() if torch.is_tensor(y) else _i32(y) for n, y in x.items()}


class Dense:
    """The same steps on dense caches of 64-bit rows."""

    def __init__(self, loop):
        self.k = [[np.zeros((0, Hkv, d)) for _ in range(B)] for _ in range(layers)]
        self.v = [[np.zeros((0, Hkv, d)) for _ in range(B)] for _ in range(layers)]
        self.w, self.wq, self.wk = (y.double().cpu().numpy() for y in (loop.w, loop.wq, loop.wk))

    def check(self, x, outs, lses, what):
        depth, anc = ref_tree_plan(x["parents"], x["new"])
        for layer in range(layers):
            q, k, v = (y.unflatten(-1, (-1, d)).double() for y in x["qkv"][layer].split([Hq * d, Hkv * d, Hkv * d], -1))

            def norm(y, w):
                y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * torch.as_tensor(w)
                return y.float().bfloat16().double().numpy()

            q, k, v = norm(q, self.wq), norm(k, self.wk), v.numpy()
            for b in range(B):
                n, ctx = int(x["new"][b]), len(self.k[layer][b])
                kk, vv = (np.concatenate([c[layer][b], y[b, :n]]) for c, y in ((self.k, k), (self.v, v)))
                o, lse, absv, size = ref_tree_attn(q[b], kk, vv, ctx, n, depth[b], anc[b], x["r"][layer][b],
                                                   self.w[layer], W if layer == 0 else 0, R, SCALE)
                # A normed query or key may round the other way: 2^-7 of a logit's absolute terms at two operands.
                slack = 2 * 2.0 ** -7 * size
                ref = (o, lse, absv * (1 + 2.0 ** 8 * slack[..., None]), size + slack * 2.0 ** 24 / (d + 16))
                assert_tree_close(outs[layer][b, :n].double().cpu().numpy(),
                                  lses[layer][b, :, :n].T.double().cpu().numpy(), ref, d, "%s layer %d" % (what, layer))
                keep = x["path"][b, :x["taken"][b]]
                self.k[layer][b] = np.concatenate([kk[:ctx], kk[ctx + keep]])
                self.v[layer][b] = np.concatenate([vv[:ctx], vv[ctx + keep]])


def test_steps_of_a_serving_loop():
    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    ops.device_status(reset=True)
    loop = Loop(0)
    dense = Dense(loop)
    for i in range(6):
        x = _inputs(rng, g)
        outs, lses, granted = loop.step(_cuda(x))
        assert granted.tolist() == x["new"].tolist()
        dense.check(x, outs, lses, "step %d" % i)
    ctx = loop.ctx.tolist()
    assert ctx == [len(y) for y in dense.k[0]]
    # Values are moved, never rounded: the cache holds the dense rows.
    for layer in range(layers):
        for b in range(B):
            j = np.arange(ctx[b])
            at = loop.table[b].cpu().numpy()[j // page] * page + j % page
            assert np.array_equal(loop.v[layer].view(-1, Hkv, d)[torch.as_tensor(at).cuda()].double().cpu().numpy(),
                                  dense.v[layer][b])
    # Every page is held by one request or free.
    held, (head, count) = loop.held.tolist(), loop.state.tolist()
    owned = [int(loop.table[b, i]) for b in range(B) for i in range(held[b])]
    free = [int(loop.ring[(head + i) % N]) for i in range(count)]
    assert sorted(owned + free) == list(range(N))
    assert ops.device_status(reset=True) == 0


def test_a_captured_step_replays():
    """Two graphs of the same step, replayed in turn with new inputs, and the eager loop
    beside them give the same bits."""
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    xs = [_inputs(rng, g) for _ in range(5)]
    eager = Loop(1)
    want = []
    for x in xs:
        outs, _, _ = eager.step(_cuda(x))
        want.append([y.clone() for y in outs])
    loop = Loop(1)
    fixed = _cuda(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs, _, _ = loop.step(fixed)
            graphs.append((graph, outs))
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        for n, y in _cuda(x).items():
            fixed[n].copy_(y)
        graph, outs = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want[i]):
            assert torch.equal(a, b)
    assert ops.device_status(reset=True) == 0
