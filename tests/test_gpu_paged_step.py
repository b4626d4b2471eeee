"""The serving-step operators around the paged cache on the GPU: page plan, tree plan,
cache write with norms, and compaction, against plain references."""
import numpy as np
import pytest
import torch

from attention_learned_relative_b200 import ops
from paged_ref import mask_words, ref_page_plan, ref_tree_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    ops.device_status(reset=True)
    yield
    assert ops.device_status(reset=True) == 0, "a kernel reported a bad status"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _np(t):
    return t.cpu().numpy().astype(np.int64)


# ------------------------------------------------------------------------------ page_plan


def _plan_inputs(rng, B, T, page, top, free_share):
    done = rng.random(B) < 0.2
    ctx = np.where(done, 0, rng.integers(0, top + 1, B))
    new = np.where(done, 0, rng.integers(0, T + 1, B))
    held = -(-ctx // page) + rng.integers(0, 3, B)
    P = -(-(top + T) // page) + 2
    grow = int(np.maximum(-(-(ctx + new) // page) - held, 0).sum())
    free = int(grow * free_share)
    N = int(held.sum()) + free + 3
    perm = rng.permutation(N)
    table, at = np.full((B, P), -5, np.int64), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    head = int(rng.integers(0, N))
    ring = np.full(N, -9, np.int64)
    ring[(head + np.arange(free)) % N] = perm[at:at + free]
    return ctx, new, held, table, ring, np.array([head, free]), page, T


def _check_plan(args):
    ctx, new, held, table, ring, state, page, T = args
    g = [_i32(x) for x in (ctx, new, held, table, ring, state)]
    got = ops.page_plan(*g[:3], g[3], g[4], g[5], page, T)
    want = ref_page_plan(ctx, new, held, table, ring, state, page, T)
    for name, x, y in zip(("slots", "granted", "held", "table", "ring", "state"),
                          (got[0], got[1], got[2], g[3], g[4], got[3]), want):
        assert np.array_equal(_np(x), y), name
    assert np.array_equal(_np(g[2]), held) and np.array_equal(_np(g[5]), state)   # inputs as they were


@pytest.mark.parametrize("B,T,page,top,share", [
    (1, 1, 16, 0, 1.0), (1, 1, 1, 5, 1.0), (5, 16, 16, 300, 1.0), (37, 7, 48, 1000, 1.0), (64, 33, 64, 4000, 0.5),
    (257, 3, 16, 200, 0.7), (600, 5, 32, 100, 0.3), (3, 5000, 256, 9000, 1.0), (4, 4097, 7, 100, 0.6),
    (8, 0, 16, 100, 1.0), (6, 9, 16, 50, 0.0),
])
def test_page_plan(B, T, page, top, share):
    rng = np.random.default_rng(B * 7919 + T)
    for _ in range(3):
        _check_plan(_plan_inputs(rng, B, T, page, top, share))


def test_page_plan_refuses_bad_lengths_and_reports_them():
    rng = np.random.default_rng(1)
    ctx, new, held, table, ring, state, page, T = _plan_inputs(rng, 6, 8, 16, 60, 1.0)
    ctx[1], new[2], new[3], held[4] = -3, 9, -1, table.shape[1] + 1
    ctx[5] = 2 ** 31 - 1
    _check_plan((ctx, new, held, table, ring, state, page, T))
    assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_LENGTH


def test_page_plan_hands_out_nothing_from_an_impossible_ring():
    rng = np.random.default_rng(2)
    ctx, new, held, table, ring, state, page, T = _plan_inputs(rng, 4, 8, 16, 60, 1.0)
    ctx[:], new[:], held[:] = [0, 1, 20, 5], [4, 2, 8, 5], [0, 1, 1, 1]
    for bad in ([-1, 3], [len(ring), 3], [0, -2], [0, len(ring) + 1]):
        slots, granted, held2, _ = ops.page_plan(_i32(ctx), _i32(new), _i32(held), _i32(table), _i32(ring), _i32(bad),
                                                 page, T)
        assert _np(granted).tolist() == [0, 2, 0, 5] and _np(held2).tolist() == held.tolist()
        assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_LENGTH


def test_page_plan_of_no_requests_keeps_the_ring():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    ring = _i32([3, 1, 2, 0])
    out = ops.page_plan(z, z, z, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), ring, _i32([2, 3]), 16, 4)
    assert _np(out[3]).tolist() == [2, 3] and _np(ring).tolist() == [3, 1, 2, 0]


# ------------------------------------------------------------------------------ tree_plan


@pytest.mark.parametrize("B,T,shape", [
    (1, 1, "wide"), (3, 2, "chain"), (5, 31, "wide"), (4, 32, "chain"), (7, 33, "mixed"), (300, 64, "mixed"),
    (2, 100, "star"), (3, 128, "chain"), (9, 128, "mixed"), (2, 97, "roots"),
])
def test_tree_plan(B, T, shape):
    rng = np.random.default_rng(T)
    t = np.arange(T)[None, :].repeat(B, 0)
    far = np.floor(rng.random((B, T)) * np.maximum(t, 1)).astype(np.int64)
    p = {"chain": t - 1, "wide": far, "star": np.minimum(t - 1, 0), "roots": np.full_like(t, -1),
         "mixed": np.where(rng.random((B, T)) < 0.6, t - 1, far)}[shape]
    p[:, 0] = -1
    lens = rng.integers(0, T + 1, B)
    lens[0] = T
    depth, mask = ops.tree_plan(_i32(p), _i32(lens))
    d_ref, anc = ref_tree_plan(p, lens)
    assert np.array_equal(_np(depth), d_ref)
    assert np.array_equal(mask.cpu().numpy(), mask_words(anc))


def test_tree_plan_reports_a_parent_after_its_child():
    p = np.array([[-1, 0, 2, 3, -7, 1]])
    depth, mask = ops.tree_plan(_i32(p), _i32([6]))
    fixed = np.array([[-1, 0, -1, -1, -1, 1]])
    assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_TREE
    d_ref, anc = ref_tree_plan(fixed, [6])
    assert np.array_equal(_np(depth), d_ref) and np.array_equal(mask.cpu().numpy(), mask_words(anc))
    for n in (-1, 7):
        ops.tree_plan(_i32(fixed), _i32([n]))
        assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_LENGTH


# ------------------------------------------------------------------------------ kv_append

EPS_OF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def _append_case(dtype, lead, Hq, Hkv, d, page, norm, fused, seed, eps=1e-6, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = int(np.prod(lead))
    N = -(-n // page) + 2
    if fused:
        qkv = (torch.randn(*lead, (Hq + 2 * Hkv) * d, generator=g) * scale).to(dtype).cuda()
        q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], -1))
    else:
        q, k, v = ((torch.randn(*lead, h, d, generator=g) * scale).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(N * page, generator=g)[:n].reshape(lead).to(torch.int32)
    slots.view(-1)[3::5] = -1
    qw, kw = (1 + 0.3 * torch.randn(2, d, generator=g)).cuda() if norm else (None, None)
    kp, vp = (torch.randn(N, page, Hkv, d, generator=g).to(dtype).cuda() for _ in range(2))
    q_out = torch.randn(*lead, Hq, d, generator=g).to(dtype).cuda()
    want = [x.double().cpu().clone() for x in (q_out, kp, vp)]
    live = slots.view(-1) >= 0
    rows = slots.view(-1)[live].long()

    def normed(x, w):
        x = x.double().cpu().reshape(n, -1, d)[live]
        if w is None:
            return x
        return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()

    want[0].view(n, Hq, d)[live] = normed(q, qw)
    want[1].view(-1, Hkv, d)[rows] = normed(k, kw)
    want[2].view(-1, Hkv, d)[rows] = normed(v, None)
    out = ops.kv_append(k, v, slots.cuda(), kp, vp, q=q, q_weight=qw, k_weight=kw, eps=eps, q_out=q_out)
    assert out is q_out
    for name, x, y in zip(("q", "k", "v"), (q_out, kp, vp), want):
        # fp32 sum of d squares, mean, root and two products: (d + 8) 2^-24 of the value, then one rounding.
        tol = ((EPS_OF[dtype] + (d + 8) * 2.0 ** -24) * y.abs()) if norm and name != "v" else torch.zeros_like(y)
        off = (x.double().cpu() - y).abs()
        assert (off <= tol).all(), "%s off by %.3g" % (name, off.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("norm,fused", [(True, True), (True, False), (False, True)])
def test_kv_append(dtype, d, norm, fused):
    _append_case(dtype, (3, 7), 8, 2, d, 16, norm, fused, seed=d)
    _append_case(dtype, (1, 1), 1, 1, d, 1, norm, fused, seed=d + 1)
    _append_case(dtype, (130,), 5, 3, d, 48, norm, fused, seed=d + 2)


def test_kv_append_scales():
    """Rows of tiny values, where eps rules the norm, and of large ones."""
    _append_case(torch.float32, (4, 4), 4, 2, 128, 16, True, True, seed=1, eps=1e-2, scale=1e-3)
    _append_case(torch.bfloat16, (4, 4), 4, 2, 128, 16, True, True, seed=2, scale=1e4)


def test_kv_append_without_queries_and_with_slots_past_the_pool():
    k = torch.randn(6, 2, 64).bfloat16().cuda()
    kp = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    assert ops.kv_append(k, k, _i32([0, 31, 32, 2 ** 31 - 1, -2 ** 31, 5]), kp, vp) is None
    assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_LENGTH
    want = torch.zeros(32, 2, 64, dtype=torch.bfloat16, device="cuda")
    want[[0, 31, 5]] = k[[0, 1, 5]]
    assert torch.equal(kp.view(32, 2, 64), want) and torch.equal(vp.view(32, 2, 64), want)


def test_kv_append_of_a_head_of_zeros():
    """A head of zeros stays zero with any eps > 0; padding rows are not looked at."""
    q = torch.zeros(2, 4, 64, device="cuda")
    q[1] = float("nan")
    kp = torch.ones(1, 16, 4, 64, device="cuda")
    vp = torch.ones(1, 16, 4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    out = torch.full_like(q, 7.0)
    ops.kv_append(q, q, _i32([3, -1]), kp, vp, q=q, q_weight=w, k_weight=w, q_out=out)
    assert (out[0] == 0).all() and (out[1] == 7).all()
    assert (kp[0, 3] == 0).all() and (kp[0, :3] == 1).all() and (kp[0, 4:] == 1).all()


# ------------------------------------------------------------------------------ kv_compact


@pytest.mark.parametrize("L,B,A,T,page,Hkv,d,dtype", [
    (1, 1, 1, 1, 16, 1, 64, torch.bfloat16), (2, 5, 4, 9, 16, 2, 64, torch.bfloat16),
    (3, 4, 20, 60, 32, 4, 128, torch.bfloat16), (1, 7, 128, 128, 48, 3, 32, torch.float32),
    (2, 3, 33, 100, 7, 8, 256, torch.float32),
])
def test_kv_compact(L, B, A, T, page, Hkv, d, dtype):
    rng = np.random.default_rng(A)
    ctx = rng.integers(0, 3 * page, B)
    need = -(-(ctx + T) // page)
    P, N = int(need.max()), int(need.sum()) + 2
    perm, table, at = rng.permutation(N), np.full((B, P), -4, np.int64), 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += int(need[b])
    kp, vp = (torch.randn(L, N, page, Hkv, d).to(dtype).cuda() for _ in range(2))
    lens = rng.integers(0, A + 1, B)
    lens[0] = A
    path = np.full((B, A), -1, np.int64)
    for b in range(B):
        path[b, :lens[b]] = np.sort(rng.choice(T, lens[b], replace=False))
    want = []
    for x in (kp, vp):
        y = x.clone().view(L, N * page, Hkv, d)
        src = y.clone()
        for b in range(B):
            at = lambda j: int(table[b, j // page] * page + j % page)   # noqa: E731
            for i in range(lens[b]):
                y[:, at(ctx[b] + i)] = src[:, at(ctx[b] + path[b, i])]
        want.append(y.view_as(x))
    args = (_i32(table), _i32(ctx), _i32(path), _i32(lens))
    if L == 1:
        ops.kv_compact(kp[0], vp[0], *args)
    else:
        ops.kv_compact(kp, vp, *args)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_kv_compact_refuses_bad_paths_and_rows():
    page, P, N = 16, 2, 4
    table = np.array([[0, 1], [2, 3]])
    for path, lens, ctx, status in [
        ([[1, 1], [0, 3]], [2, 2], [0, 0], ops.RELBIAS_STATUS_BAD_TREE),        # not increasing
        ([[-1, 2], [0, 3]], [2, 2], [0, 0], ops.RELBIAS_STATUS_BAD_TREE),       # negative
        ([[0, 40], [0, 3]], [2, 2], [0, 0], ops.RELBIAS_STATUS_BAD_LENGTH),     # past the table
        ([[0, 2 ** 31 - 1], [0, 3]], [2, 2], [9, 0], ops.RELBIAS_STATUS_BAD_LENGTH),
        ([[0, 3], [0, 3]], [3, 2], [0, 0], ops.RELBIAS_STATUS_BAD_LENGTH),      # longer than the row
        ([[0, 3], [0, 3]], [-1, 2], [0, 0], ops.RELBIAS_STATUS_BAD_LENGTH),
        ([[0, 3], [0, 3]], [2, 2], [-5, 0], ops.RELBIAS_STATUS_BAD_LENGTH),
    ]:
        kp, vp = (torch.randn(N, page, 2, 64).bfloat16().cuda() for _ in range(2))
        k0 = kp.clone()
        ops.kv_compact(kp, vp, _i32(table), _i32(ctx), _i32(path), _i32(lens))
        assert ops.device_status(reset=True) == status
        assert torch.equal(kp[:2], k0[:2])                       # the bad sequence is untouched
        assert torch.equal(kp[2, 1], k0[2, 3])                   # the other one has moved
    bad = table.copy()
    bad[0, 0] = N
    kp, vp = (torch.randn(N, page, 2, 64).bfloat16().cuda() for _ in range(2))
    k0 = kp.clone()
    ops.kv_compact(kp, vp, _i32(bad), _i32([0, 0]), _i32([[0, 3], [0, 3]]), _i32([2, 2]))
    assert ops.device_status(reset=True) == ops.RELBIAS_STATUS_BAD_LENGTH
    assert torch.equal(kp[:2], k0[:2]) and torch.equal(kp[2, 1], k0[2, 3])
