"""Plain references of the serving-step operators over a paged cache, in 64 bits or whole
numbers, on the CPU: one loop per definition, sharing no code with the library."""
import math

import numpy as np


def ref_page_plan(ctx, new, held, table, ring, state, page, T):
    """(slots, granted, held', table', ring', state'), by walking the requests in order."""
    table, ring, held = table.copy(), ring.copy(), held.copy()
    B, P = table.shape
    N = len(ring)
    head, count = int(state[0]), int(state[1])
    slots = np.full((B, T), -1, np.int64)
    granted = np.zeros(B, np.int64)
    asked = taken = returned = 0
    for b in range(B):
        need = -(-(int(ctx[b]) + int(new[b])) // page)
        if ctx[b] < 0 or new[b] < 0 or new[b] > T or held[b] < 0 or held[b] > P or need > P:
            continue
        grow = max(0, need - int(held[b]))
        first, asked = asked, asked + grow
        if grow and asked > count:
            continue
        for i in range(grow):
            table[b, held[b] + i] = ring[(head + first + i) % N]
        taken = max(taken, asked if grow else 0)
        for i in range(need, int(held[b])):
            ring[(head + count + returned) % N] = table[b, i]
            returned += 1
        held[b] = need
        granted[b] = new[b]
        for t in range(int(new[b])):
            pos = int(ctx[b]) + t
            slots[b, t] = table[b, pos // page] * page + pos % page
    return slots, granted, held, table, ring, np.array([(head + taken) % N, count - taken + returned])


def ref_tree_plan(parents, lens):
    B, T = parents.shape
    depth = np.zeros((B, T), np.int64)
    anc = np.zeros((B, T, T), bool)
    for b in range(B):
        for t in range(int(lens[b])):
            x = t
            while x >= 0:
                anc[b, t, x] = True
                x = int(parents[b, x])
            depth[b, t] = anc[b, t].sum() - 1
    return depth, anc


def mask_words(anc):
    """[B, T, ceil(T/32)] int32 words of a [B, T, T] truth array."""
    B, T, _ = anc.shape
    W = (T + 31) // 32
    out = np.zeros((B, T, W), np.uint32)
    for s in range(T):
        out[:, :, s // 32] |= anc[:, :, s].astype(np.uint32) << np.uint32(s % 32)
    return out.view(np.int32)


def ref_tree_attn(q, k, v, ctx, n, depth, anc, r, w, window, R, scale, temp_n0=0):
    """One sequence: q [T,Hq,d], k and v [ctx+n,Hkv,d] in logical order, depth [T], anc
    [T,T], r [T,Hq], w [Hq,R].  Returns o [n,Hq,d], lse [n,Hq], and two sizes for error bounds:
    the weighted mean of |v| (of o's shape) and the largest sum of a logit's absolute terms."""
    q, k, v, r = (np.asarray(x, np.float64) for x in (q, k, v, r))
    Hq, d, G = q.shape[1], q.shape[2], q.shape[1] // k.shape[1]
    o, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    absv, size = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    rel = np.concatenate([np.arange(ctx) - ctx, depth[:n]]).astype(np.int64)
    for t in range(n):
        dist = int(depth[t]) - rel
        seen = np.concatenate([np.ones(ctx, bool), anc[t, :n]]) & (dist >= 0)
        if window > 0:
            seen &= dist < window
        if not seen.any():
            continue
        pos = ctx + int(depth[t])
        cnt = min(pos + 1, window) if window > 0 else pos + 1
        tau = max(1.0, math.log(cnt) / math.log(temp_n0)) if temp_n0 > 1 else 1.0
        near = seen & (dist < R)
        for h in range(Hq):
            kk, vv = k[seen, h // G], v[seen, h // G]
            bias = np.zeros(len(dist))
            if R > 0:
                bias[near] = r[t, h] * np.asarray(w, np.float64)[h, dist[near]]
            logit = tau * (scale * kk @ q[t, h] + bias[seen])
            top = logit.max()
            p = np.exp(logit - top)
            o[t, h] = p @ vv / p.sum()
            absv[t, h] = p @ np.abs(vv) / p.sum()
            lse[t, h] = top + math.log(p.sum())
            size[t, h] = (tau * (scale * np.abs(kk) @ np.abs(q[t, h]) + np.abs(bias[seen]))).max()
    return o, lse, absv, size


def assert_tree_close(o, lse, ref, d, what):
    """Against ref_tree_attn's answer.  Each weight p is rounded to bf16 before the product
    with V (off by 2^-8 of itself at most), the output once more, and the sum runs over the
    unrounded weights: |error| <= 2^-8 (mean |v| + |o|), and the fp32 arithmetic of logits and
    exponentials adds (d + 16) 2^-24 of a logit's absolute terms, relative to the weights,
    twice (numerator and sum).  The log-sum-exp carries that last error once, and 2^-20 for
    the fp32 exponential, logarithm and final product."""
    o_ref, lse_ref, absv, size = ref
    arith = (d + 16) * 2.0 ** -24 * size + 2.0 ** -20
    tol = 2.0 ** -8 * (absv + np.abs(o_ref)) * (1 + 2.0 ** -8) + 2 * arith[..., None] * absv
    err = np.abs(o - o_ref)
    assert np.isfinite(o).all(), what + ": not finite"
    assert (err <= tol).all(), "%s: output off by %.3g where %.3g is allowed" % (
        what, err.flat[(err - tol).argmax()], tol.flat[(err - tol).argmax()])
    empty = np.isinf(lse_ref)
    assert (lse[empty] == -np.inf).all(), what + ": log-sum-exp of rows that see nothing"
    bound = arith + 2.0 ** -22 * np.abs(np.where(empty, 0, lse_ref))
    off = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, lse_ref))
    assert (off <= bound).all(), "%s: log-sum-exp off by %.3g" % (what, off.max())
