"""One step of speculative decoding over the paged cache, operator by operator.

The operators, in the order a serving loop calls them:
  page_plan    block tables and slot maps built on the GPU from request lengths
  kv_append    query/key norm per head, and the write of new K and V rows into their pages
  tree_plan    node positions and ancestor masks of drafted token trees
  tree_attn    attention of the drafted nodes over the paged cache, with the learned relative bias
  kv_compact   the accepted path's rows moved to the rows they will keep

`own` selects the library's kernels; otherwise `run` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # A decode step of 64 running requests, 16 drafted tokens each.
        dict(name="plan_step", op="page_plan", B=64, T=16, page=64, ctx=8192, tight=False),
        # Admission of a batch of long prompts: 8192 new rows per request.
        dict(name="plan_prompts", op="page_plan", B=256, T=8192, page=256, ctx=65536, tight=True),
        # One request's tree, built once per step and read by every layer.
        dict(name="tree_one", op="tree_plan", B=1, T=16, chain=0.3),
        # A large batch of wide trees.
        dict(name="tree_batch", op="tree_plan", B=256, T=64, chain=0.6),
        # The new rows of a decode step, q, k and v sliced from one projection's output.
        dict(name="append_step", op="kv_append", B=8, T=16, Hq=32, Hkv=4, d=128, page=64, norm=True, dtype="bf16"),
        # The rows of two 8192-token prompts.
        dict(name="append_prompts", op="kv_append", B=2, T=8192, Hq=32, Hkv=4, d=128, page=256, norm=True,
             dtype="bf16"),
        # The smallest call: one short request, where latency counts.
        dict(name="attn_short", op="tree_attn", B=1, T=4, ctx=300, spread=0, Hq=8, Hkv=2, d=64, page=16, window=64,
             R=64, temp_n0=0, chain=0.3),
        # A local layer (512-key window, 512-distance bias) of a running batch.
        dict(name="attn_local", op="tree_attn", B=64, T=16, ctx=8192, spread=6000, Hq=32, Hkv=4, d=128, page=32,
             window=512, R=512, temp_n0=0, chain=0.5),
        # A global layer of one request near the 1,048,576-row context.
        dict(name="attn_long", op="tree_attn", B=1, T=8, ctx=1048560, spread=0, Hq=32, Hkv=4, d=128, page=256,
             window=0, R=1024, temp_n0=131072, chain=0.5),
        # A global layer of eight long requests with wide trees: products outweigh the cache traffic.
        dict(name="attn_large", op="tree_attn", B=8, T=64, ctx=131072, spread=65536, Hq=32, Hkv=4, d=128, page=64,
             window=0, R=1024, temp_n0=0, chain=0.6),
        # One layer's cache after a step of eight requests.
        dict(name="compact_step", op="kv_compact", L=1, B=8, A=5, T=16, ctx=2000, Hkv=4, d=128, page=64),
        # All layers' caches after a step of a running batch.
        dict(name="compact_layers", op="kv_compact", L=32, B=64, A=8, T=64, ctx=100, Hkv=4, d=128, page=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["page_plan", "tree_plan", "kv_append", "tree_attn", "tree_attn", "kv_compact"])
    page = rng.choice([16, 32, 48, 64, 96, 128, 256])
    Hq, Hkv = rng.choice([(32, 4), (8, 2), (16, 4), (12, 4), (8, 8), (6, 1), (16, 1), (10, 2)])
    if op == "page_plan":
        B = _log_int(rng, 1, 512)
        return dict(op=op, B=B, T=_log_int(rng, 1, min(8192, (1 << 21) // B)), page=page,
                    ctx=_log_int(rng, 1, 65536), tight=rng.random() < 0.3)
    if op == "tree_plan":
        T = _log_int(rng, 8, 64 if rng.random() < 0.7 else 128)
        return dict(op=op, B=_log_int(rng, 1, 256 if T <= 64 else 85), T=T, chain=rng.choice([0.0, 0.5, 0.8]))
    if op == "kv_append":
        B, d = _log_int(rng, 1, 64), rng.choice([32, 64, 128, 256])
        most = max(1, 40_000_000 // (B * (Hq + 2 * Hkv) * d))
        return dict(op=op, B=B, T=_log_int(rng, 1, min(8192, most)), Hq=Hq, Hkv=Hkv, d=d, page=page,
                    norm=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "kv_compact":
        A, B, d = rng.randint(1, 12), _log_int(rng, 1, 64), rng.choice([64, 128])
        return dict(op=op, L=_log_int(rng, 1, max(1, min(32, 6_000_000 // (B * A * Hkv * d)))), B=B, A=A,
                    T=2 * A + rng.randint(0, 40), ctx=rng.randint(0, 200), Hkv=Hkv, d=d, page=page)
    window, d = rng.choice([0, 0, 64, 500, 512]), rng.choice([64, 128])
    T = _log_int(rng, 1, 128)
    if window:
        B, ctx = _log_int(rng, 1, 64), _log_int(rng, 1, 8192)
    else:
        B = _log_int(rng, 1, 32)
        ctx = _log_int(rng, 1, min(262144, 1_500_000_000 // (4 * B * Hkv * d), 1_500_000_000 // (B * T * Hq)))
    return dict(op=op, B=B, T=T, ctx=ctx, spread=rng.choice([0, ctx // 2, ctx]), Hq=Hq, Hkv=Hkv, d=d, page=page, window=window, R=rng.choice([1, 64, 300, 512, 1024]),
                temp_n0=rng.choice([0, 0, 1000]), chain=rng.choice([0.0, 0.5, 1.0]))


# ------------------------------------------------------------------------------------- inputs

def _ctx(case):
    """Rows of each request's cache: from ctx down by `spread` over the batch."""
    return [case["ctx"] - (b * case["spread"]) // case["B"] for b in range(case["B"])]


def _lens(case):
    """Drafted nodes of each request: T, or one or two fewer."""
    return [max(1, case["T"] - b % 3) for b in range(case["B"])]


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _parents(case, rs):
    """[B, T] parent of each node, -1 at the root: the previous node with probability `chain`, else any earlier one."""
    B, T = case["B"], case["T"]
    t = np.arange(T)[None, :]
    far = np.floor(rs.random((B, T)) * np.maximum(t, 1)).astype(np.int64)
    p = np.where(rs.random((B, T)) < case["chain"], t - 1, far)
    p[:, 0] = -1
    return p


def _tree(parents):
    """Depths [B, T] and ancestor-or-self words [B, T, ceil(T/32)] of the trees, on the host."""
    B, T = parents.shape
    depth = np.zeros((B, T), np.int64)
    anc = np.zeros((B, T, T), bool)
    rows = np.arange(B)
    for t in range(T):
        p = parents[:, t]
        has = p >= 0
        depth[:, t] = np.where(has, depth[rows, np.maximum(p, 0)] + 1, 0)
        anc[:, t] = anc[rows, np.maximum(p, 0)] & has[:, None]
        anc[:, t, t] = True
    W = (T + 31) // 32
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :T] = anc
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return depth, words.view(np.int32)


def _table(rows, page, rs, most=None):
    """Block table of requests with these row counts (room for `most` each), over a shuffled pool, and its size."""
    need = [-(-n // page) for n in rows]
    room = need if most is None else [-(-most // page)] * len(rows)
    P, N = max(1, max(room)), sum(room) + 3
    perm = rs.permutation(N)
    table, at = np.zeros((len(rows), P), np.int64), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, N


def prepare(case, seed):
    rs = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, B = case["op"], case["B"]

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        return x if std == 1.0 else x * std

    if op == "page_plan":
        T, page, top = case["T"], case["page"], case["ctx"]
        ctx = rs.integers(0, top + 1, B)
        new = rs.integers(0, T + 1, B)
        done = rs.random(B) < 0.1                      # finished requests give their pages back
        held = -(-ctx // page) + rs.integers(0, 2, B)  # some hold a page of a rejected draft
        ctx, new = np.where(done, 0, ctx), np.where(done, 0, new)
        need = -(-(ctx + new) // page)
        grow = int(np.maximum(need - held, 0).sum())
        P = -(-(top + T) // page) + 1
        free = max(1, int(grow * 0.8) if case["tight"] else grow + 5)
        N = B * P + 5                                  # the rest of the pool belongs to other batches
        perm = rs.permutation(N)
        table, at = np.full((B, P), -1, np.int64), 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += int(held[b])
        head = int(rs.integers(0, N))
        ring = np.full(N, -1, np.int64)
        ring[(head + np.arange(free)) % N] = perm[at:at + free]
        return dict(case=case, ctx=_i32(ctx), new=_i32(new), held=_i32(held), table=_i32(table), ring=_i32(ring),
                    state=_i32([head, free]))
    if op == "tree_plan":
        return dict(case=case, parents=_i32(_parents(case, rs)), lens=_i32(rs.integers(case["T"] // 2, case["T"] + 1, B)))
    if op == "kv_append":
        T, Hq, Hkv, d, page = (case[k] for k in ("T", "Hq", "Hkv", "d", "page"))
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        lens = _lens(case)
        table, N = _table([7 + T] * B, page, rs)
        t = 7 + np.arange(T)
        slots = np.where(np.arange(T)[None] < np.asarray(lens)[:, None], table[:, t // page] * page + t % page, -1)
        qkv = normal(B, T, (Hq + 2 * Hkv) * d, dtype=dt)
        return dict(case=case, qkv=qkv, slots=_i32(slots), wq=1 + normal(d, dtype=torch.float32, std=0.1),
                    wk=1 + normal(d, dtype=torch.float32, std=0.1), k_pages=normal(N, page, Hkv, d, dtype=dt),
                    v_pages=normal(N, page, Hkv, d, dtype=dt),
                    q_out=torch.zeros(B, T, Hq, d, dtype=dt, device="cuda"))
    if op == "tree_attn":
        T, Hq, Hkv, d, page, R = (case[k] for k in ("T", "Hq", "Hkv", "d", "page", "R"))
        ctx, lens = _ctx(case), _lens(case)
        table, N = _table([c + n for c, n in zip(ctx, lens)], page, rs)
        depth, words = _tree(_parents(case, rs))
        return dict(case=case, q=normal(B, T, Hq, d), k_pages=normal(N, page, Hkv, d),
                    v_pages=normal(N, page, Hkv, d), table=_i32(table), ctx=_i32(ctx), lens=_i32(lens),
                    depth=_i32(depth), mask=_i32(words), r=normal(B, T, Hq, dtype=torch.float32),
                    w=normal(Hq, R, dtype=torch.float32, std=0.5), max_ctx=max(ctx), scale=1.0 / math.sqrt(d),
                    o=torch.zeros(B, T, Hq, d, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(B, Hq, T, dtype=torch.float32, device="cuda"))
    L, A, T, Hkv, d, page = (case[k] for k in ("L", "A", "T", "Hkv", "d", "page"))
    ctx = case["ctx"] + rs.integers(0, page, B)
    table, N = _table([int(c) + T for c in ctx], page, rs, most=case["ctx"] + page + T)
    # The root is accepted, then nodes from past the rows that are filled (a level-ordered tree whose first
    # levels are wide), so that a step can be repeated.
    path = np.zeros((B, A), np.int64)
    for b in range(B):
        path[b, 1:] = np.sort(rs.choice(np.arange(A, T), A - 1, replace=False))
    return dict(case=case, k_pages=normal(L, N, page, Hkv, d), v_pages=normal(L, N, page, Hkv, d), table=_i32(table),
                ctx=_i32(ctx), path=_i32(path), lens=_i32([1 + b % A for b in range(B)]))


# ------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        from attention_learned_relative_b200 import ops
        if op == "page_plan":
            slots, granted, held, state = ops.page_plan(s["ctx"], s["new"], s["held"], s["table"], s["ring"],
                                                        s["state"], s["case"]["page"], s["case"]["T"])
            return dict(slots=slots, granted=granted, held=held, state=state, table=s["table"], ring=s["ring"])
        if op == "tree_plan":
            depth, mask = ops.tree_plan(s["parents"], s["lens"])
            return dict(depth=depth, mask=mask)
        if op == "kv_append":
            q, k, v = _split(s)
            norm = s["case"]["norm"]
            ops.kv_append(k, v, s["slots"], s["k_pages"], s["v_pages"], q=q, q_weight=s["wq"] if norm else None,
                          k_weight=s["wk"] if norm else None, eps=EPS, q_out=s["q_out"])
            return dict(q=s["q_out"], k=s["k_pages"], v=s["v_pages"])
        if op == "tree_attn":
            c = s["case"]
            o = ops.attn_tree_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["lens"], s["depth"],
                                    s["mask"], s["r"], s["w"], c["window"], c["R"], s["max_ctx"], scale=s["scale"],
                                    out=s["o"], lse=s["lse"], temp_n0=c["temp_n0"])
            return dict(o=o, lse=s["lse"])
        ops.kv_compact(s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["path"], s["lens"])
        return dict(k=s["k_pages"], v=s["v_pages"])
    return dict(page_plan=_plain_page_plan, tree_plan=_plain_tree_plan, kv_append=_plain_append,
                tree_attn=_plain_attn, kv_compact=_plain_compact)[op](s)


def _split(s):
    """q, k, v [B, T, heads, d]: slices of the projection's output, not copied."""
    c = s["case"]
    B, T, Hq, Hkv, d = (c[k] for k in ("B", "T", "Hq", "Hkv", "d"))
    q, k, v = s["qkv"].split([Hq * d, Hkv * d, Hkv * d], dim=2)
    return q.unflatten(2, (Hq, d)), k.unflatten(2, (Hkv, d)), v.unflatten(2, (Hkv, d))


def _plain_page_plan(s):
    page, T = s["case"]["page"], s["case"]["T"]
    table, ring = s["table"], s["ring"]
    ctx, new, held = s["ctx"].long(), s["new"].long(), s["held"].long()
    head, count = s["state"][0].long(), s["state"][1].long()
    N, P = ring.numel(), table.shape[1]
    need = (ctx + new + page - 1) // page
    grow, shrink = (need - held).clamp(min=0), (held - need).clamp(min=0)
    cum = grow.cumsum(0)
    ok = (grow == 0) | (cum <= count)
    granted = torch.where(ok, new, 0)
    taken = torch.where(cum <= count, cum, 0).amax()
    now = torch.where(ok, need, held)
    col = torch.arange(P, device=ctx.device)[None, :]
    fresh = (col >= held[:, None]) & (col < now[:, None])
    source = (head + (cum - grow)[:, None] + col - held[:, None]) % N
    back = (col >= need[:, None]) & (col < held[:, None])
    given = shrink.cumsum(0)
    target = (head + count + (given - shrink)[:, None] + col - need[:, None]) % N
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer.scatter_(0, torch.where(back, target, N).flatten(), table.flatten())
    table.copy_(torch.where(fresh, ring[source], table))
    ring.copy_(longer[:N])
    pos = ctx[:, None] + torch.arange(T, device=ctx.device)[None, :]
    inside = torch.arange(T, device=ctx.device)[None, :] < granted[:, None]
    block = torch.gather(table, 1, torch.where(inside, pos // page, 0)).long()
    slots = torch.where(inside, block * page + pos % page, -1)
    state = torch.stack([(head + taken) % N, count - taken + given[-1]])
    return dict(slots=slots.int(), granted=granted.int(), held=now.int(), state=state.int(), table=table, ring=ring)


def _plain_tree_plan(s):
    parents, lens = s["parents"].long(), s["lens"]
    B, T = parents.shape
    node = torch.arange(T, device=parents.device)
    live = node[None, :] < lens[:, None]
    # Reach of at most 2^k steps by k squarings of (identity + parent).
    reach = (parents[:, :, None] == node[None, None, :]) & live[:, :, None]
    reach = (reach | (node[:, None] == node[None, :])).float()
    for _ in range(max(1, (T - 1).bit_length())):
        reach = (reach @ reach).clamp(max=1.0)
    reach = (reach > 0) & live[:, :, None]
    depth = (reach.sum(2) - 1).clamp(min=0)
    W = (T + 31) // 32
    bits = torch.nn.functional.pad(reach, (0, W * 32 - T)).view(B, T, W, 32).long()
    words = (bits << torch.arange(32, device=parents.device)).sum(3)
    return dict(depth=depth.int(), mask=words.int())


def _plain_append(s):
    q, k, v = _split(s)
    dt = q.dtype
    if s["case"]["norm"]:
        q, k = q.float(), k.float()
        q = (q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["wq"]).to(dt)
        k = (k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["wk"]).to(dt)
    slots = s["slots"].long()
    live = slots >= 0
    s["q_out"].copy_(torch.where(live[:, :, None, None], q, s["q_out"]))
    # Rows without a slot repeat the write of the batch's first row, which always has one.
    at = torch.where(live, slots, slots[0, 0]).flatten()
    flat = live.flatten()[:, None, None]
    k, v = k.flatten(0, 1), v.flatten(0, 1)
    s["k_pages"].flatten(0, 1).index_copy_(0, at, torch.where(flat, k, k[:1]))
    s["v_pages"].flatten(0, 1).index_copy_(0, at, torch.where(flat, v, v[:1]))
    return dict(q=s["q_out"], k=s["k_pages"], v=s["v_pages"])


def _plain_attn(s):
    c = s["case"]
    B, T, Hq, Hkv, d, page, W, R = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "page", "window", "R"))
    G = Hq // Hkv
    ctx, depth = s["ctx"].long(), s["depth"].long()
    back = min(W - 1, s["max_ctx"]) if W > 0 else s["max_ctx"]     # prefix rows that any node may see
    e = torch.arange(-back, T, device=ctx.device)                  # key rows relative to the end of the prefix
    node = e.clamp(min=0)
    row = ctx[:, None] + e[None, :]
    inside = (row >= 0) & (e[None, :] < s["lens"][:, None])
    row = torch.where(inside, row, 0)
    at = torch.gather(s["table"].long(), 1, row // page) * page + row % page
    k = s["k_pages"].flatten(0, 1)[at].float()                     # [B, S, Hkv, d]
    v = s["v_pages"].flatten(0, 1)[at].float()
    rel = torch.where(e[None, :] < 0, e[None, :], depth[:, node])  # position of each key less ctx
    dist = depth[:, :, None] - rel[:, None, :]                     # [B, T, S]
    word = torch.gather(s["mask"].long(), 2, (node // 32)[None, None, :].expand(B, T, -1))
    bit = (word >> (node % 32)) & 1
    seen = inside[:, None, :] & ((e < 0) | (bit == 1)) & (dist >= 0)
    if W > 0:
        seen &= dist < W
    q = s["q"].float().unflatten(2, (Hkv, G))
    logit = torch.einsum("btgnd,bsgd->bgnts", q, k).mul_(s["scale"])
    near = max(0, e.numel() - T - R)                               # the bias reaches the last R prefix rows
    dn = dist[:, :, near:]
    bias = torch.where((dn >= 0) & (dn < R), s["w"][:, dn.clamp(0, R - 1)], 0.0)       # [Hq, B, T, S']
    bias = bias.permute(1, 0, 2, 3) * s["r"].transpose(1, 2)[..., None]
    logit[..., near:] += bias.unflatten(1, (Hkv, G))
    if c["temp_n0"] > 1:
        n = ctx[:, None] + depth + 1
        n = n.clamp(max=W) if W > 0 else n
        tau = (n.double().log() / math.log(c["temp_n0"])).clamp(min=1.0).float()
        logit *= tau[:, None, None, :, None]
    logit = logit.masked_fill_(~seen[:, None, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = logit.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bgnts,bsgd->bgntd", p, v) / torch.where(total == 0, 1.0, total)
    live = torch.arange(T, device=ctx.device)[None, :] < s["lens"][:, None]
    o = o.flatten(1, 2).transpose(1, 2)
    lse = (top + total.log()).squeeze(-1).flatten(1, 2)
    return dict(o=torch.where(live[:, :, None, None], o, 0.0).to(torch.bfloat16),
                lse=torch.where(live[:, None, :], lse, 0.0))


def _plain_compact(s):
    page, A = s["case"]["page"], s["case"]["A"]
    i = torch.arange(A, device=s["ctx"].device)[None, :]
    live = i < s["lens"][:, None]
    ctx, table = s["ctx"].long()[:, None], s["table"].long()
    src, dst = ctx + torch.where(live, s["path"].long(), 0), ctx + torch.where(live, i, 0)
    src = (torch.gather(table, 1, src // page) * page + src % page).flatten()
    dst = (torch.gather(table, 1, dst // page) * page + dst % page).flatten()
    k, v = s["k_pages"].flatten(1, 2), s["v_pages"].flatten(1, 2)
    k.index_copy_(1, dst, k[:, src])
    v.index_copy_(1, dst, v[:, src])
    return dict(k=s["k_pages"], v=s["v_pages"])


# ------------------------------------------------------------------------------------- measures

def work(case):
    op, B = case["op"], case["B"]
    if op == "page_plan":
        # Lengths in and out, the slot map, and about the pages that change hands.
        return dict(bytes=4.0 * (5 * B + B * case["T"] + 4 * B * (1 + case["T"] / 2 / case["page"])), flops=0)
    if op == "tree_plan":
        return dict(bytes=4.0 * B * (1 + case["T"] * (2 + (case["T"] + 31) // 32)), flops=0)
    if op == "kv_append":
        rows, e = sum(_lens(case)), 2 if case["dtype"] == "bf16" else 4
        heads = case["Hq"] + 2 * case["Hkv"]
        return dict(bytes=float(rows * (2 * heads * case["d"] * e + 4)),
                    flops=4.0 * rows * (case["Hq"] + case["Hkv"]) * case["d"] if case["norm"] else 0)
    if op == "tree_attn":
        Hq, Hkv, d, W = (case[k] for k in ("Hq", "Hkv", "d", "window"))
        ctx, lens = _ctx(case), _lens(case)
        seen = [min(c, W - 1) if W > 0 else c for c in ctx]
        keys = sum(x + n for x, n in zip(seen, lens))
        pairs = sum(n * (x + 1) for x, n in zip(seen, lens))
        return dict(bytes=float(4 * keys * Hkv * d + sum(lens) * Hq * (4 * d + 8)), flops=4.0 * d * Hq * pairs)
    moved = sum(b % case["A"] for b in range(B))
    return dict(bytes=float(2 * 2 * 2 * case["L"] * moved * case["Hkv"] * case["d"] + 4 * B * (2 + case["A"])), flops=0)


def exact(case, seed):
    op = case["op"]
    if op not in ("kv_append", "tree_attn"):
        return None          # whole numbers, or values that are moved
    s = prepare(case, seed)
    if op == "kv_append":
        B, T, Hq, Hkv, d = (case[k] for k in ("B", "T", "Hq", "Hkv", "d"))
        x = s["qkv"].view(B * T, Hq + 2 * Hkv, d).double()
        q_out, k_pages, v_pages = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
        slot = s["slots"].view(-1).long()
        rows = torch.nonzero(slot >= 0).view(-1)
        x, slot = x[rows], slot[rows]
        if case["norm"]:
            size = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            gain = torch.ones(Hq + 2 * Hkv, d, dtype=torch.float64, device=x.device)
            gain[:Hq], gain[Hq:Hq + Hkv] = s["wq"].double(), s["wk"].double()
            size[:, Hq + Hkv:] = 1.0
            x = x / size * gain
        q_out.view(B * T, Hq, d)[rows] = x[:, :Hq]
        k_pages.view(-1, Hkv, d)[slot] = x[:, Hq:Hq + Hkv]
        v_pages.view(-1, Hkv, d)[slot] = x[:, Hq + Hkv:]
        return dict(q=q_out, k=k_pages, v=v_pages)
    B, T, Hq, Hkv, d, page, W, R = (case[k] for k in ("B", "T", "Hq", "Hkv", "d", "page", "window", "R"))
    G = Hq // Hkv
    o = torch.zeros(B, T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, T, dtype=torch.float64, device="cuda")
    words = s["mask"].cpu().numpy().view(np.uint32)
    for b, (c, n) in enumerate(zip(_ctx(case), _lens(case))):
        first = max(0, c - W + 1) if W > 0 else 0
        j = torch.arange(first, c + n, device="cuda")
        slot = s["table"][b].long()[j // page] * page + j % page
        dep = s["depth"][b, :n].long()
        kpos = torch.cat([j[:c - first], c + dep])
        delta = (c + dep)[:, None] - kpos[None, :]
        sees = torch.ones(n, c - first + n, dtype=torch.bool)
        for t in range(n):
            for u in range(n):
                sees[t, c - first + u] = bool((int(words[b, t, u // 32]) >> (u % 32)) & 1)
        sees = sees.cuda() & (delta >= 0) & (delta < (W if W > 0 else 1 << 62))
        tau = torch.ones(n, dtype=torch.float64, device="cuda")
        if case["temp_n0"] > 1:
            count = (c + dep + 1).double()
            if W > 0:
                count = torch.minimum(count, torch.full_like(count, W))
            tau = torch.maximum(tau, torch.log(count) / math.log(case["temp_n0"]))
        for g in range(Hkv):
            k = s["k_pages"].view(-1, Hkv, d)[slot, g].double()
            v = s["v_pages"].view(-1, Hkv, d)[slot, g].double()
            for h in range(g * G, (g + 1) * G):
                a = s["q"][b, :n, h].double() @ k.T * s["scale"]
                reach = (delta >= 0) & (delta < R)
                a = a + reach * s["r"][b, :n, h].double()[:, None] * s["w"][h].double()[delta.clamp(0, R - 1)]
                a = (a * tau[:, None]).masked_fill(~sees, -math.inf)
                z = torch.logsumexp(a, 1)
                o[b, :n, h] = torch.exp(a - z[:, None]) @ v
                lse[b, h, :n] = z
    return dict(o=o, lse=lse)
