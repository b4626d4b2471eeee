"""Batches whose (sequence, key/value head) pairs are as many as the SMs, and one of whose
sequences is much longer than the others: results, and that the long one is shared out."""
import pytest
import torch

from attention_learned_relative_b200 import ops
from test_gpu_tree_attn import check, make

pytestmark = pytest.mark.gpu


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("d,Hq,Hkv,T,window", [(64, 8, 4, 3, 0), (128, 16, 2, 20, 0), (64, 8, 4, 5, 1900)])
def test_one_long_sequence_among_as_many_segments_as_sms(d, Hq, Hkv, T, window):
    ops.device_status(reset=True)
    B = _sms() // Hkv
    ctxs = [4000 if b == B // 2 else 30 + 7 * b for b in range(B)]
    check(make(ctxs, [T - b % 2 for b in range(B)], T, Hq, Hkv, d, 32, window, 64, seed=B), what="ragged")
    assert ops.device_status(reset=True) == 0


def _time(ctxs, T, Hq, Hkv, d, page):
    """Microseconds of a call on caches of these lengths: the least of six, from the device's clock."""
    B, blocks = len(ctxs), -(-(max(ctxs) + T) // page)
    need = [-(-(c + T) // page) for c in ctxs]
    table, at = torch.zeros(B, blocks, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    i32 = dict(dtype=torch.int32, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros(at, page, Hkv, d, **bf16), torch.zeros(at, page, Hkv, d, **bf16)
    q, r, w = torch.zeros(B, T, Hq, d, **bf16), torch.zeros(B, T, Hq, device="cuda"), torch.zeros(Hq, 64, device="cuda")
    lens = torch.full((B,), T, **i32)
    depth, mask = ops.tree_plan(torch.arange(-1, T - 1, **i32).repeat(B, 1), lens)
    args = (q, k, v, table.cuda(), torch.tensor(ctxs, **i32), lens, depth, mask, r, w, 0, 64, max(ctxs))
    best = float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        ops.attn_tree_paged(*args)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def test_a_long_sequence_is_shared_out_whatever_the_batch():
    """One sequence of 65536 rows among short ones: the call takes at most three times as long
    as one on the same rows spread evenly (an SM that walks the long one's key tiles of a head
    alone takes eight times as long and more)."""
    Hkv = 4
    B = _sms() // Hkv
    ragged = [65536] + [1000] * (B - 1)
    even = [sum(ragged) // B] * B
    t_ragged, t_even = _time(ragged, 16, 32, Hkv, 128, 64), _time(even, 16, 32, Hkv, 128, 64)
    assert t_ragged <= 3 * t_even, (t_ragged, t_even)


@pytest.mark.parametrize("R,temp_n0", [(32, 0), (12000, 500)])
def test_more_parts_than_a_warp_has_lanes(R, temp_n0):
    """One cache head of 12000 rows is a key tile to a CTA: 94 parts, so that a lane of the
    combine merges several, with the bias near the end only and over all parts."""
    ops.device_status(reset=True)
    for T in (2, 70):   # one row tile, and two
        check(make([12000], [T], T, 2, 1, 64, 64, 0, R, seed=R), temp_n0=temp_n0, what="94 parts")
    assert ops.device_status(reset=True) == 0


def test_a_sequence_alone_and_in_a_batch():
    """Where segments are cut depends on the batch, so bits may differ; both answers are within
    the bound of the exact one."""
    ops.device_status(reset=True)
    args = (16, 32, 4, 128, 32)
    ctxs, lens = [900, 200, 31], [16, 9, 16]
    for window in (0, 100):
        x = make(ctxs, lens, *args, window, 128, seed=3)
        check(x, what="batch")
        for b in range(3):
            y = dict(x, ctxs=ctxs[b:b + 1], lens=lens[b:b + 1], q=x["q"][b:b + 1].contiguous(),
                     r=x["r"][b:b + 1].contiguous(), table=x["table"][b:b + 1].contiguous(), ks=x["ks"][b:b + 1],
                     vs=x["vs"][b:b + 1], depth=x["depth"][b:b + 1], anc=x["anc"][b:b + 1])
            check(y, what="alone")
    assert ops.device_status(reset=True) == 0
