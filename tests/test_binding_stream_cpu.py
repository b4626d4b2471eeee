"""The `stream` argument of the serving-step calls, in every way of passing the others."""
from types import SimpleNamespace

import pytest
import torch

from attention_learned_relative_b200 import ops


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _f(*shape):
    return torch.zeros(shape)


# Keywords in an order that begins with something other than a tensor.
CALLS = [
    (ops.page_plan, dict(page_size=16, T=4, slots=None, ctx_lens=_i(3), new_lens=_i(3), num_blocks=_i(3),
                         block_table=_i(3, 4), free_ring=_i(9), ring_state=_i(2))),
    (ops.tree_plan, dict(depth=None, mask=None, parents=_i(2, 8), tree_lens=_i(2))),
    (ops.kv_append, dict(eps=1e-6, q=None, k=_f(4, 2, 64), v=_f(4, 2, 64), slots=_i(4), k_pages=_f(3, 16, 2, 64),
                         v_pages=_f(3, 16, 2, 64))),
    (ops.attn_tree_paged, dict(window=0, R=16, max_ctx_len=10, w=None, q=_f(2, 4, 8, 64), k_pages=_f(6, 16, 2, 64),
                               v_pages=_f(6, 16, 2, 64), block_table=_i(2, 3), ctx_lens=_i(2), tree_lens=_i(2),
                               depth=_i(2, 4), mask=_i(2, 4, 1), r=_f(2, 4, 8))),
]


@pytest.mark.parametrize("fn,kw", CALLS, ids=lambda x: getattr(x, "__name__", ""))
def test_keywords_in_any_order(fn, kw):
    """The stream's device is compared with the first tensor's, wherever it stands."""
    stream = SimpleNamespace(device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="the stream is not on the tensors' device"):
        fn(**kw, stream=stream)
