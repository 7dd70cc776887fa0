"""The 8-bit cache's calls as torch sees them: outputs made through the
dispatcher, and queries that require gradients."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import decoder_only_transformer_sdpa_b200 as A
from tests.test_q8_gpu import dev, filled, queries, status, tokens

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.tensors = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        self.tensors.append((func, out))
        return out


def test_dispatch_modes_see_the_outputs():
    k, v = tokens(1, 1, 2, 300, 64)
    c, L = filled(k, v, (300,))
    q = queries(1, 1, 2, 1, 64).to(dev())
    for call, outputs in ((lambda: A.attn_q8_decode(q, c, L, weight="set"), 2), (lambda: (A.attn_q8_select(q, c, L, 2),), 1),
                          (lambda: A.attn_q8_read(c, L, 300), 2), (lambda: A.attn_q8_evict(c, L, 3), 2)):
        with Seen() as mode:
            got = call()
        assert len(got) == outputs
        for t in got:
            assert any(x is t or (isinstance(x, torch.Tensor) and x.data_ptr() == t.data_ptr()) for _, x in mode.tensors)
        assert all(f is torch.ops.aten.empty.memory_format for f, _ in mode.tensors)
    assert status() == 0


def test_outputs_in_inference_mode_and_of_queries_with_gradients():
    """As attn_decode: the outputs carry no graph."""
    k, v = tokens(2, 1, 2, 100, 64)
    c, L = filled(k, v, (100,))
    q = queries(2, 1, 2, 1, 64).to(dev())
    want = A.attn_q8_decode(q, c, L)
    for o, lse in (A.attn_q8_decode(q.clone().requires_grad_(), c, L), A.attn_decode(q.clone().requires_grad_(), k.to(dev()), v.to(dev()))):
        assert not o.requires_grad and not lse.requires_grad and o.grad_fn is None
    with torch.inference_mode():
        o, lse = A.attn_q8_decode(q, c, L)
        assert o.is_inference() and lse.is_inference()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and status() == 0
