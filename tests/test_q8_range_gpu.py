"""The 8-bit cache's decode where numbers of very different sizes meet:
against the definition in 64 bits, within the bounds that
tests/q8_reference.py derives."""
import pytest
import torch

import decoder_only_transformer_sdpa_b200 as A
from tests.test_q8_gpu import check_decode, dev, filled, queries, sequences, status, tokens

pytestmark = pytest.mark.gpu


# ------------------------------------- products of queries and keys near zero


@pytest.mark.parametrize("D,G,tq", [(64, 1, 1), (32, 3, 3), (64, 5, 4), (128, 2, 8)])
@pytest.mark.parametrize("qs,ks", [(1e-20, 1e-20), (1e-30, 1e-30), (1e-3, 1e-36), (1.5, 5e-39), (1e-38, 1.0)])
def test_decode_products_that_vanish(D, G, tq, qs, ks):
    """Scores that float32 holds as next to nothing, or not at all, are next to nothing: every token counts alike."""
    lens = (500, 70)
    k, v = tokens(31 + D, 2, 2, 500, D)
    k = (k.float() * ks).to(torch.bfloat16)
    c, L = filled(k, v, lens)
    q = (queries(2, 2, 2 * G, tq, D).float() * qs).to(torch.bfloat16)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, weight="set")
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, lens), lens, weight=c.weight.double().cpu().numpy(), label=f"{qs} {ks}")


@pytest.mark.parametrize("D,G,tq", [(64, 1, 1), (32, 9, 2), (64, 5, 4), (128, 1, 1)])
@pytest.mark.parametrize("qs,ks,tiny", [(1.0, 1.0, 5e-39), (1e-20, 1e20, 1e-20), (1e-8, 1e8, 1e-33), (1.0, 1.0, 0.0)])
def test_decode_blocks_of_tiny_keys_among_others(D, G, tq, qs, ks, tiny):
    lens = (64 * 9 + 11, 64 * 5)
    k, v = tokens(41 + D, 2, 2, max(lens), D)
    size = torch.full((max(lens), 1), ks)
    size[64 * 2:64 * 3] = size[64 * 4:64 * 5] = tiny
    k = (k.float() * size).to(torch.bfloat16)
    c, L = filled(k, v, lens)
    q = (queries(3, 2, 2 * G, tq, D).float() * qs).to(torch.bfloat16)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, weight="set")
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, lens), lens, weight=c.weight.double().cpu().numpy(), label=f"{qs} {ks} {tiny}")
    blocks = torch.tensor([1, 2, 4], dtype=torch.int32).expand(2, 2, tq, 3).contiguous()
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=blocks.to(dev()))
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, lens), lens, lists=blocks.numpy(), label=f"lists {qs} {ks} {tiny}")
