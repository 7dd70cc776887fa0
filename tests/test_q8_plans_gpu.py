"""The 8-bit cache's choice of blocks where its launch plan changes: lists that
take clusters of eight CTAs down to one, and more lists than the GPU has SMs."""
import pytest
import torch

import decoder_only_transformer_sdpa_b200 as A
from tests import q8_reference as R
from tests.test_q8_gpu import dev, status

pytestmark = pytest.mark.gpu


def leveled(B, H, D, lens, seed=0):
    """A cache whose block j of a head scores level[b, h, j] * sum(q) for queries of equal channels."""
    blocks = max(lens) // 64
    c = A.Q8Cache.empty(B, H, D, 64 * blocks, device=dev())
    level = torch.randint(0, 100, (B, H, blocks), generator=torch.Generator().manual_seed(seed))
    c.bounds[:, :, :, 1] = level[..., None].to(torch.int8).to(dev())
    c.scales[..., 0] = 1.0
    return c, level, torch.tensor(lens, dtype=torch.int32, device=dev())


@pytest.mark.parametrize("D,B,H,tq", [(64, 3, 4, 1), (64, 4, 12, 1), (64, 2, 37, 1), (128, 5, 15, 1), (64, 4, 37, 1),
                                      (64, 149, 1, 1), (32, 8, 12, 4), (128, 3, 50, 2)])
@pytest.mark.parametrize("blocks", [300, 2100])
def test_select_from_few_lists_to_many(D, B, H, tq, blocks):
    lens = [64 * (blocks - 5 * b % blocks) + b % 64 for b in range(B)]
    lens[B // 2] = 0
    c, level, L = leveled(B, H, D, lens, seed=blocks + B)
    q = torch.ones(B, H, tq, D, dtype=torch.bfloat16, device=dev())
    for n in (1, 64, 290):
        got = A.attn_q8_select(q, c, L, n).cpu()
        assert status() == 0
        for b in range(B):
            for h in range(H if b < 3 else 1):
                want = R.best_of(level[b, h, :lens[b] // 64].numpy(), n)
                for r in range(tq):
                    assert got[b, h, r].tolist() == want, (b, h, r, n)
