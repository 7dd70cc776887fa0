"""The 8-bit cache's decode where numbers of very different sizes meet, and over
lists out of order: against the definition in 64 bits, within the bounds that
tests/q8_reference.py derives."""
import numpy as np
import pytest
import torch

import decoder_only_transformer_sdpa_b200 as A
from tests import q8_reference as R
from tests.test_q8_gpu import E_LENGTH, check_decode, dev, filled, queries, sequences, status, tokens

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


# ------------------------------ one token far above the others, worth nothing


def sink(D, rows_q, n, at, gap, seed=0):
    """One key head: token `at` has the score `gap` and the value 0, the others' scores lie around 0 and their values
    around exp(gap), up to 10^26. Queries [1, Hq, Tq, D], to be used with scale 1."""
    k, v = (torch.randn(1, 1, n, D, generator=torch.Generator().manual_seed(seed + i)) for i in range(2))
    k[..., 0] = 0
    k[0, 0, at] = 0
    k[0, 0, at, 0] = gap / 8
    v = v * min(float(np.exp(gap)), 1e26)
    v[0, 0, at] = 0
    q = queries(seed, 1, *rows_q, D, scale=D**-0.5)
    q[..., 0] = 8
    return k.to(torch.bfloat16), v.to(torch.bfloat16), q


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("rows_q", [(1, 1), (3, 4), (20, 1), (5, 8)])
@pytest.mark.parametrize("gap", [12.0, 16.0, 20.0, 24.0, 32.0, 48.0, 80.0])
def test_decode_tokens_far_below_one_without_a_value(D, rows_q, gap):
    """What the softmax leaves to the other tokens is all of the output."""
    n = 64 * 11 + 5
    for at in (3, 64 * 6 + 63, n - 1):
        k, v, q = sink(D, rows_q, n, at, gap)
        for room in (n, 64 * 16000):  # in clusters, and in runs
            c, L = filled(k, v, (n,), max_tokens=room)
            o, lse = A.attn_q8_decode(q.to(dev()), c, L, scale=1.0, weight="set")
            assert status() == 0
            check_decode(q, o, lse, sequences(k, v, (n,)), (n,), scale=1.0, weight=c.weight.double().cpu().numpy(),
                         label=f"gap {gap} at {at} room {room}")


@pytest.mark.parametrize("D", [64, 128])
def test_decode_scores_at_many_distances(D):
    """Every power of e from 0 to -80 below the largest, in each block, and a value's size that makes each count."""
    n = 64 * 8
    k, v = torch.zeros(1, 1, n, D), torch.zeros(1, 1, n, D)
    far = (torch.arange(n) * 7 % 81).float()
    k[0, 0, :, 0] = -far
    v[0, 0] = torch.randn(n, D, generator=torch.Generator().manual_seed(7))
    v[0, 0, far < 40] = 0  # the largest that counts is e^-40 of the whole
    k, v = k.to(torch.bfloat16), (v * 1e17).to(torch.bfloat16)
    c, L = filled(k, v, (n,))
    q = torch.zeros(1, 2, 2, D, dtype=torch.bfloat16)
    q[:, :, :, 0] = 1.0
    q[:, 1] = 0.5
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, scale=1.0)
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, (n,)), (n,), scale=1.0, label="many distances")


# ----------------------------------------------------- very large and small values


@pytest.mark.parametrize("size,n,room", [(1e30, 102409, 102409), (1e30, 102409, 64 * 30000), (1e30, 50, 50), (1e-30, 500, 500),
                                         (1e-33, 500, 64 * 16000), (1e-35, 700, 700)])
@pytest.mark.parametrize("D", [32, 128])
def test_decode_values_near_the_ends_of_float32(D, size, n, room):
    """Sums over many tokens of one weight stay finite, and small values keep their bits."""
    if D == 128 and n > 1000:
        n = room = 64 * 700 + 9
    g = torch.Generator().manual_seed(5)
    k = (torch.randn(1, 1, n, D, generator=g) * 0.1).to(torch.bfloat16)
    v = ((torch.rand(1, 1, n, D, generator=g) / 2 + 0.5) * size).to(torch.bfloat16)
    c, L = filled(k, v, (n,), max_tokens=room)
    q = queries(8, 1, 2, 1, D, scale=0.1)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L)
    assert status() == 0
    s = sequences(k, v, (n,))[0][0]
    for h in range(2):
        row = q[0, h, 0].double().numpy()
        eo, el, _, a_max, s_max, pv = R.attend(row, s.held_k, s.held_v, np.ones(n, bool), D**-0.5)
        to, tl, _ = R.tolerances(D, s.closed, D**-0.5, row, s.held_k, a_max, s_max, eo, el, pv)
        assert np.all(np.abs(o[0, h, 0].double().cpu().numpy() - eo) <= to - 1e-30 + 2.0**-133)  # (the smallest bf16)
        assert abs(float(lse[0, h, 0]) - el) <= tl


@pytest.mark.parametrize("D", [32, 64, 128])
def test_lse_of_equal_scores(D):
    """n scores of zero: lse = log n. Rounded are log2 (one unit of its result, 2^-23 of it at most), the product with
    ln 2 and ln 2 itself (2^-24 and 2^-25), and the sum of exp2's (2^-22 each, and so of the sum)."""
    lens = [*range(1, 40), 63, 64, 65, 100, 127, 128, 500, 777, 1000, 3000]
    c = A.Q8Cache.empty(len(lens), 1, D, max(lens), device=dev())
    o, lse = A.attn_q8_decode(torch.zeros(len(lens), 1, 1, D, dtype=torch.bfloat16, device=dev()), c,
                              torch.tensor(lens, dtype=torch.int32, device=dev()))
    assert status() == 0 and (o == 0).all()
    want = np.log(np.array(lens, np.float64))
    err = np.abs(lse[:, 0, 0].double().cpu().numpy() - want)
    assert np.all(err <= 2.0**-22 * (1 + want)), list(zip(lens, err / (2.0**-22 * (1 + want))))


# ------------------------------------------------------ lists out of order


def taken(given, closed):
    """The entries that count: closed blocks above every one before them, up to the first negative entry."""
    out = []
    for x in given:
        if x < 0:
            break
        if x < closed and (not out or x > out[-1]):
            out.append(x)
    return out


@pytest.mark.parametrize("D,G", [(64, 1), (32, 9), (128, 20)])
def test_sparse_entries_count_once_whatever_came_before_them(D, G):
    closed = 40
    n = 64 * closed + 9
    k, v = tokens(14 + D, 1, 1, n, D)
    q = queries(6, 1, G, 2, D)
    seqs = sequences(k, v, (n,))
    g = np.random.default_rng(5)
    lists = [[3, 5, 4, 5], [0, 7, 2, 7, 7, 3, 8], [39, 0, 1, 2, 39], [41, 3, 3, 4], [-1, 3, 4, 5], [2, -1, 3, -1, 4],
             [5, -7, 6], [9] * 11, [*range(20), *range(10, 30)], [1, 2**31 - 1, 2, 40, 3], [*range(40), 40, 41, *range(40)],
             [int(x) for x in g.integers(0, 44, 300)], [*range(0, 40, 2)] + [-1] * 200 + [5]]
    for room in (closed + 1, 20000):  # in clusters, and (long lists) in runs
        c, L = filled(k, v, (n,), max_tokens=64 * room)
        for given in lists:
            width = max(len(given), 4, 30000 if room > 1000 else 0)
            both = torch.full((1, 1, 2, width), -1, dtype=torch.int32)
            both[0, 0, 0, :len(given)] = torch.tensor(given, dtype=torch.int64).int()
            both[0, 0, 1, :4] = torch.tensor([0, 1, 30, 39])  # another token's list in order
            o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=both.to(dev()))
            assert status() == E_LENGTH, given
            want = np.full((1, 1, 2, closed), -1)
            counts = taken(given, closed)
            want[0, 0, 0, :len(counts)] = counts
            want[0, 0, 1, :4] = [0, 1, 30, 39]
            check_decode(q, o, lse, seqs, (n,), lists=want, label=str(given[:12]))
        o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=torch.arange(40, dtype=torch.int32).expand(1, 1, 2, 40).contiguous().to(dev()))
        assert status() == 0
        check_decode(q, o, lse, seqs, (n,), label="every block")
