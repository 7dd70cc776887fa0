"""The 8-bit block cache on the GPU against its definition in 64 bits
(tests/q8_reference.py): what an append holds bit by bit, the attention within
bounds derived there, the choice of blocks and evictions exactly."""
import sys

import numpy as np
import pytest
import torch

import decoder_only_transformer_sdpa_b200 as A
from tests import q8_reference as R

pytestmark = pytest.mark.gpu

E_LENGTH = -12
NAN, INF = float("nan"), float("inf")


def dev():
    return torch.device("cuda", 0)


def tokens(seed, B, H, n, D, scale=1.0):
    """k, v [B, H, n, D] bf16 on the CPU, with a strong channel and a few strong tokens."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, H, n, D, generator=g) * scale for _ in range(2))
    k[..., D // 3] *= 4
    if n > 2:
        k[:, :, n // 2] *= 3
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def filled(k, v, lens, max_tokens=None, poison=True):
    """A cache with the first lens[b] tokens of each sequence, appended as one padded batch.  With `poison`, what
    is not written holds NaN and garbage."""
    B, H, n, D = k.shape
    c = A.Q8Cache.empty(B, H, D, max_tokens or max(n, 1), device=dev())
    if poison:
        for t in (c.recent_k, c.recent_v, c.scales, c.weight):
            t.fill_(NAN)
        c.k_codes.fill_(77)
        c.v_codes.fill_(200)
        c.bounds.fill_(99)
    L = ints(*lens)
    A.attn_q8_append(c, k.to(dev()), v.to(dev()), L, L)
    return c, L


def sequences(k, v, lens):
    B, H = k.shape[:2]
    return [[R.Sequence(k[b, h, :lens[b]].double().numpy(), v[b, h, :lens[b]].double().numpy()) for h in range(H)]
            for b in range(B)]


def status():
    torch.cuda.synchronize()
    return A.attn_device_error()


def check_held(c, seqs, recents=True):
    """The cache holds exactly what the definition says (codes, scales, bounds, recent positions)."""
    S = min(c.D, 64)
    kc = c.k_codes.cpu().numpy().transpose(0, 1, 2, 4, 3, 5).reshape(c.B, c.H, c.blocks, 64, c.D)
    vc = c.v_codes.cpu().numpy().transpose(0, 1, 2, 4, 3)
    sc, bo = c.scales.cpu().numpy(), c.bounds.cpu().numpy()
    rk, rv = (t.double().cpu().numpy() for t in (c.recent_k, c.recent_v))
    assert S * (c.D // S) == c.D
    for b in range(c.B):
        for h in range(c.H):
            s = seqs[b][h]
            for j in range(s.closed):
                np.testing.assert_array_equal(kc[b, h, j], s.k_codes[j], f"keys {b} {h} {j}")
                np.testing.assert_array_equal(vc[b, h, j], s.v_codes[j], f"values {b} {h} {j}")
                np.testing.assert_array_equal(sc[b, h, j], np.array(s.scales[j], np.float32), f"scales {b} {h} {j}")
            if s.closed:
                np.testing.assert_array_equal(bo[b, h, :s.closed], s.bounds())
            if recents:
                for p in range(max(0, (s.closed - 1) * 64), len(s.k)):
                    np.testing.assert_array_equal(rk[b, h, p % 128], s.k[p], f"recent key {b} {h} {p}")
                    np.testing.assert_array_equal(rv[b, h, p % 128], s.v[p], f"recent value {b} {h} {p}")


def check_decode(q, o, lse, seqs, lens, scale=None, lists=None, weight=None, label=""):
    """o, lse (and the blocks' weights) of queries q [B, Hq, Tq, D] against the definition, within its bounds."""
    B, Hq, Tq, D = q.shape
    H = len(seqs[0])
    G = Hq // H
    scale = D**-0.5 if scale is None else scale
    q = q.double().cpu().numpy()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        L = lens[b]
        for h in range(H):
            s = seqs[b][h]
            got = np.zeros(L)
            loosest = 0.0
            for g in range(G):
                for r in range(Tq):
                    use = np.arange(L) <= L - Tq + r
                    if lists is not None:
                        some = np.zeros(L, bool)
                        for j in lists[b, h, r]:
                            if j >= 0:
                                some[64 * j:64 * j + 64] = True
                        some[64 * s.closed:] = True
                        use &= some
                    row = q[b, h * G + g, r]
                    eo, el, p, a_max, s_max, pv = R.attend(row, s.held_k, s.held_v, use, scale)
                    to, tl, tw = R.tolerances(D, s.closed, scale, row, s.held_k, a_max, s_max, eo, el if np.isfinite(el) else 0.0, pv)
                    here = f"{label} b={b} h={h} g={g} r={r} L={L}"
                    if not use.any():
                        assert np.all(o[b, h * G + g, r] == 0) and lse[b, h * G + g, r] == -np.inf, here
                        continue
                    err = np.abs(o[b, h * G + g, r] - eo)
                    assert np.all(err <= to), f"{here} o: {np.max(err / to):.3g} of the bound"
                    dl = abs(lse[b, h * G + g, r] - el)
                    assert dl <= tl, f"{here} lse: {dl:.3g} over {tl:.3g}"
                    got += p
                    loosest = max(loosest, tw)
            if weight is not None:
                for j in range(s.closed):
                    want = got[64 * j:64 * j + 64].sum()
                    assert abs(weight[b, h, j] - want) <= loosest * want + 1e-30, (label, b, h, j, weight[b, h, j], want)


def queries(seed, B, Hq, Tq, D, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Hq, Tq, D, generator=g) * scale).to(torch.bfloat16)


# ------------------------------------------------------------------- append


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lens", [(1,), (63, 64), (65, 0, 127), (128, 129), (200, 1, 333)])
def test_append_padded_prompts(D, lens):
    k, v = tokens(sum(lens) + D, len(lens), 2, max(lens), D)
    c, L = filled(k, v, lens)
    assert status() == 0
    check_held(c, sequences(k, v, lens))


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("steps", [(1,) * 70, (63, 1, 1, 63, 1), (5, 16, 60, 130, 3, 64, 64), (300, 20)])
def test_append_in_pieces_holds_what_one_append_does(D, steps):
    n = sum(steps)
    k, v = tokens(n + D, 2, 3, n, D)
    c = A.Q8Cache.empty(2, 3, D, n, device=dev())
    at = 0
    for m in steps:
        at += m
        A.attn_q8_append(c, k[:, :, at - m:at].contiguous().to(dev()), v[:, :, at - m:at].contiguous().to(dev()),
                         ints(at, at))
    assert status() == 0
    check_held(c, sequences(k, v, (n, n)))


def test_append_ragged_new_tokens_touches_nothing_else():
    """Sequences take 0 .. n of the n rows; one that takes none, blocks that do not close and rows of the recent
    positions that are not new stay as they were, bit by bit."""
    B, H, D, n = 4, 2, 64, 70
    before = (10, 100, 63, 190)
    new = (0, 70, 1, 33)
    k, v = tokens(3, B, H, 400, D)
    c, _ = filled(k, v, before, max_tokens=400)
    old = {x: getattr(c, x).clone() for x in ("k_codes", "v_codes", "scales", "bounds", "weight", "recent_k", "recent_v")}
    after = tuple(x + y for x, y in zip(before, new))
    kn, vn = torch.zeros(2, B, H, n, D, dtype=torch.bfloat16)
    for b in range(B):
        kn[b, :, :new[b]], vn[b, :, :new[b]] = k[b, :, before[b]:after[b]], v[b, :, before[b]:after[b]]
    kn[:, :, 69], vn[2, :, 1:], kn[3, :, 33:] = NAN, NAN, NAN
    kn[1, :, 69] = k[1, :, 169]
    A.attn_q8_append(c, kn.to(dev()), vn.to(dev()), ints(*after), ints(*new))
    assert status() == 0
    check_held(c, sequences(k, v, after))
    same = lambda x, y: torch.equal(x.flatten().repeat(1).view(torch.uint8), y.flatten().repeat(1).view(torch.uint8))
    for name, t in old.items():
        now = getattr(c, name)
        assert same(now[0], t[0]), name
        if name not in ("recent_k", "recent_v"):
            for b in range(B):
                was, is_ = before[b] // 64, after[b] // 64
                assert same(now[b, :, :was], t[b, :, :was]) and same(now[b, :, is_:], t[b, :, is_:]), (name, b)
                if name == "weight":
                    assert torch.all(now[b, :, was:is_] == 0)
        else:
            for b in range(B):
                fresh = {p % 128 for p in range(max(before[b], (after[b] // 64 - 1) * 64), after[b])}
                rest = [i for i in range(128) if i not in fresh]
                assert same(now[b, :, rest], t[b, :, rest]), (name, b)


def test_append_from_packed_projection():
    """k and v are slices of a [B, T, 3 C] projection; the result is that of contiguous tensors."""
    B, H, T, D = 2, 3, 150, 64
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn(B, T, 3 * H * D, generator=g).to(torch.bfloat16).to(dev())
    k, v = (qkv[:, :, i * H * D:(i + 1) * H * D].view(B, T, H, D).permute(0, 2, 1, 3) for i in (1, 2))
    c = A.Q8Cache.empty(B, H, D, T, device=dev())
    A.attn_q8_append(c, k, v, ints(T, T))
    assert status() == 0
    check_held(c, sequences(k.cpu(), v.cpu(), (T, T)))


def test_append_ties_zeros_and_extremes():
    """Half-way numbers go to even codes; a block of zeros, of the smallest and of the largest numbers."""
    D = 64
    x = torch.zeros(1, 1, 5 * 64, D)
    x[0, 0, 0, 0] = 2.0
    x[0, 0, :64, 1] = torch.arange(64) / 64.0      # 127 x / 2 hits halves where x = odd / 127 does not; 1 -> 63.5
    x[0, 0, 1, 2], x[0, 0, 2, 2] = 1.0, -1.0       # 63.5 -> 64, -63.5 -> -64
    x[0, 0, 3, 2], x[0, 0, 4, 2] = 0.0078125, 2.0  # 127 / 256 < 1/2
    x[0, 0, 128:192, 3] = 2.0**-133                # the smallest bf16
    x[0, 0, 192:256] = 3.3895313892515355e38       # the largest
    x[0, 0, 192:256, ::2] *= -1
    x[0, 0, 256:320] = torch.randn(64, D, generator=torch.Generator().manual_seed(1)) * 1e-20
    k = x.to(torch.bfloat16)
    v = -k
    c, _ = filled(k, v, (320,))
    assert status() == 0
    check_held(c, sequences(k, v, (320,)))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_append_non_finite_block_reads_as_nan(bad):
    k, v = tokens(5, 1, 2, 200, 64)
    k[0, 0, 70, 3] = bad
    v[0, 1, 130, 60] = bad
    c, L = filled(k, v, (200,))
    rk, rv = A.attn_q8_read(c, L, 200)
    assert status() == 0
    check_held(c, sequences(k, v, (200,)))
    assert torch.isnan(rk[0, 0, 64:128]).all() and torch.isfinite(rk[0, 1]).all() and torch.isfinite(rk[0, 0, 128:]).all()
    assert torch.isnan(rv[0, 1, 128:192]).all() and torch.isfinite(rv[0, 0]).all()
    q = queries(1, 1, 2, 1, 64).to(dev())
    o, lse = A.attn_q8_decode(q, c, L, weight="set")
    assert status() == 0
    assert torch.isnan(o[0, 0]).all() and torch.isnan(lse[0, 0]).all(), "a NaN among the keys reaches the output"
    assert torch.isnan(o[0, 1]).all() and torch.isfinite(lse[0, 1]).all()
    assert torch.isnan(c.weight[0, 0, :3]).all() and torch.isfinite(c.weight[0, 1, :3]).all()


def test_append_twice_and_taken_back():
    """An append of up to 64 tokens may be repeated, and tokens taken back to the start of the last closed block."""
    n = 300
    k, v = tokens(21, 1, 2, n, 64)
    other_k, other_v = tokens(22, 1, 2, 64, 64)
    kd, vd = k.to(dev()), v.to(dev())
    put = lambda c, x, y, at: A.attn_q8_append(c, x.contiguous(), y.contiguous(), ints(at))
    for start in (64, 100, 127, 128):
        for m in (1, 28, 64):
            c, _ = filled(k[:, :, :start], v[:, :, :start], (start,), max_tokens=n)
            put(c, other_k[:, :, :m].to(dev()), other_v[:, :, :m].to(dev()), start + m)  # drafted and refused
            back = max(start, (start + m) // 64 * 64 - 64)
            assert back == start
            for _ in range(2):
                put(c, kd[:, :, start:start + m], vd[:, :, start:start + m], start + m)
            put(c, kd[:, :, start + m:start + m + 70], vd[:, :, start + m:start + m + 70], start + m + 70)
            assert status() == 0
            check_held(c, sequences(k, v, (start + m + 70,)))


# --------------------------------------------------------------------- read


@pytest.mark.parametrize("D", [32, 64, 128])
def test_read(D):
    lens = (200, 0, 64, 129)
    k, v = tokens(D, 4, 2, 200, D)
    c, L = filled(k, v, lens)
    seqs = sequences(k, v, lens)
    for n, starts in ((200, None), (1, None), (77, (130, 0, 10, 127)), (300, (5, 7, 64, 0)), (64, (64, 64, 64, 64))):
        o = [torch.full((4, 2, n, D), NAN, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
        A.attn_q8_read(c, L, n, starts=None if starts is None else ints(*starts), k=o[0], v=o[1])
        assert status() == 0
        for b in range(4):
            for h in range(2):
                s = seqs[b][h]
                for got, held in ((o[0], s.held_k), (o[1], s.held_v)):
                    want = np.zeros((n, D))
                    s0 = starts[b] if starts else 0
                    m = max(0, min(n, lens[b] - s0))
                    # the float32 product of two numbers, rounded to bf16
                    want[:m] = R.bf16(held[s0:s0 + m].astype(np.float32))
                    np.testing.assert_array_equal(got[b, h].double().cpu().numpy(), want, f"n={n} b={b} h={h}")


# ------------------------------------------------------------------- decode


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("tq", [1, 2, 16])
@pytest.mark.parametrize("lens", [(1, 0), (15, 63), (64, 65), (80, 127), (128, 1000), (4099, 17)])
def test_decode_lengths(D, tq, lens):
    k, v = tokens(7 * sum(lens) + tq + D, 2, 2, max(lens), D)
    c, L = filled(k, v, lens)
    q = queries(tq, 2, 2, tq, D)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L)
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, lens), lens, label=f"D={D} tq={tq}")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("G,tq", [(2, 1), (3, 3), (8, 1), (8, 2), (9, 1), (16, 1), (17, 1), (64, 1), (5, 16)])
def test_decode_shared_key_heads(D, G, tq):
    lens = (300, 70)
    k, v = tokens(G + tq + D, 2, 2, 300, D)
    c, L = filled(k, v, lens)
    q = queries(G, 2, 2 * G, tq, D)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, weight="set")
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, lens), lens, weight=c.weight.double().cpu().numpy(), label=f"G={G} tq={tq}")


@pytest.mark.parametrize("B,H,n", [(1, 1, 20000), (1, 7, 3000), (40, 8, 130)])
def test_decode_from_one_to_many_heads(B, H, n):
    lens = tuple(max(0, n - 37 * b) for b in range(B))
    k, v = tokens(B + n, B, H, n, 64)
    c, L = filled(k, v, lens, max_tokens=2 * n)
    q = queries(n, B, H, 1, 64)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, weight="set")
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, lens), lens, weight=c.weight.double().cpu().numpy(), label=f"B={B} H={H}")


@pytest.mark.parametrize("D,B,H,G,tq,room", [(64, 40, 3, 1, 1, 400), (32, 70, 2, 2, 1, 400), (128, 5, 1, 12, 3, 4000),
                                             (64, 3, 2, 1, 16, 4000), (64, 33, 1, 20, 1, 700), (64, 2, 2, 1, 2, 9000)])
def test_decode_shared_out_by_the_lengths(D, B, H, G, tq, room):
    """Caches with room for so much that CTAs take equal runs of all blocks: very unequal lengths, empty sequences at
    the start, in the middle and at the end, more sequences than a warp has lanes, several row tiles, weights."""
    lens = [(0, 1, 63, 64, 65, 700, 200, 1500, 0, 129)[(b + B) % 10] for b in range(B)]
    k, v = tokens(B + D, B, H, 1500, D)
    c, L = filled(k, v, lens, max_tokens=64 * room)
    q = queries(B, B, H * G, tq, D)
    seqs = sequences(k, v, lens)
    for weight in (None, "set"):
        o, lse = A.attn_q8_decode(q.to(dev()), c, L, weight=weight)
        assert status() == 0
        check_decode(q, o, lse, seqs, lens, weight=c.weight.double().cpu().numpy() if weight else None, label=f"runs {weight}")
    o, lse = A.attn_q8_decode(q.to(dev()), c, 0 * L)
    assert status() == 0 and (o == 0).all() and (lse == -INF).all()
    bad = L.clone()
    bad[B // 2] = 64 * room + 64
    A.attn_q8_decode(q.to(dev()), c, bad)
    assert status() == E_LENGTH
    # lists long enough for the same, mostly -1
    blocks = A.attn_q8_select(q.to(dev()), c, L, room)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=blocks)
    assert status() == 0
    lists = blocks.cpu().numpy()
    for b in range(B):
        assert all((x >= 0).sum() <= lens[b] // 64 for x in lists[b].reshape(-1, room))
    check_decode(q, o, lse, seqs, lens, label="lists of every block")


@pytest.mark.parametrize("D,G,tq", [(32, 4, 8), (64, 4, 4), (64, 2, 16), (128, 8, 1), (128, 4, 4)])
@pytest.mark.parametrize("B,room", [(31, 130), (51, 64 * 40)])
def test_decode_more_row_tiles_than_are_taken_at_once(D, G, tq, B, room):
    """Ten key heads a sequence: with short texts and, in equal runs, with long ones. Some sequences are checked."""
    H = 10
    lens = [room - (b * 37) % (room + 1) for b in range(B)]
    lens[1], lens[-2], lens[-1] = 0, 1, 64
    k, v = tokens(D + G + B, B, H, room, D)
    c, L = filled(k, v, lens)
    q = queries(B + tq, B, H * G, tq, D)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, weight="set")
    assert status() == 0
    some = [0, 1, B // 2, B - 2, B - 1] if room < 1000 else [B // 2, B - 1]
    heads = range(H) if room < 1000 else range(3, 5)
    weight = c.weight.double().cpu().numpy()
    for b in some:
        seqs = [[R.Sequence(k[b, h, :lens[b]].double().numpy(), v[b, h, :lens[b]].double().numpy()) for h in heads]]
        rows = slice(heads[0] * G, (heads[-1] + 1) * G)
        check_decode(q[b:b + 1, rows], o[b:b + 1, rows], lse[b:b + 1, rows], seqs, [lens[b]],
                     weight=weight[b:b + 1, heads[0]:heads[-1] + 1], label=f"sequence {b}")


@pytest.mark.parametrize("qs,ks,vs", [(100.0, 10.0, 1.0), (1e-3, 1e-3, 1e3), (1e10, 1e-10, 1e-20), (0.0, 1.0, 1.0),
                                      (1e-30, 1e30, 1e30), (20.0, 1.0, 0.0)])
def test_decode_magnitudes(qs, ks, vs):
    """Peaked and flat rows, and factors far from one."""
    k, v = tokens(31, 1, 2, 500, 64)
    k, v = (k.float() * ks).to(torch.bfloat16), (v.float() * vs).to(torch.bfloat16)
    c, L = filled(k, v, (500,))
    q = (queries(2, 1, 2, 3, 64).float() * qs).to(torch.bfloat16)
    q[0, 0, 0] = 0
    q[0, 1, 1, 5:] = 0
    o, lse = A.attn_q8_decode(q.to(dev()), c, L)
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, (500,)), (500,), label=f"{qs} {ks} {vs}")


def test_decode_one_heavy_and_many_light_tokens():
    """One token far above the others, which are so many that they count: their small weights are not lost."""
    n, D = 65536, 64
    k, v = torch.zeros(1, 1, n, D), torch.ones(1, 1, n, D)
    k[0, 0, 5, 0] = 8.0
    v[0, 0, 5] = -1.0
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c, L = filled(k, v, (n,))
    q = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16)
    q[0, 0, 0, 0] = 11.0  # s = 11: e^11 = 59874 against 65535
    o, lse = A.attn_q8_decode(q.to(dev()), c, L)
    assert status() == 0
    check_decode(q, o, lse, sequences(k, v, (n,)), (n,), label="heavy")


def test_decode_scale_strides_and_lent_buffers():
    B, H, tq, D, n = 2, 6, 3, 64, 190
    lens = (190, 77)
    k, v = tokens(6, B, 3, n, D)
    c, L = filled(k, v, lens)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, tq, 3 * H * D, generator=g).to(torch.bfloat16).to(dev())
    q = qkv[:, :, :H * D].view(B, tq, H, D).permute(0, 2, 1, 3)
    room = torch.full((B, tq, H, D), NAN, dtype=torch.bfloat16, device=dev())
    guard = torch.full((B * H * tq + 64,), NAN, device=dev())
    lse = guard[32:32 + B * H * tq].view(B, H, tq)
    need = A.attn_q8_decode_workspace_bytes(c, H, tq, weight="set")
    ws = torch.full((need + 512,), 171, dtype=torch.uint8, device=dev())
    o, _ = A.attn_q8_decode(q, c, L, o=room.permute(0, 2, 1, 3), lse=lse, scale=0.3, weight="set", workspace=ws[256:256 + need])
    assert status() == 0
    assert torch.isfinite(room.float()).all()
    assert torch.isnan(guard[:32]).all() and torch.isnan(guard[-32:]).all()
    assert (ws[:256] == 171).all() and (ws[256 + need:] == 171).all()
    check_decode(q.cpu(), o, lse, sequences(k, v, lens), lens, scale=0.3, weight=c.weight.double().cpu().numpy())
    with pytest.raises(A.AttnError):
        A.attn_q8_decode(q, c, L, workspace=ws[256:256 + need - 256], weight="set")


def test_decode_weights_add_up():
    lens = (300, 64, 20)
    k, v = tokens(16, 3, 2, 300, 64)
    c, L = filled(k, v, lens)
    q1, q2 = queries(1, 3, 4, 2, 64), queries(2, 3, 4, 2, 64)
    A.attn_q8_decode(q1.to(dev()), c, L, weight="set")
    w1 = c.weight.clone()
    A.attn_q8_decode(q2.to(dev()), c, L, weight="set")
    w2 = c.weight.clone()
    A.attn_q8_decode(q1.to(dev()), c, L, weight="set")
    A.attn_q8_decode(q2.to(dev()), c, L, weight="add")
    assert status() == 0
    for b, n in enumerate(lens):
        m = n // 64
        assert torch.equal(c.weight[b, :, :m], w1[b, :, :m] + w2[b, :, :m])
        assert torch.isnan(c.weight[b, :, m:]).all(), "places behind the closed blocks are left alone"


def test_decode_poison_behind_the_end_and_in_unseen_tokens():
    """NaN and infinities behind a sequence's end, and in tokens that only later queries see, reach nobody else."""
    n, D, tq = 70, 64, 4
    k, v = tokens(9, 1, 1, n, D)
    k[0, 0, 68] = INF
    v[0, 0, 69] = NAN
    v[0, 0, 68, 7] = -INF
    c, L = filled(k, v, (n,))
    q = queries(3, 1, 1, tq, D)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L)
    assert status() == 0
    short = sequences(k[:, :, :68], v[:, :, :68], (68,))
    check_decode(q[:, :, :2], o[:, :, :2], lse[:, :, :2], short, (68,), label="rows before the bad tokens")
    assert torch.isnan(o[0, 0, 3]).all(), "the row that sees the NaN is NaN"


def test_decode_infinite_value_in_the_open_block():
    k, v = tokens(10, 1, 1, 40, 64)
    v[0, 0, 11, 3], v[0, 0, 30, 9] = INF, -INF
    c, L = filled(k, v, (40,))
    o, lse = A.attn_q8_decode(queries(4, 1, 1, 1, 64).to(dev()), c, L)
    assert status() == 0
    o = o[0, 0, 0].float()
    assert o[3] == INF and o[9] == -INF and torch.isfinite(o).sum() == 62 and torch.isfinite(lse).all()


def test_decode_lengths_out_of_range_are_reported():
    lens = (100, 100)
    k, v = tokens(12, 2, 1, 100, 64)
    c, L = filled(k, v, lens)  # holds up to 2 * 64 + 63
    q = queries(5, 2, 1, 1, 64)
    for bad in (-1, 192, 2**31 - 1, -2**31):
        o, lse = A.attn_q8_decode(q.to(dev()), c, ints(100, bad))
        assert status() == E_LENGTH and status() == 0
        check_decode(q[:1], o[:1], lse[:1], sequences(k, v, lens)[:1], (100,))
        assert (o[1] == 0).all() and (lse[1] == -INF).all()
        before = c.recent_k.clone()
        A.attn_q8_append(c, k[:, :, :1].contiguous().to(dev()), v[:, :, :1].contiguous().to(dev()), ints(100, bad), ints(0, 1))
        assert status() == E_LENGTH
        assert torch.equal(before.view(torch.int16), c.recent_k.view(torch.int16))
    o, _ = A.attn_q8_decode(q.to(dev()), c, ints(191, 0))  # as long as it may be: rows never written, not out of range
    assert status() == 0
    for new in ((101, 0), (-1, 0), (2, 0)):
        A.attn_q8_append(c, k[:, :, :1].contiguous().to(dev()), v[:, :, :1].contiguous().to(dev()), ints(100, 100), ints(*new))
        assert status() == E_LENGTH
    A.attn_q8_read(c, ints(100, 100), 10, starts=ints(0, -5))
    assert status() == E_LENGTH
    A.attn_q8_select(q.to(dev()), c, ints(100, -3), 1)
    assert status() == E_LENGTH


def test_decode_cache_beyond_four_gib():
    """Offsets beyond 32 bits: the last head of a cache of 8.6 GB."""
    B, H, D, n = 2, 1, 128, 2 * 1024 * 1024 - 64
    c = A.Q8Cache.empty(B * 16, H, D, n, device=dev())
    assert c.k_codes.numel() > 2**32
    lens = [0] * (B * 16)
    lens[-1] = n + 7
    for t in (c.k_codes, c.v_codes):
        t[-1].random_(1, 256, generator=torch.Generator(device=dev()).manual_seed(4))
    c.scales[-1] = 0.01
    c.recent_k[-1], c.recent_v[-1] = 0.5, -0.25
    q = torch.zeros(B * 16, 1, 1, D, dtype=torch.bfloat16, device=dev())
    q[-1, 0, 0] = queries(4, 1, 1, 1, D)[0, 0, 0].to(dev())
    o, lse = A.attn_q8_decode(q, c, ints(*lens))
    assert status() == 0
    k = torch.cat([(c.k_codes[-1, 0].permute(0, 2, 1, 3).reshape(-1, D).double() - 128) * float(c.scales[-1, 0, 0, 0]),
                   c.recent_k[-1, 0, :7].double()])
    s = k @ q[-1, 0, 0].double() / D**0.5
    p = torch.softmax(s, 0)
    v = torch.cat([(c.v_codes[-1, 0].transpose(1, 2).reshape(-1, D).double() - 128) * float(c.scales[-1, 0, 0, 1]),
                   c.recent_v[-1, 0, :7].double()])
    want, abs_v = p @ v, p @ v.abs()
    # as in q8_reference.tolerances; a chain is 64 + 2 * 32768 / 8 additions at most
    bound = 2.0**-8 * want.abs() + (2.0**-11 + 2.0**-12 + (64 + 8192) * 2.0**-23) * abs_v
    assert ((o[-1, 0, 0].double() - want).abs() <= bound).all()
    assert abs(float(lse[-1]) - float(torch.logsumexp(s, 0))) <= 1e-4
    assert (o[:-1] == 0).all() and (lse[:-1] == -INF).all()
    r = A.attn_q8_read(c, ints(*lens), 100, starts=ints(*([0] * (B * 16 - 1)), n - 50))
    assert status() == 0
    assert torch.equal(r[0][-1, 0, :57], k[n - 50:].float().to(torch.bfloat16)) or \
        ((r[0][-1, 0, :57].double() - k[n - 50:]).abs() <= 2.0**-8 * k[n - 50:].abs()).all()


# ------------------------------------------------------- choosing blocks


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("G,tq", [(1, 1), (4, 1), (2, 5)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_select_and_sparse_decode(D, G, tq, n):
    lens = (64 * 23 + 5, 64 * 3, 40, 0)
    k, v = tokens(D + G + tq, 4, 2, max(lens), D)
    c, L = filled(k, v, lens)
    q = queries(n, 4, 2 * G, tq, D)
    blocks = A.attn_q8_select(q.to(dev()), c, L, n)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=blocks)
    assert status() == 0
    seqs, lists = sequences(k, v, lens), blocks.cpu().numpy()
    for b in range(4):
        for h in range(2):
            for r in range(tq):
                last = lens[b] - tq + r
                some = 0 if last < 0 else min(lens[b] // 64, last // 64 + 1)
                heads = [q[b, h * G + g, r].double().numpy() for g in range(G)]
                want = R.best_of(R.scores(seqs[b][h], heads, some), n)
                assert lists[b, h, r].tolist() == want, (b, h, r)
    check_decode(q, o, lse, seqs, lens, lists=lists, label=f"sparse n={n} G={G} tq={tq}")


def test_select_ties_zeros_and_many_blocks():
    """All scores alike: the first blocks; a block that stands out; thousands of blocks with few distinct scores."""
    n, D = 64 * 5000, 32
    c = A.Q8Cache.empty(1, 1, D, n, device=dev())
    g = torch.Generator().manual_seed(3)
    level = torch.randint(0, 4, (5000,), generator=g)
    c.bounds[0, 0, :, 1] = level[:, None].to(torch.int8).to(dev())
    c.scales[0, 0, :, 0] = 1.0
    q = torch.ones(1, 1, 1, D, dtype=torch.bfloat16, device=dev())
    for some in (1, 7, 255, 256, 257, 1300, 4999, 5000):
        got = A.attn_q8_select(q, c, ints(n), some)[0, 0, 0].tolist()
        assert got == R.best_of(level.numpy(), some), some
        assert A.attn_q8_select(0 * q, c, ints(n), some)[0, 0, 0].tolist() == list(range(some))
    assert A.attn_q8_select(q, c, ints(n), 5003)[0, 0, 0].tolist() == list(range(5000)) + [-1] * 3
    c.scales[0, 0, 4321, 0] = NAN
    c.scales[0, 0, 17, 0] = INF
    assert A.attn_q8_select(q, c, ints(n), 1)[0, 0, 0].tolist() == [4321]
    assert status() == 0


@pytest.mark.parametrize("count", [2, 127, 128, 129, 200, 255, 256, 257, 511, 513])
def test_select_and_evict_few_and_many_blocks(count):
    """Around the counts at which blocks are chosen in another way, with ties, for several numbers kept."""
    D = 32
    c = A.Q8Cache.empty(2, 2, D, 64 * count, device=dev())
    room = A.Q8Cache.empty(2, 2, D, 64 * count, device=dev())
    g = torch.Generator().manual_seed(count)
    level = torch.randint(0, 40, (2, 2, count), generator=g)
    c.bounds[:, :, :, 1] = level[..., None].to(torch.int8).to(dev())
    c.scales[..., 0] = 1.0
    c.weight.copy_(level)
    q = torch.ones(2, 2, 1, D, dtype=torch.bfloat16, device=dev())
    L = ints(64 * count, 64 * count)
    for n in sorted({1, 2, count // 3 + 1, count - 1, count}):
        got = A.attn_q8_select(q, c, L, n)
        _, kept = A.attn_q8_evict(c, L, n, recent=0, out=room)
        for b in range(2):
            for h in range(2):
                want = R.best_of(level[b, h].numpy(), n)
                assert got[b, h, 0].tolist() == want, (n, b, h)
                assert kept[b, h].tolist() == want, (n, b, h)
    assert status() == 0


def test_sparse_lists_that_are_wrong_are_skipped_and_reported():
    lens = (64 * 6 + 9,)
    k, v = tokens(14, 1, 1, lens[0], 64)
    c, L = filled(k, v, lens)
    q = queries(6, 1, 1, 1, 64)
    seqs = sequences(k, v, lens)
    for given, counts in (((0, 3, 6), (0, 3)), ((2, 2, 4), (2, 4)), ((5, 1, -1), (5,)), ((1, 2**31 - 1, -1), (1,)),
                          ((-1, 4, -1), ())):
        lists = torch.tensor(given, dtype=torch.int32).reshape(1, 1, 1, 3)
        o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=lists.to(dev()))
        assert status() == E_LENGTH, given
        check_decode(q, o, lse, seqs, lens, lists=np.array(counts + (-1,)).reshape(1, 1, 1, -1), label=str(given))
    empty = torch.full((1, 1, 1, 5), -1, dtype=torch.int32)
    o, lse = A.attn_q8_decode(q.to(dev()), c, L, blocks=empty.to(dev()))
    assert status() == 0
    check_decode(q, o, lse, seqs, lens, lists=empty.numpy(), label="the open block alone")


def test_sparse_with_every_block_is_dense():
    lens = (64 * 40 + 30, 64 * 40)
    k, v = tokens(15, 2, 2, max(lens), 128)
    c, L = filled(k, v, lens)
    q = queries(7, 2, 2, 1, 128).to(dev())
    blocks = A.attn_q8_select(q, c, L, 40)
    o, lse = A.attn_q8_decode(q, c, L, blocks=blocks)
    assert status() == 0
    check_decode(q.cpu(), o, lse, sequences(k, v, lens), lens)


# ------------------------------------------------------------------ eviction


def evicted(seqs, lens, weight, keep, sink, recent):
    """Places kept, per sequence and head."""
    out = []
    for b, heads in enumerate(seqs):
        out.append([])
        for h in range(len(heads)):
            m = lens[b] // 64
            rank = [(-np.inf if j < sink or j >= m - recent else -float(weight[b, h, j]), j) for j in range(m)]
            kept = sorted(j for _, j in sorted(rank, key=lambda x: (x[0], x[1]))[:keep])
            out[-1].append(kept)
    return out


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 0, 1), (5, 1, 2), (6, 0, 1), (40, 2, 2)])
def test_evict(D, inplace, keep, sink, recent):
    lens = (64 * 7 + 3, 64 * 6 + 63, 64 * 40, 50, 0)
    k, v = tokens(D + keep, 5, 2, max(lens), D)
    c, L = filled(k, v, lens)
    g = torch.Generator().manual_seed(keep)
    w = torch.randint(0, 9, (5, 2, c.blocks), generator=g).float()  # ties
    c.weight.copy_(w)
    old = {x: getattr(c, x).clone() for x in ("k_codes", "v_codes", "scales", "bounds", "recent_k", "recent_v")}
    room = c if inplace else A.Q8Cache.empty(5, 2, D, 64 * keep, device=dev())
    lens_out = L if inplace else None
    after, kept = A.attn_q8_evict(c, L, keep, sink=sink, recent=recent, out=None if inplace else room, lens_out=lens_out)
    assert status() == 0
    want = evicted(sequences(k, v, lens), lens, w.numpy(), keep, sink, recent)
    same = lambda x, y: torch.equal(x.flatten().repeat(1).view(torch.uint8), y.flatten().repeat(1).view(torch.uint8))
    assert after.tolist() == [min(n // 64, keep) * 64 + n % 64 for n in lens]
    for b in range(5):
        for h in range(2):
            places = want[b][h]
            m = len(places)
            assert kept[b, h].tolist() == places + [-1] * (keep - m), (b, h)
            for name in ("k_codes", "v_codes", "scales", "bounds"):
                assert same(getattr(room, name)[b, h, :m], old[name][b, h, places]), (name, b, h)
            assert same(room.weight[b, h, :m], w[b, h, places].to(dev()))
            n0, n1 = lens[b], int(after[b])
            for name in ("recent_k", "recent_v"):
                for x in range(min(n0, 64 + n0 % 64)):
                    assert same(getattr(room, name)[b, h, (n1 - 1 - x) % 128], old[name][b, h, (n0 - 1 - x) % 128]), (name, b, h, x)
    if not inplace:
        for name, t in old.items():
            assert same(getattr(c, name), t), f"{name}: the source is left alone"


def test_evict_long_in_place():
    """More blocks than one round of loads holds, most of them moving, in several heads."""
    n = 64 * 700 + 11
    k, v = tokens(77, 1, 3, n, 64)
    c, L = filled(k, v, (n,))
    w = torch.rand(1, 3, c.blocks, generator=torch.Generator().manual_seed(5))
    c.weight.copy_(w)
    room = A.Q8Cache.empty(1, 3, 64, 64 * 500, device=dev())
    a1, k1 = A.attn_q8_evict(c, L, 500, sink=1, recent=4, out=room)
    a2, k2 = A.attn_q8_evict(c, L, 500, sink=1, recent=4, lens_out=L)
    assert status() == 0
    assert k1[0, 0].tolist() == evicted(sequences(k[:, :1], v[:, :1], (n,)), (n,), w.numpy(), 500, 1, 4)[0][0]
    assert torch.equal(k1, k2) and torch.equal(a1, a2) and L.tolist() == [500 * 64 + 11]
    for name in ("k_codes", "v_codes", "scales", "bounds", "weight"):
        x, y = getattr(c, name)[:, :, :500], getattr(room, name)
        assert torch.equal(x, y), name
    bits = lambda t: t.view(torch.int16)  # (rows that were never written hold NaN)
    assert torch.equal(bits(c.recent_k), bits(room.recent_k)) and torch.equal(bits(c.recent_v), bits(room.recent_v))


def test_evict_reports_lengths_out_of_range():
    k, v = tokens(1, 2, 2, 300, 64)
    c, _ = filled(k, v, (300, 300))
    old = c.k_codes.clone()
    after, kept = A.attn_q8_evict(c, ints(-7, 300), 4, sink=1)
    assert status() == E_LENGTH
    assert after.tolist() == [-7, 300] and (kept[0] == -1).all() and torch.equal(old, c.k_codes)
    c.weight.zero_()
    after, kept = A.attn_q8_evict(c, ints(-7, 300), 2, sink=1)
    assert status() == E_LENGTH
    assert after.tolist() == [-7, 2 * 64 + 44] and kept[1].tolist() == [[0, 3], [0, 3]]
    assert torch.equal(old[0], c.k_codes[0])


# -------------------------------------------------- together, as they are used


def test_a_text_from_prompt_to_eviction():
    """A padded batch of prompts through the causal forward and into the cache, then tokens one and several at a
    time: append, decode with kept weights, a sparse step, an eviction, and on."""
    B, H, Hkv, D = 3, 4, 2, 64
    lens = [150, 64, 9]
    k, v = tokens(50, B, Hkv, 600, D)
    c = A.Q8Cache.empty(B, Hkv, D, 600, device=dev())
    # the prompt: exact attention over the prompt's own tokens, then the cache takes them
    q = queries(1, B, Hkv, 150, D).to(dev())
    kp, vp = k[:, :, :150].contiguous().to(dev()), v[:, :, :150].contiguous().to(dev())
    o, lse = A.attn_fwd(q, kp, vp)
    L = ints(*lens)
    A.attn_q8_append(c, kp, vp, L, L)
    text_k, text_v = [k[b, :, :lens[b]] for b in range(B)], [v[b, :, :lens[b]] for b in range(B)]
    at = 150
    weight = [[np.zeros(lens[b] // 64) for _ in range(Hkv)] for b in range(B)]
    for step, m in enumerate([1, 1, 4, 1, 16, 1, 30, 1, 1]):
        new = k[:, :, at:at + m], v[:, :, at:at + m]
        at += m
        L += m
        for b in range(B):
            text_k[b], text_v[b] = torch.cat([text_k[b], new[0][b]], 1), torch.cat([text_v[b], new[1][b]], 1)
            lens[b] += m
        A.attn_q8_append(c, new[0].contiguous().to(dev()), new[1].contiguous().to(dev()), L)
        qs = queries(100 + step, B, H, min(m, 16), D)
        o, lse = A.attn_q8_decode(qs.to(dev()), c, L, weight="add")
        seqs = [[R.Sequence(text_k[b][h].double().numpy(), text_v[b][h].double().numpy()) for h in range(Hkv)] for b in range(B)]
        assert status() == 0
        check_decode(qs, o, lse, seqs, lens, label=f"step {step}")
    check_held(c, seqs)
    assert torch.all(c.weight >= 0) and torch.all(c.weight[0, :, 0] > 0)
    # a sparse step
    blocks = A.attn_q8_select(qs.to(dev()), c, L, 1)
    o, lse = A.attn_q8_decode(qs.to(dev()), c, L, blocks=blocks)
    assert status() == 0
    check_decode(qs, o, lse, seqs, lens, lists=blocks.cpu().numpy(), label="sparse")
    # an eviction in place, then on with the shorter texts: the open block and what comes after are unharmed
    kept = A.attn_q8_evict(c, L, 2, recent=1, lens_out=L)[1].cpu().numpy()
    short = []
    for b in range(B):
        short.append([])
        for h in range(Hkv):
            s = seqs[b][h]
            places = [j for j in kept[b, h] if j >= 0]
            keep = np.concatenate([np.arange(64 * j, 64 * j + 64) for j in places] + [np.arange(64 * s.closed, len(s.k))])
            short[-1].append(R.Sequence(s.k[keep], s.v[keep]))  # whole blocks quantise to the same codes
    lens = [min(n // 64, 2) * 64 + n % 64 for n in lens]
    assert L.tolist() == lens
    o, lse = A.attn_q8_decode(qs.to(dev()), c, L)
    assert status() == 0
    check_held(c, short)
    check_decode(qs, o, lse, short, lens, label="after the eviction")
    m = 70
    L += m
    kn, vn = k[:, :, at:at + m].contiguous(), v[:, :, at:at + m].contiguous()
    A.attn_q8_append(c, kn.to(dev()), vn.to(dev()), L)
    for b in range(B):
        lens[b] += m
        for h in range(Hkv):
            s = short[b][h]
            short[b][h] = R.Sequence(np.concatenate([s.k, kn[b, h].double().numpy()]), np.concatenate([s.v, vn[b, h].double().numpy()]))
    o, lse = A.attn_q8_decode(qs.to(dev()), c, L)
    assert status() == 0
    check_held(c, short)
    check_decode(qs, o, lse, short, lens, label="appended after the eviction")


def test_near_the_decode_over_bf16():
    """The same step over bf16 keys and values: what the 8 bits cost is within what half a step of each value
    (most / 254) can do to the sums."""
    B, H, n, D = 2, 3, 500, 64
    k, v = tokens(60, B, H, n, D)
    c, L = filled(k, v, (n, n))
    q = queries(9, B, H, 1, D)
    o8, lse8 = A.attn_q8_decode(q.to(dev()), c, L)
    o, lse = A.attn_decode(q.to(dev()), k.to(dev()), v.to(dev()))
    assert status() == 0
    for b in range(B):
        for h in range(H):
            s = R.Sequence(k[b, h].double().numpy(), v[b, h].double().numpy())
            row = q[b, h, 0].double().numpy()
            ds = np.abs(s.held_k - s.k) @ np.abs(row) / D**0.5  # how far each score moves at most
            dv = np.abs(s.held_v - s.v).max(axis=0)
            e = np.expm1(2 * ds.max())  # the weights then change by this factor at most
            bound = dv + e * np.abs(s.v).max(axis=0) + 2.0**-7 * np.abs(s.v).max(axis=0)
            assert np.all(np.abs((o8 - o)[b, h, 0].double().cpu().numpy()) <= bound)
            assert abs(float((lse8 - lse)[b, h, 0])) <= ds.max() + 1e-3


def test_captured_steps_replay_with_growing_lengths():
    """One captured step (append, select, sparse decode, dense decode with weights) replayed while the lengths on
    the device grow; a second graph shares the workspace on the same stream."""
    B, H, D = 2, 2, 64
    k, v = tokens(70, B, H, 400, D)
    lens = [120, 62]
    c, L = filled(k[:, :, :120], v[:, :, :120], lens, max_tokens=400)
    kn, vn = (torch.zeros(B, H, 1, D, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    q = queries(1, B, H, 1, D).to(dev())
    ws = torch.empty(A.attn_q8_decode_workspace_bytes(c, H, 1, weight="set"), dtype=torch.uint8, device=dev())
    blocks = torch.empty(B, H, 1, 2, dtype=torch.int32, device=dev())
    outs = [torch.empty(B, H, 1, D, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    lses = [torch.empty(B, H, 1, device=dev()) for _ in range(2)]

    def first():
        L.add_(1)
        A.attn_q8_append(c, kn, vn, L)
        A.attn_q8_decode(q, c, L, o=outs[0], lse=lses[0], weight="set", workspace=ws)

    def second():
        A.attn_q8_select(q, c, L, 2, blocks=blocks)
        A.attn_q8_decode(q, c, L, o=outs[1], lse=lses[1], blocks=blocks, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once before the capture
        first(), second()
        L.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    text = [[k[b, :, :lens[b]], v[b, :, :lens[b]]] for b in range(B)]
    for step in range(12):
        kn.copy_(k[:, :, 200 + step:201 + step])
        vn.copy_(v[:, :, 200 + step:201 + step])
        q.copy_(queries(300 + step, B, H, 1, D))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b in range(B):
            lens[b] += 1
            text[b] = [torch.cat([t, s[b, :, 200 + step:201 + step]], 1) for t, s in zip(text[b], (k, v))]
        if step % 3 == 1 or step == 11:
            seqs = [[R.Sequence(text[b][0][h].double().numpy(), text[b][1][h].double().numpy()) for h in range(H)] for b in range(B)]
            assert status() == 0
            assert L.tolist() == lens
            check_held(c, seqs)
            check_decode(q.cpu(), outs[0], lses[0], seqs, lens, weight=c.weight.double().cpu().numpy(), label=f"replay {step}")
            check_decode(q.cpu(), outs[1], lses[1], seqs, lens, lists=blocks.cpu().numpy(), label=f"sparse replay {step}")


def test_other_streams_and_two_caches_at_once():
    """Calls on two streams over two caches, with temporaries of their own, and a call on a stream that is not the
    current one."""
    B, H, D, n = 2, 4, 64, 3000
    sets = []
    for i in range(2):
        k, v = tokens(80 + i, B, H, n, D)
        c, L = filled(k, v, (n, n // 2))
        sets.append((k, v, c, L, queries(i, B, H, 1, D).to(dev()), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for k, v, c, L, q, st in sets:
            got.append(A.attn_q8_decode(q, c, L, stream=st))
    torch.cuda.synchronize()
    assert status() == 0
    for i, (k, v, c, L, q, st) in enumerate(sets):
        for o, lse in got[i::2]:
            assert torch.equal(o, got[i][0]) and torch.equal(lse, got[i][1])
        check_decode(q.cpu(), *got[i], sequences(k, v, (n, n // 2)), (n, n // 2))


def test_every_call_on_a_stream_that_is_not_current():
    """What a call on another stream allocates is not memory that work queued on the current stream still reads."""
    B, H, D, n = 2, 4, 64, 700
    k, v = tokens(85, B, H, n, D)
    c, L = filled(k, v, (n, n - 200))
    q = queries(9, B, H, 1, D).to(dev())
    side = torch.cuda.Stream()
    want = [*A.attn_q8_decode(q, c, L, weight="set"), A.attn_q8_select(q, c, L, 3), *A.attn_q8_read(c, L, n),
            c.weight.clone()]
    room = A.Q8Cache.empty(B, H, D, n, device=dev())
    want += A.attn_q8_evict(c, L, 5, sink=1, recent=1, out=room)
    torch.cuda.synchronize()
    # memory of the results' sizes, read by queued work and given back: the allocator hands it to the current stream's calls
    lent = [torch.ones_like(x) for x in want]
    copies = [torch.zeros_like(x) for x in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for to, x in zip(copies, lent):
        to.copy_(x)
    x = None
    del lent
    got = [*A.attn_q8_decode(q, c, L, weight="set", stream=side), A.attn_q8_select(q, c, L, 3, stream=side),
           *A.attn_q8_read(c, L, n, stream=side)]
    with torch.cuda.stream(side):
        got.append(c.weight.clone())
    got += A.attn_q8_evict(c, L, 5, sink=1, recent=1, out=room, stream=side)
    assert A.attn_q8_append(c, k[:, :, :1].to(dev()), v[:, :, :1].to(dev()), L, ints(0, 0), stream=side) is None
    side.synchronize()
    torch.cuda.synchronize()
    assert status() == 0
    assert all((x == 1).all() for x in copies)
    closed = (n // 64, (n - 200) // 64)
    for i, (x, y) in enumerate(zip(got, want)):
        if i == 5:  # (what is not closed has no weight)
            assert all(torch.equal(x[b, :, :closed[b]], y[b, :, :closed[b]]) for b in range(B))
        else:
            assert torch.equal(x, y), i


def test_strided_queries_choose_as_contiguous_ones():
    B, H, G, D, tq, n = 2, 2, 3, 64, 4, 64 * 11 + 9
    k, v = tokens(86, B, H, n, D)
    c, L = filled(k, v, (n, 300))
    packed = queries(11, B, tq, H * G + 2, D).to(dev())  # [B, T, heads, D]
    q = packed.transpose(1, 2)[:, 1:-1]
    got = A.attn_q8_select(q, c, L, 2)
    assert torch.equal(got, A.attn_q8_select(q.contiguous(), c, L, 2)) and status() == 0


def test_launches_and_timing_hook():
    """One launch a call where the interface says so, and events around the main kernel."""
    k, v = tokens(87, 2, 2, 640, 64)
    c, L = filled(k, v, (640, 100))
    q = queries(12, 2, 2, 1, 64).to(dev())
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in events:
        e.record()  # (made before they are handed over)
    one = ints(0, 0)
    for call, launches in ((lambda: A.attn_q8_append(c, k[:, :, :1].to(dev()), v[:, :, :1].to(dev()), L, one), 1),
                           (lambda: A.attn_q8_read(c, L, 640), 1), (lambda: A.attn_q8_select(q, c, L, 2), 1),
                           (lambda: A.attn_q8_decode(q, c, L, weight="set"), 1), (lambda: A.attn_q8_evict(c, L, 3), 2)):
        A.attn_profile_next_call(*events)
        call()
        assert A.lib().attn_last_launch_count() == launches
        torch.cuda.synchronize()
        assert 0 < events[0].elapsed_time(events[1]) < 1000
    assert status() == 0


def test_evict_into_a_cache_without_bounds_and_weight():
    n = 64 * 9 + 20
    k, v = tokens(88, 1, 2, n, 32)
    c, L = filled(k, v, (n,))
    c.weight.copy_(torch.rand(1, 2, c.blocks, generator=torch.Generator().manual_seed(1)))
    room = A.Q8Cache.empty(1, 2, 32, n, device=dev(), bounds=False, weight=False)
    after, kept = A.attn_q8_evict(c, L, 30000, sink=1, out=room)  # (more than there are: a copy)
    assert status() == 0 and after.tolist() == [n] and (kept[:, :, 9:] == -1).all()
    q = queries(13, 1, 2, 1, 32).to(dev())
    for x, y in zip(A.attn_q8_decode(q, room, after), A.attn_q8_decode(q, c, L)):
        assert torch.equal(x, y)
    after, kept = A.attn_q8_evict(c, L, 4, sink=1, out=room)
    assert status() == 0 and after.tolist() == [4 * 64 + 20]
    for h in range(2):
        assert torch.equal(room.k_codes[0, h, :4], c.k_codes[0, h, kept[0, h].long()])


def test_results_do_not_depend_on_the_run():
    """The same call gives the same bits, with the workspace holding anything."""
    k, v = tokens(90, 2, 3, 2000, 128)
    c, L = filled(k, v, (2000, 999))
    q = queries(3, 2, 6, 2, 128).to(dev())
    need = A.attn_q8_decode_workspace_bytes(c, 6, 2, weight="set")
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=dev())
        o, lse = A.attn_q8_decode(q, c, L, weight="set", workspace=ws)
        now = (o, lse, c.weight.clone()[:, :, :15])
        first = first or now
        assert all(torch.equal(x, y) for x, y in zip(now, first))
    assert status() == 0


def test_outputs_are_new_or_the_lent_ones_and_nothing_is_kept():
    k, v = tokens(91, 1, 2, 200, 64)
    c, L = filled(k, v, (200,))
    q = queries(14, 1, 2, 1, 64).to(dev())
    o, lse = torch.empty_like(q), torch.empty(1, 2, 1, device=dev())
    kept, after = torch.empty(1, 2, 9, dtype=torch.int32, device=dev()), torch.empty(1, dtype=torch.int32, device=dev())
    blocks, room = torch.empty(1, 2, 1, 2, dtype=torch.int32, device=dev()), torch.empty(1, 2, 200, 64, dtype=torch.bfloat16, device=dev())
    lent = (q, L, o, lse, kept, after, blocks, room)

    def calls():
        got = A.attn_q8_decode(q, c, L, o=o, lse=lse)
        assert got[0] is o and got[1] is lse
        assert A.attn_q8_select(q, c, L, 2, blocks=blocks) is blocks
        x, y = A.attn_q8_read(c, L, 200, k=room)
        assert x is room and y is not room
        got = A.attn_q8_evict(c, L, 9, lens_out=after, kept=kept)
        assert got[0] is after and got[1] is kept
        for bad in (lambda: A.attn_q8_decode(q, c, L, o=o, lse=o), lambda: A.attn_q8_decode(q, c, L, o=o, lse=lse, scale=-1.0),
                    lambda: A.attn_q8_decode(q, c, L, workspace=L.cpu()), lambda: A.attn_q8_read(c, L, 200, k=room, v=o),
                    lambda: A.attn_q8_decode(q, c, L, scale="1"), lambda: A.attn_q8_evict(c, L, 9, kept=after)):
            with pytest.raises((TypeError, ValueError, A.AttnError)):
                bad()

    calls()
    torch.cuda.synchronize()
    counts, held = [sys.getrefcount(t) for t in lent], torch.cuda.memory_allocated()
    for _ in range(20):
        calls()
    assert [sys.getrefcount(t) for t in lent] == counts
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held and status() == 0


def test_binding_refusals_on_the_gpu():
    k, v = tokens(1, 1, 2, 70, 64)
    c, L = filled(k, v, (70,))
    q = queries(1, 1, 2, 1, 64).to(dev())
    with pytest.raises(TypeError):
        A.attn_q8_decode(q.float(), c, L)
    with pytest.raises(TypeError):
        A.attn_q8_decode(q, c, L.long())
    with pytest.raises(ValueError):
        A.attn_q8_decode(q, c, L.cpu())
    with pytest.raises(ValueError):
        A.attn_q8_decode(q[:, :, :, :32], c, L)
    with pytest.raises(ValueError):
        A.attn_q8_decode(q, c, L, weight="sum")
    with pytest.raises(A.AttnError):
        A.attn_q8_decode(q[:, :1], c, L)
    with pytest.raises(ValueError):
        A.attn_q8_decode(q, c, L, blocks=torch.zeros(1, 2, 2, 1, dtype=torch.int32, device=dev()))
    with pytest.raises(ValueError):
        A.attn_q8_append(c, k.to(dev()), v.to(dev())[:, :, :3], L)
    with pytest.raises(ValueError):
        A.attn_q8_append(c, k.to(dev()).transpose(2, 3), v.to(dev()).transpose(2, 3), L)
    with pytest.raises(A.AttnError):
        A.attn_q8_select(q, c, L, 0)
    bare = A.Q8Cache.empty(1, 2, 64, 100, device=dev(), bounds=False, weight=False)
    A.attn_q8_append(bare, k.to(dev()), v.to(dev()), L)
    A.attn_q8_decode(q, bare, L)
    with pytest.raises(A.AttnError):
        A.attn_q8_select(q, bare, L, 1)
    with pytest.raises(A.AttnError):
        A.attn_q8_evict(bare, L, 1)
    with pytest.raises(A.AttnError):
        A.attn_q8_decode(q, bare, L, weight="set")
    with pytest.raises(ValueError):
        A.Q8Cache(c.k_codes, c.v_codes, c.scales[:, :, :1], None, None, c.recent_k, c.recent_v)
    assert status() == 0
