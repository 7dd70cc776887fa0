"""Refusals of the 8-bit cache's entry points, before anything touches CUDA
(the addresses here are never read), and the sizes of their workspaces."""
import ctypes

import pytest

import decoder_only_transformer_sdpa_b200 as A

E_NULL, E_SHAPE, E_D, E_ALIGN, E_WS, E_SCALE, E_OPTION, E_LENGTH = -1, -2, -3, -4, -7, -9, -10, -12
P = 1 << 20


def cache(**kw):
    f = dict(k_codes=P, v_codes=2 * P, scales=3 * P, bounds=4 * P, weight=5 * P, recent_k=6 * P, recent_v=7 * P,
             B=2, H=3, blocks=4, D=64)
    f.update(kw)
    return A.attn_q8_cache(*(f[n] for n, _ in A.attn_q8_cache._fields_))


BAD_CACHES = [(dict(k_codes=None), E_NULL), (dict(v_codes=None), E_NULL), (dict(scales=None), E_NULL),
              (dict(recent_k=None), E_NULL), (dict(recent_v=None), E_NULL), (dict(B=0), E_SHAPE), (dict(H=-1), E_SHAPE),
              (dict(blocks=0), E_SHAPE), (dict(blocks=32769), E_SHAPE), (dict(D=48), E_D), (dict(D=256), E_D),
              (dict(B=1 << 16, H=1 << 16), E_SHAPE), (dict(B=1 << 12, H=1 << 12, blocks=1 << 12), E_SHAPE),
              (dict(k_codes=P + 8), E_ALIGN), (dict(v_codes=P + 1), E_ALIGN), (dict(scales=P + 4), E_ALIGN),
              (dict(bounds=P + 8), E_ALIGN), (dict(weight=P + 2), E_ALIGN), (dict(recent_k=P + 8), E_ALIGN)]


def strides(*rows):
    return (A.attn_strides * len(rows))(*(A.attn_strides(*r) for r in rows))


GOOD = (192, 64, 64)


def append(c=None, k=P, v=P, n=5, lens=P, new=None, st=None):
    c = cache() if c is None else c
    return A.lib().attn_q8_append(ctypes.byref(c), k, v, n, lens, new, st, None)


def read(c=None, lens=P, starts=None, n=5, k=P, v=P):
    c = cache() if c is None else c
    return A.lib().attn_q8_read(ctypes.byref(c), lens, starts, n, k, v, None)


def decode(c=None, q=P, o=P, lse=P, lens=P, H=6, Tq=2, scale=0.125, st=None, opts=None, ws=P, ws_bytes=1 << 40):
    c = cache() if c is None else c
    return A.lib().attn_q8_decode(ctypes.byref(c), q, o, lse, lens, H, Tq, scale, st,
                                  None if opts is None else ctypes.byref(opts), ws, ws_bytes, None)


def select(c=None, q=P, lens=P, blocks=P, n=2, H=6, Tq=2, st=None):
    c = cache() if c is None else c
    return A.lib().attn_q8_select(ctypes.byref(c), q, lens, blocks, n, H, Tq, st, None)


def evict(c=None, out=None, lens=P, lens_out=P, kept=P, keep=2, sink=0, recent=1, ws=P, ws_bytes=1 << 40):
    c = cache() if c is None else c
    out = c if out is None else out
    return A.lib().attn_q8_evict(ctypes.byref(c), ctypes.byref(out), lens, lens_out, kept, keep, sink, recent, ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("kw,expect", BAD_CACHES)
@pytest.mark.parametrize("call", [append, read, decode, select, evict])
def test_bad_caches(call, kw, expect):
    assert call(cache(**kw)) == expect


def test_null_cache():
    lib = A.lib()
    assert lib.attn_q8_append(None, P, P, 1, P, None, None, None) == E_NULL
    assert lib.attn_q8_read(None, P, None, 1, P, P, None) == E_NULL
    assert lib.attn_q8_decode(None, P, P, P, P, 3, 1, 0.1, None, None, P, 1 << 30, None) == E_NULL
    assert lib.attn_q8_select(None, P, P, P, 1, 3, 1, None, None) == E_NULL
    assert lib.attn_q8_evict(None, None, P, P, P, 1, 0, 0, P, 1 << 30, None) == E_NULL
    assert lib.attn_q8_decode_workspace_bytes(None, 3, 1, None) == 0
    assert lib.attn_q8_evict_workspace_bytes(None) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), E_NULL), (dict(v=None), E_NULL), (dict(lens=None), E_NULL), (dict(n=0), E_SHAPE),
    (dict(n=-3), E_SHAPE), (dict(n=4 * 64 + 64), E_SHAPE), (dict(k=P + 8), E_ALIGN), (dict(v=P + 2), E_ALIGN),
    (dict(lens=P + 2), E_ALIGN), (dict(new=P + 1), E_ALIGN), (dict(st=strides(GOOD, (192, 60, 64))), E_ALIGN),
    (dict(st=strides((0, 64, 64), GOOD)), E_ALIGN),
])
def test_append_refusals(kw, expect):
    assert append(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), E_NULL), (dict(lens=None), E_NULL), (dict(n=0), E_SHAPE), (dict(n=64 * 32769 + 1), E_SHAPE),
    (dict(v=P + 8), E_ALIGN), (dict(starts=P + 2), E_ALIGN),
])
def test_read_refusals(kw, expect):
    assert read(**kw) == expect


KEEP = A.attn_q8_decode_options(None, 0, 1)  # kept weights need a workspace


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), E_NULL), (dict(o=None), E_NULL), (dict(lse=None), E_NULL), (dict(lens=None), E_NULL),
    (dict(H=4), E_SHAPE), (dict(H=0), E_SHAPE), (dict(H=3 * 65), E_SHAPE), (dict(Tq=0), E_SHAPE), (dict(Tq=17), E_SHAPE),
    (dict(scale=0.0), E_SCALE), (dict(scale=float("nan")), E_SCALE), (dict(scale=float("inf")), E_SCALE),
    (dict(q=P + 8), E_ALIGN), (dict(o=P + 8), E_ALIGN), (dict(lse=P + 2), E_ALIGN), (dict(lens=P + 3), E_ALIGN),
    (dict(st=strides(GOOD, (-64, 64, 64))), E_ALIGN),
    (dict(opts=KEEP, ws=None), E_WS), (dict(opts=KEEP, ws=P + 16), E_WS), (dict(opts=KEEP, ws_bytes=16), E_WS),
    (dict(opts=A.attn_q8_decode_options(None, 0, 3)), E_OPTION),
    (dict(opts=A.attn_q8_decode_options(None, 0, -1)), E_OPTION),
    (dict(opts=A.attn_q8_decode_options(None, 2, 0)), E_OPTION),
    (dict(opts=A.attn_q8_decode_options(P, 0, 0)), E_OPTION),
    (dict(opts=A.attn_q8_decode_options(P, 32769, 0)), E_OPTION),
    (dict(opts=A.attn_q8_decode_options(P, 2, 1)), E_OPTION),
    (dict(opts=A.attn_q8_decode_options(P + 2, 2, 0)), E_ALIGN),
    (dict(c=cache(weight=None), opts=A.attn_q8_decode_options(None, 0, 2)), E_OPTION),
])
def test_decode_refusals(kw, expect):
    assert decode(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), E_NULL), (dict(blocks=None), E_NULL), (dict(lens=None), E_NULL), (dict(c=cache(bounds=None)), E_NULL),
    (dict(n=0), E_SHAPE), (dict(n=32769), E_SHAPE), (dict(H=5), E_SHAPE), (dict(Tq=17), E_SHAPE),
    (dict(q=P + 8), E_ALIGN), (dict(blocks=P + 2), E_ALIGN), (dict(st=strides((1, 64, 64))), E_ALIGN),
])
def test_select_refusals(kw, expect):
    assert select(**kw) == expect


OTHER = dict(k_codes=11 * P, v_codes=12 * P, scales=13 * P, bounds=14 * P, weight=15 * P, recent_k=16 * P,
             recent_v=17 * P)


@pytest.mark.parametrize("kw,expect", [
    (dict(lens=None), E_NULL), (dict(lens_out=None), E_NULL), (dict(kept=None), E_NULL),
    (dict(c=cache(weight=None)), E_NULL), (dict(c=cache(bounds=None), out=cache(**OTHER)), E_NULL),
    (dict(keep=0), E_SHAPE), (dict(keep=32769), E_SHAPE), (dict(sink=-1), E_SHAPE), (dict(recent=-1), E_SHAPE),
    (dict(sink=2, recent=1), E_SHAPE), (dict(sink=3), E_SHAPE), (dict(keep=5, sink=2**31 - 1, recent=2**31 - 1), E_SHAPE),
    (dict(out=cache(**{**OTHER, "blocks": 1})), E_SHAPE), (dict(out=cache(**{**OTHER, "B": 1})), E_SHAPE),
    (dict(out=cache(**{**OTHER, "H": 1})), E_SHAPE), (dict(out=cache(**{**OTHER, "D": 32})), E_SHAPE),
    (dict(out=cache(**{**OTHER, "k_codes": P})), E_OPTION), (dict(out=cache(**{**OTHER, "scales": 3 * P})), E_OPTION),
    (dict(out=cache(**{**OTHER, "recent_v": 7 * P})), E_OPTION), (dict(out=cache(**{**OTHER, "bounds": 4 * P})), E_OPTION),
    (dict(out=cache(**{**OTHER, "weight": 5 * P})), E_OPTION), (dict(out=cache(blocks=3)), E_OPTION),
    (dict(out=cache(**{**OTHER, "k_codes": P + 64})), E_OPTION), (dict(out=cache(**{**OTHER, "v_codes": 2 * P - 64})), E_OPTION),
    (dict(out=cache(**{**OTHER, "scales": 3 * P + 8})), E_OPTION), (dict(out=cache(**{**OTHER, "bounds": 4 * P + 16})), E_OPTION),
    (dict(out=cache(**{**OTHER, "weight": 5 * P - 4})), E_OPTION), (dict(out=cache(**{**OTHER, "recent_k": 6 * P + 256})), E_OPTION),
    (dict(out=cache(**{**OTHER, "recent_v": 7 * P - 16})), E_OPTION),
    (dict(out=cache(bounds=None)), E_OPTION), (dict(lens_out=P + 2), E_ALIGN), (dict(kept=P + 2), E_ALIGN),
    # (lens_out is lens: only then is there a workspace)
    (dict(ws=None), E_WS), (dict(ws=P + 128), E_WS), (dict(ws_bytes=40), E_WS),
])
def test_evict_refusals(kw, expect):
    assert evict(**kw) == expect


PARTS = dict(k_codes=2 * 3 * 4 * 64 * 64, v_codes=2 * 3 * 4 * 64 * 64, scales=2 * 3 * 4 * 8, bounds=2 * 3 * 4 * 128,
             weight=2 * 3 * 4 * 4, recent_k=2 * 3 * 128 * 64 * 2, recent_v=2 * 3 * 128 * 64 * 2)  # bytes of cache()


@pytest.mark.parametrize("part", PARTS)
@pytest.mark.parametrize("other", PARTS)
def test_evict_refuses_to_share_memory_in_any_part(part, other):
    """Part `part` of the target at the first byte of part `other` of the source, at its last 16, and behind it (these
    calls lack a workspace, so that none gets any further)."""
    at, n = getattr(cache(), other), PARTS[other]
    for off, expect in ((0, E_OPTION), (n - 16, E_OPTION), ((n + 15) // 16 * 16, E_WS)):
        assert evict(out=cache(**{**OTHER, part: at + off}), ws=None) == expect


@pytest.mark.parametrize("kw", [dict(lens_out=20 * P + 4), dict(lens_out=20 * P - 4), dict(kept=20 * P), dict(kept=20 * P - 44),
                                dict(kept=20 * P + 4), dict(lens_out=22 * P, kept=22 * P + 4), dict(lens_out=20 * P, kept=20 * P)])
def test_evict_refuses_lengths_and_lists_that_overlap(kw):
    """2 sequences' lengths, and 2 x 3 heads' lists of 2; nothing beyond the checks runs."""
    assert evict(**{**dict(lens=20 * P, lens_out=20 * P, kept=21 * P), **kw}) == E_OPTION


def test_workspace_sizes():
    up = lambda x: (x + 255) // 256 * 256
    c = cache(B=7, H=30, blocks=100)
    ws = lambda c, H, Tq, *o: A.lib().attn_q8_decode_workspace_bytes(
        ctypes.byref(c), H, Tq, ctypes.byref(A.attn_q8_decode_options(*o)) if o else None)
    # little work is joined within clusters; kept weights take a block's log-sum for each row
    small = cache(B=3, H=4, blocks=10)
    assert ws(small, 4, 1) == 0
    assert ws(small, 4, 1, None, 0, 1) == up(3 * 4 * 10 * 4)
    assert ws(c, 31, 1) == 0 and ws(c, 30, 17) == 0 and ws(c, 30, 1, None, -1, 0) == 0
    assert ws(cache(D=40), 3, 1) == 0 and ws(cache(blocks=0), 3, 1) == 0
    one = cache(B=1, H=1, blocks=32768)
    some = ws(one, 1, 1)  # one head over millions of tokens: several clusters
    assert some > 0 and some % 256 == 0
    assert ws(one, 1, 1, None, 8, 0) == 0 and ws(one, 1, 1, None, 0, 2) > 4 * 32768
    assert A.lib().attn_q8_evict_workspace_bytes(ctypes.byref(c)) == up(7 * 30 * 12)
    assert A.lib().attn_q8_evict_workspace_bytes(ctypes.byref(cache(H=0))) == 0


def test_long_lists_of_many_row_tiles_are_counted_as_the_kernel_counts_them():
    """131072 row tiles of 32768 places each are more units than runs are made of, however few blocks the cache has."""
    many = cache(B=4096, H=32, blocks=1, D=32)
    opts = lambda n: ctypes.byref(A.attn_q8_decode_options(None, n, 0))
    assert A.lib().attn_q8_decode_workspace_bytes(ctypes.byref(many), 32, 1, opts(32768)) == 0


def test_status_string():
    assert A.attn_status_string(E_LENGTH) != A.attn_status_string(12345)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    t = lambda dtype, *s: torch.zeros(*s, dtype=dtype)
    with pytest.raises(ValueError, match="v_codes"):
        A.Q8Cache(None, t(torch.uint8, 2, 3), None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        A.Q8Cache.empty(1, 1, 64, 100, device="cpu")
    q = t(torch.bfloat16, 1, 1, 1, 64)
    for call in (lambda: A.attn_q8_append(None, q, q, q), lambda: A.attn_q8_read(None, q, 3),
                 lambda: A.attn_q8_decode(q, None, q), lambda: A.attn_q8_select(q, None, q, 1),
                 lambda: A.attn_q8_evict(None, q, 1)):
        with pytest.raises(TypeError, match="Q8Cache"):
            call()


class TestBinding:
    """The module behind the binding, given a structure and CPU tensors: what it refuses before it touches a device."""

    @staticmethod
    def module():
        m = A._binding()
        return m, m.cache(ctypes.addressof(cache(B=1, H=2, D=64)), 0)

    def test_tensors(self):
        import torch
        m, c = self.module()
        q, lens = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
        for call in (lambda q: m.append(c, q, q, lens, None), lambda q: m.decode(c, q, lens, None, None, None, None, 0, None),
                     lambda q: m.select(c, q, lens, 1, None)):
            with pytest.raises(ValueError, match="must be a CUDA tensor"):
                call(q)
            with pytest.raises(ValueError, match="expected"):
                call(q[0])
            for bad in (None, 3, "q", [q]):
                with pytest.raises(TypeError, match="torch.Tensor"):
                    call(bad)
        with pytest.raises(ValueError, match="lens must be a CUDA tensor"):
            m.read(c, lens, 3, None, None, None)
        with pytest.raises(ValueError, match="lens must be a CUDA tensor"):
            m.evict(c, c, lens, 3, 0, 0, None, None, None)
        with pytest.raises(TypeError, match="lens must be a torch.Tensor"):
            m.read(c, None, 3, None, None, None)

    def test_numbers(self):
        m, c = self.module()
        for n in (0, -1, 64 * 32769 + 1, 2**31, 2**70):
            with pytest.raises(A.AttnError) as e:
                m.read(c, None, n, None, None, None)
            assert e.value.status == E_SHAPE
        for keep, sink, recent in ((0, 0, 0), (32769, 0, 0), (2**40, 0, 0), (3, -1, 0), (3, 0, 2**33)):
            with pytest.raises(A.AttnError) as e:
                m.evict(c, c, None, keep, sink, recent, None, None, None)
            assert e.value.status == E_SHAPE
        with pytest.raises(TypeError):
            m.read(c, None, 1.5, None, None, None)

    def test_arguments(self):
        m, c = self.module()
        for f in (m.append, m.read, m.decode, m.select, m.evict):
            with pytest.raises(TypeError, match="arguments"):
                f(c)
        with pytest.raises(ValueError):  # not a cache's capsule
            m.read(object(), None, 1, None, None, None)
        m2, c2 = m, m.cache(ctypes.addressof(cache(B=1, H=2, D=64)), 1)
        with pytest.raises(ValueError, match="out must be on cuda:0"):
            m2.evict(c, c2, None, 1, 0, 0, None, None, None)
