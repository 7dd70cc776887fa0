"""Cases that measure the operators of the 8-bit cache of keys and values:

* append: new tokens' keys and values into the cache (quantised by blocks);
* decode: attention of the newest tokens over the cache, which can also keep
  the attention weight that each block received;
* sparse: choosing blocks by a cheap score, and attention over those alone;
* evict: dropping the blocks with the least kept attention weight.

A cache holds, for each sequence b and key/value head h, the closed blocks of
64 tokens as 8-bit codes (value = (code - 128) * scale, one scale for the keys
and one for the values of a block), each block's smallest and largest key code
per channel, the attention weight it has received, and the newest 128
positions in bf16 (position p in row p % 128), from which the open block is
read.  Keys of a block lie as [D / S, 64, S] with S = min(D, 64), values as
[D, 64].

Where `own` is false, `run` computes an operator with elementary torch
operations in float32; where it is true it calls the package.
"""
import torch

own = False

BLOCK = 64
RING = 2 * BLOCK


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one conversation, a short text: GPT-2's 12 heads, latency is all that counts
        dict(name="decode_one_short", op="decode", B=1, H=12, Hkv=12, D=64, len=100, tq=1, ragged=False, weights=False),
        # GPT-2 124M at its training batch, the whole context of 1024 tokens held
        dict(name="decode_gpt2_batch", op="decode", B=12, H=12, Hkv=12, D=64, len=1024, tq=1, ragged=False, weights=False),
        # a serving batch of long, unequal texts, one slot empty
        dict(name="decode_long_ragged", op="decode", B=16, H=12, Hkv=12, D=64, len=32768, tq=1, ragged=True, weights=False),
        # four drafted tokens verified at once, four query heads to a key head, wide heads
        dict(name="decode_draft_grouped", op="decode", B=4, H=32, Hkv=8, D=128, len=16411, tq=4, ragged=False, weights=False),
        # GPT-2 XL's 25 heads, the weight of each block kept for a later eviction
        dict(name="decode_xl_weights", op="decode", B=8, H=25, Hkv=25, D=64, len=4133, tq=1, ragged=True, weights=True),
        # one long text, 1024 of its 8200 tokens attended to
        dict(name="sparse_one_text", op="sparse", B=1, H=12, Hkv=12, D=64, len=8200, tq=1, n=16, ragged=False),
        # a batch of very long texts, 4096 of up to 131072 tokens attended to
        dict(name="sparse_very_long", op="sparse", B=8, H=12, Hkv=12, D=64, len=131072, tq=1, n=64, ragged=True),
        # one new token each for the character model's batch of 64 sequences with 6 heads
        dict(name="append_one_token", op="append", B=64, Hkv=6, D=64, len=2048, new=1, ragged=True),
        # GPT-2's prompts of 1024 tokens, read back as they are held
        dict(name="append_gpt2_prompt", op="append", B=12, Hkv=12, D=64, len=1024, new=1024, ragged=False),
        # long prompts in a padded batch, wide heads
        dict(name="append_long_prompt", op="append", B=4, Hkv=8, D=128, len=16411, new=16411, ragged=True),
        # GPT-2's batch at its full context, half of the blocks dropped
        dict(name="evict_gpt2_half", op="evict", B=12, Hkv=12, D=64, len=1027, keep=8, sink=1, recent=2, ragged=False),
        # long texts with GPT-2 XL's heads, a quarter of the blocks kept
        dict(name="evict_long", op="evict", B=4, Hkv=25, D=64, len=32800, keep=128, sink=1, recent=16, ragged=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["decode", "decode", "sparse", "append", "evict"])
    D = rng.choice([32, 64, 64, 128])
    heads = _spread(rng, 1, 32)
    B = _spread(rng, 1, 64)
    ragged = rng.random() < 0.5
    most = 1 << 28  # elements of the keys: the largest listed case has 1.5 times as many
    if op == "append":
        longest = max(1, min(16384, most // 8 // (B * heads * D)))
        if rng.random() < 0.4:  # a few tokens onto what is there
            n = rng.randint(1, 16)
            return dict(op=op, B=B, Hkv=heads, D=D, len=n + _spread(rng, 1, longest), new=n, ragged=ragged)
        n = _spread(rng, 1, longest)
        return dict(op=op, B=B, Hkv=heads, D=D, len=n, new=n, ragged=ragged)
    if op == "evict":
        longest = max(256, min(65536, most // 4 // (B * heads * D)))
        length = _spread(rng, 200, longest)
        closed = length // BLOCK
        keep = rng.randint(1, closed)
        recent = rng.randint(0, min(4, keep))
        return dict(op=op, B=B, Hkv=heads, D=D, len=length, keep=keep, sink=rng.randint(0, min(1, keep - recent)), recent=recent, ragged=ragged)
    group = rng.choice([1, 1, 1, 2, 4, 8])
    tq = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
    longest = max(256, min(131072, most // (B * heads * D * (4 if tq * group > 8 else 1))))
    length = _spread(rng, 17, longest)
    case = dict(op=op, B=B, H=heads * group, Hkv=heads, D=D, len=length, tq=tq, ragged=ragged)
    if op == "decode":
        case["weights"] = rng.random() < 0.4
    else:
        case["n"] = _spread(rng, 1, max(1, min(96, (most // 4) // (B * heads * tq * BLOCK * D))))
    return case


def _lengths(case):
    """Tokens of each sequence: all alike, or falling from the longest to a quarter with the last slot of four or more empty."""
    B, longest = case["B"], case["len"]
    if not case["ragged"]:
        return [longest] * B
    at = [longest - (3 * longest * b) // (4 * max(1, B - 1)) for b in range(B)]
    if B >= 4:
        at[-1] = 0
    return at


def work(case):
    lens = _lengths(case)
    hkv, D = case["Hkv"], case["D"]
    held = lambda n: hkv * ((n // BLOCK) * (2 * BLOCK * D + 8) + (n % BLOCK) * 4 * D)  # bytes of n tokens in the cache
    if case["op"] == "decode":
        rows = case["H"] * case["tq"]
        n = sum(held(x) for x in lens) + case["B"] * rows * (4 * D + 4)
        if case["weights"]:
            n += sum(4 * hkv * (x // BLOCK) for x in lens)
        return {"bytes": n, "flops": sum(4 * D * rows * x for x in lens)}
    if case["op"] == "sparse":
        rows = case["H"] * case["tq"]
        n = case["B"] * rows * (4 * D + 4) + case["B"] * hkv * case["tq"] * case["n"] * 4
        f = 0
        for x in lens:
            closed = x // BLOCK
            some = min(closed, case["n"])
            n += hkv * closed * (2 * D + 4) + held(min(closed, some * case["tq"]) * BLOCK + x % BLOCK)
            f += rows * (4 * D * closed + 4 * D * (some * BLOCK + x % BLOCK))
        return {"bytes": n, "flops": f}
    if case["op"] == "append":
        n = f = 0
        back = min(case["len"], RING) if case["new"] < case["len"] else case["len"]  # tokens read back
        for x in lens:
            new = min(case["new"], x)
            first = (x - new) // BLOCK
            closing = (x // BLOCK - first) * BLOCK  # tokens of the blocks that close
            old = (x - new) % BLOCK if closing else 0
            ring = min(new, max(0, x - (x // BLOCK - 1) * BLOCK))
            n += hkv * (4 * D * (new + old + ring) + 2 * D * closing + (closing // BLOCK) * (2 * D + 12))
            seen = min(x, back)
            n += hkv * (4 * D * back + held(seen))
            f += hkv * 6 * D * closing
        n += case["B"] * hkv * RING * 4 * D
        return {"bytes": n, "flops": f}
    n = 0
    for x in lens:
        closed = x // BLOCK
        kept = min(closed, case["keep"])
        n += hkv * (4 * closed + 2 * held(kept * BLOCK) + 4 * D * kept * BLOCK + 2 * kept * 2 * D + 8 * kept + 2 * RING * 4 * D)
    return {"bytes": n, "flops": sum(hkv * (x // BLOCK) for x in lens)}


# ------------------------------------------------- the cache's plain arithmetic


def _quantise(x):
    """Codes 1 .. 255 of [..., 64, D] tokens, as numbers around zero, and the scale of each block."""
    most = x.abs().amax(dim=(-2, -1), keepdim=True)
    codes = torch.where(most > 0, torch.round(x * 127 / most), torch.zeros_like(x))
    return codes, (most / 127)[..., 0, 0]


def _keys_out(codes):
    """[..., D / S, 64, S] codes to [..., 64, D] numbers."""
    x = codes.float() - 128
    return x.transpose(-3, -2).reshape(*x.shape[:-3], BLOCK, -1)


def _keys_in(x):
    """[..., 64, D] numbers to [..., D / S, 64, S] codes."""
    D = x.shape[-1]
    S = min(D, 64)
    return (x + 128).to(torch.uint8).reshape(*x.shape[:-1], D // S, S).transpose(-3, -2)


def _values_out(codes):
    return (codes.float() - 128).transpose(-2, -1)


def _values_in(x):
    return (x + 128).to(torch.uint8).transpose(-2, -1)


def _open_tokens(ring, lens):
    """The open block of each sequence, [B, Hkv, 64, D] (rows past its end are whatever the ring holds)."""
    at = (lens // BLOCK % 2 * BLOCK)[:, None] + torch.arange(BLOCK, device=ring.device)
    return ring.gather(2, at[:, None, :, None].expand(-1, ring.shape[1], -1, ring.shape[3]))


# ------------------------------------------------------------------ the inputs


def _rounds(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)
    B, hkv, D, op = case["B"], case["Hkv"], case["D"], case["op"]
    nb = max(1, _rounds(case["len"]))
    S = min(D, 64)
    s = {"case": case, "lens": torch.tensor(_lengths(case), dtype=torch.int32, device=dev)}
    shape = (B, hkv, nb)
    if op == "append":
        k_codes = torch.full((*shape, D // S, BLOCK, S), 128, dtype=torch.uint8, device=dev)
        v_codes = torch.full((*shape, D, BLOCK), 128, dtype=torch.uint8, device=dev)
        scales = torch.zeros(*shape, 2, device=dev)
        bounds = torch.zeros(*shape, 2, D, dtype=torch.int8, device=dev)
        weight = torch.zeros(*shape, device=dev)
    else:
        # keys share a part within a block, as neighbouring tokens do, and have strong channels
        keys = randn(*shape, BLOCK, D).mul_(0.8).add_(randn(*shape, 1, D), alpha=0.6)
        keys.mul_(1 + 2 * (torch.rand(1, hkv, 1, 1, D, generator=g, device=dev) < 0.05).float())
        numbers, k_scale = _quantise(keys)
        k_codes = _keys_in(numbers).contiguous()
        bounds = torch.stack([numbers.amin(dim=-2), numbers.amax(dim=-2)], dim=-2).to(torch.int8)
        del keys, numbers
        values = randn(*shape, BLOCK, D)
        numbers, v_scale = _quantise(values)
        v_codes = _values_in(numbers).contiguous()
        del values, numbers
        scales = torch.stack([k_scale, v_scale], dim=-1).contiguous()
        # what earlier steps left: a few blocks hold most of it; a decode step sets it anew
        weight = torch.exp(2 * randn(*shape)) if op == "evict" else torch.zeros(*shape, device=dev)
    ring = [randn(B, hkv, RING, D).to(torch.bfloat16) for _ in range(2)]
    s.update(k_codes=k_codes, v_codes=v_codes, scales=scales, bounds=bounds, weight=weight, recent_k=ring[0], recent_v=ring[1])
    if op in ("decode", "sparse"):
        s["q"] = (1.5 * randn(B, case["H"], case["tq"], D)).to(torch.bfloat16)
    if op == "append":
        n = case["new"]
        s["k"], s["v"] = ((randn(B, hkv, n, D) * (1 + (torch.rand(1, hkv, 1, D, generator=g, device=dev) < 0.05).float())).to(torch.bfloat16) for _ in range(2))
        s["new"] = torch.minimum(s["lens"], torch.full_like(s["lens"], n))
        s["back"] = case["len"] if n == case["len"] else min(case["len"], RING)
        # read back from the start of the oldest block that an append touches
        s["starts"] = torch.clamp((s["lens"] - s["new"]) // BLOCK * BLOCK, min=0).to(torch.int32)
    if own:
        import decoder_only_transformer_sdpa_b200 as attn

        parts = ("k_codes", "v_codes", "scales", "bounds", "weight", "recent_k", "recent_v")
        s["cache"] = attn.Q8Cache(*(s[p] for p in parts))
        if op == "evict":
            s["room"] = attn.Q8Cache.empty(B, hkv, D, case["keep"] * BLOCK, device=dev)
    return s


# ---------------------------------------------------------------- the plain form


def _dense(q, keys, values, seen, scale):
    """Softmax attention of q [B, Hkv, R, D] over keys and values [B, Hkv, T, D] where `seen` [B, 1 or Hkv, R, T]: o, lse and weights."""
    s = torch.matmul(q, keys.transpose(-2, -1)) * scale
    s = s.masked_fill(~seen, float("-inf"))
    most = s.amax(dim=-1, keepdim=True)
    most = torch.where(most > float("-inf"), most, torch.zeros_like(most))
    p = torch.exp(s - most)
    total = p.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    return torch.matmul(p, values), (most + torch.log(total))[..., 0], p


def _plain_decode(s):
    case = s["case"]
    q, lens, tq = s["q"], s["lens"], case["tq"]
    B, H, _, D = q.shape
    hkv, nb = case["Hkv"], s["k_codes"].shape[2]
    rows = q.float().reshape(B, hkv, -1, D)
    closed = lens // BLOCK
    keys = (_keys_out(s["k_codes"]) * s["scales"][..., 0, None, None]).reshape(B, hkv, -1, D)
    values = (_values_out(s["v_codes"]) * s["scales"][..., 1, None, None]).reshape(B, hkv, -1, D)
    keys = torch.cat([keys, _open_tokens(s["recent_k"], lens).float()], dim=2)
    values = torch.cat([values, _open_tokens(s["recent_v"], lens).float()], dim=2)
    at = torch.arange(nb * BLOCK, device=q.device)
    position = torch.cat([at.expand(B, -1), (closed * BLOCK)[:, None] + torch.arange(BLOCK, device=q.device)], dim=1)
    there = torch.cat([at < (closed * BLOCK)[:, None], torch.ones(B, BLOCK, dtype=torch.bool, device=q.device)], dim=1)
    mine = lens[:, None] - tq + torch.arange(tq, device=q.device)
    seen = there[:, None, :] & (position[:, None, :] <= mine[:, :, None])
    seen = seen.repeat(1, H // hkv, 1)[:, None]
    o, lse, p = _dense(rows, keys, values, seen, D**-0.5)
    out = {"o": o.reshape(B, H, tq, D).to(torch.bfloat16), "lse": lse.reshape(B, H, tq)}
    if case["weights"]:
        got = p[..., : nb * BLOCK].reshape(B, hkv, -1, nb, BLOCK).sum(dim=(2, 4))
        s["weight"].copy_(torch.where(torch.arange(nb, device=q.device) < closed[:, None, None], got, s["weight"]))
        out["weight"] = s["weight"]
    return out


def _plain_select(s):
    """The n best blocks of each key head for each new token, ascending, -1 where there are fewer."""
    case = s["case"]
    q, lens, tq, n = s["q"], s["lens"], case["tq"], case["n"]
    B, H, _, D = q.shape
    hkv, nb = case["Hkv"], s["k_codes"].shape[2]
    x = q.float().reshape(B, hkv, H // hkv, tq, D)
    most = x.abs().amax(dim=-1, keepdim=True)
    c = torch.where(most > 0, torch.round(x * 127 / most), torch.zeros_like(x))
    low, high = s["bounds"][:, :, None, :, 0].float(), s["bounds"][:, :, None, :, 1].float()
    # sums of whole numbers below 2^24, exact in float32
    dot = torch.matmul(c.clamp(min=0), high.transpose(-2, -1)) + torch.matmul(c.clamp(max=0), low.transpose(-2, -1))
    score = (dot * s["scales"][:, :, None, None, :, 0] * (most / 127)).amax(dim=2)
    last = lens[:, None] - tq + torch.arange(tq, device=q.device)
    j = torch.arange(nb, device=q.device)
    open_to = (j < (lens // BLOCK)[:, None, None]) & (j * BLOCK <= last[:, :, None])
    score = score.masked_fill(~open_to[:, None], float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True)
    best = torch.where(order.values > float("-inf"), order.indices, nb)
    best = torch.nn.functional.pad(best, (0, max(0, n - nb)), value=nb)[..., :n].sort(dim=-1).values
    return torch.where(best < nb, best, -1).to(torch.int32)


def _plain_sparse(s):
    case = s["case"]
    q, lens, tq = s["q"], s["lens"], case["tq"]
    B, H, _, D = q.shape
    hkv = case["Hkv"]
    blocks = _plain_select(s)
    n = blocks.shape[-1]
    b = torch.arange(B, device=q.device)[:, None, None, None]
    h = torch.arange(hkv, device=q.device)[None, :, None, None]
    at = blocks.long().clamp(min=0)
    scales = s["scales"][b, h, at]
    keys = (_keys_out(s["k_codes"][b, h, at]) * scales[..., 0, None, None]).reshape(B, hkv, tq, -1, D)
    values = (_values_out(s["v_codes"][b, h, at]) * scales[..., 1, None, None]).reshape(B, hkv, tq, -1, D)
    last_k = _open_tokens(s["recent_k"], lens).float()[:, :, None].expand(-1, -1, tq, -1, -1)
    last_v = _open_tokens(s["recent_v"], lens).float()[:, :, None].expand(-1, -1, tq, -1, -1)
    i = torch.arange(BLOCK, device=q.device)
    position = torch.cat([(at[..., None] * BLOCK + i).reshape(B, hkv, tq, -1), (lens // BLOCK * BLOCK)[:, None, None, None].expand(-1, hkv, tq, -1) + i], dim=-1)
    there = torch.cat([(blocks >= 0)[..., None].expand(-1, -1, -1, -1, BLOCK).reshape(B, hkv, tq, -1), torch.ones(B, hkv, tq, BLOCK, dtype=torch.bool, device=q.device)], dim=-1)
    mine = lens[:, None] - tq + torch.arange(tq, device=q.device)
    seen = there & (position <= mine[:, None, :, None])
    rows = q.float().reshape(B, hkv, H // hkv, tq, D).transpose(2, 3)
    o, lse, _ = _dense(rows, torch.cat([keys, last_k], dim=3), torch.cat([values, last_v], dim=3), seen[..., None, :], D**-0.5)
    return {"blocks": blocks, "o": o.transpose(2, 3).reshape(B, H, tq, D).to(torch.bfloat16), "lse": lse.transpose(2, 3).reshape(B, H, tq)}


def _plain_read(codes_k, codes_v, scales, ring_k, ring_v, lens, starts, n):
    """Keys and values of positions starts + 0 .. n - 1 as they are held, zero past the end."""
    B, hkv, nb = scales.shape[:3]
    at = starts[:, None].long() + torch.arange(n, device=lens.device)
    closed = (lens // BLOCK * BLOCK)[:, None]
    b = torch.arange(B, device=lens.device)[:, None, None]
    h = torch.arange(hkv, device=lens.device)[None, :, None]
    block, row, spot = (at // BLOCK).clamp(max=nb - 1)[:, None], (at % BLOCK)[:, None], (at % RING)[:, None]
    x = codes_k[b, h, block, :, row].float().flatten(-2) - 128
    y = codes_v[b, h, block, :, row].float() - 128
    scale = scales[b, h, block]
    old = (at < closed)[:, None, :, None]
    held = (at < lens[:, None])[:, None, :, None]
    x = torch.where(old, x * scale[..., 0, None], ring_k[b, h, spot].float())
    y = torch.where(old, y * scale[..., 1, None], ring_v[b, h, spot].float())
    return tuple(torch.where(held, t, torch.zeros_like(t)).to(torch.bfloat16) for t in (x, y))


def _plain_append(s):
    case = s["case"]
    k, v, lens, new = s["k"], s["v"], s["lens"].long(), s["new"].long()
    B, hkv, n, D = k.shape
    nb = s["k_codes"].shape[2]
    dev = k.device
    first = (lens - new) // BLOCK  # the oldest block with a new token
    nt = min(nb, n // BLOCK + 2 if n < case["len"] else _rounds(n))
    block = first[:, None] + torch.arange(nt, device=dev)
    at = (block * BLOCK)[..., None] + torch.arange(BLOCK, device=dev)
    row = (at - (lens - new)[:, None, None]).reshape(B, -1)
    closing = block < (lens // BLOCK)[:, None]
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(hkv, device=dev)[None, :, None]
    shut = closing[:, None].expand(-1, hkv, -1)
    bi, hi, ji = (t.expand(B, hkv, nt)[shut] for t in (b, h, block[:, None]))
    for x, ring, side in ((k, s["recent_k"], 0), (v, s["recent_v"], 1)):
        fresh = x[b, h, row.clamp(min=0, max=n - 1)[:, None]]
        tokens = torch.where((row >= 0)[:, None, :, None], fresh, ring[b, h, (at.reshape(B, -1) % RING)[:, None]])
        numbers, scale = _quantise(tokens.float().reshape(B, hkv, nt, BLOCK, D)[shut])
        s["scales"][bi, hi, ji, side] = scale
        if side == 0:
            s["k_codes"][bi, hi, ji] = _keys_in(numbers)
            s["bounds"][bi, hi, ji] = torch.stack([numbers.amin(dim=-2), numbers.amax(dim=-2)], dim=-2).to(torch.int8)
        else:
            s["v_codes"][bi, hi, ji] = _values_in(numbers)
        # the newest positions, as far back as the start of the last closed block, stay in bf16
        spot = torch.arange(RING, device=dev)
        newest = spot + torch.div(lens[:, None] - 1 - spot, RING, rounding_mode="floor") * RING
        goes = (newest >= (lens - new)[:, None]) & (newest >= ((lens // BLOCK - 1) * BLOCK)[:, None]) & (newest >= 0)
        from_row = (newest - (lens - new)[:, None]).clamp(min=0, max=n - 1)
        ring.copy_(torch.where(goes[:, None, :, None], x[b, h, from_row[:, None]], ring))
    s["weight"][bi, hi, ji] = 0
    held = _plain_read(s["k_codes"], s["v_codes"], s["scales"], s["recent_k"], s["recent_v"], s["lens"], s["starts"], s["back"])
    return {"k": held[0], "v": held[1], "scales": s["scales"], "bounds": s["bounds"], "weight": s["weight"], "recent_k": s["recent_k"], "recent_v": s["recent_v"]}


def _plain_evict(s):
    case = s["case"]
    lens, keep = s["lens"], case["keep"]
    B, hkv, nb = s["weight"].shape
    dev = lens.device
    closed = (lens // BLOCK)[:, None, None]
    j = torch.arange(nb, device=dev)
    weight = s["weight"].masked_fill((j < case["sink"]) | (j >= closed - case["recent"]), float("inf"))
    weight = weight.masked_fill(j >= closed, float("-inf"))
    order = torch.sort(weight, dim=-1, descending=True, stable=True)
    best = torch.where(order.values > float("-inf"), order.indices, nb)
    best = torch.nn.functional.pad(best, (0, max(0, keep - nb)), value=nb)[..., :keep].sort(dim=-1).values
    kept = torch.where(best < nb, best, -1).to(torch.int32)
    some = kept >= 0
    at = kept.long().clamp(min=0)
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(hkv, device=dev)[None, :, None]
    none = lambda t, m: torch.where(some.reshape(some.shape + (1,) * (t.dim() - 3)), t, torch.full_like(t, m))
    after = (torch.minimum(closed[:, 0, 0], torch.full_like(lens, keep)) * BLOCK + lens % BLOCK).to(torch.int32)
    # the recent positions move with the count of blocks that go: an odd count exchanges the halves
    odd = ((lens - after) // BLOCK % 2 == 1)[:, None, None, None]
    ring = [torch.where(odd, s[r].roll(BLOCK, dims=2), s[r]) for r in ("recent_k", "recent_v")]
    k_codes, v_codes = s["k_codes"][b, h, at], s["v_codes"][b, h, at]
    scales = none(s["scales"][b, h, at], 0)
    held = _plain_read(k_codes, v_codes, scales, ring[0], ring[1], after, torch.zeros_like(lens), keep * BLOCK)
    return {"lens": after, "kept": kept, "k": held[0], "v": held[1], "scales": scales, "bounds": none(s["bounds"][b, h, at], 0), "weight": none(s["weight"][b, h, at], 0), "recent_k": ring[0], "recent_v": ring[1]}


# ------------------------------------------------------------- the package's calls


def _own(s):
    import decoder_only_transformer_sdpa_b200 as attn

    case, cache, lens = s["case"], s["cache"], s["lens"]
    if case["op"] == "decode":
        if case["weights"]:
            o, lse = attn.attn_q8_decode(s["q"], cache, lens, weight="set")
            return {"o": o, "lse": lse, "weight": s["weight"]}
        o, lse = attn.attn_q8_decode(s["q"], cache, lens)
        return {"o": o, "lse": lse}
    if case["op"] == "sparse":
        blocks = attn.attn_q8_select(s["q"], cache, lens, case["n"])
        o, lse = attn.attn_q8_decode(s["q"], cache, lens, blocks=blocks)
        return {"blocks": blocks, "o": o, "lse": lse}
    if case["op"] == "append":
        attn.attn_q8_append(cache, s["k"], s["v"], lens, s["new"])
        k, v = attn.attn_q8_read(cache, lens, s["back"], starts=s["starts"])
        return {"k": k, "v": v, "scales": s["scales"], "bounds": s["bounds"], "weight": s["weight"], "recent_k": s["recent_k"], "recent_v": s["recent_v"]}
    room = s["room"]
    after, kept = attn.attn_q8_evict(cache, lens, case["keep"], sink=case["sink"], recent=case["recent"], out=room)
    k, v = attn.attn_q8_read(room, after, case["keep"] * BLOCK)
    return {"lens": after, "kept": kept, "k": k, "v": v, "scales": room.scales, "bounds": room.bounds, "weight": room.weight, "recent_k": room.recent_k, "recent_v": room.recent_v}


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "sparse": _plain_sparse, "append": _plain_append, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------- the definition in 64 bits


def _held_exactly(s, b):
    """Sequence b's keys and values, [Hkv, length, D] in 64 bits, by walking over its tokens."""
    n = int(s["lens"][b])
    closed = n // BLOCK
    hkv, D = s["recent_k"].shape[1], s["recent_k"].shape[3]
    k = s["k_codes"][b, :, :closed].double().permute(0, 1, 3, 2, 4).reshape(hkv, closed, BLOCK, D) - 128
    v = s["v_codes"][b, :, :closed].double().permute(0, 1, 3, 2).reshape(hkv, closed, BLOCK, D) - 128
    k = k * s["scales"][b, :, :closed, 0].double()[:, :, None, None]
    v = v * s["scales"][b, :, :closed, 1].double()[:, :, None, None]
    spots = [p % RING for p in range(closed * BLOCK, n)]
    k = torch.cat([k.reshape(hkv, -1, D), s["recent_k"][b][:, spots].double()], dim=1)
    v = torch.cat([v.reshape(hkv, -1, D), s["recent_v"][b][:, spots].double()], dim=1)
    return k, v


def _chosen_exactly(s):
    """The blocks of the sparse attention. The score is a sum of whole numbers, multiplied by two float32 numbers with a rounding to float32 after each."""
    case, q, lens = s["case"], s["q"].double(), s["lens"].tolist()
    B, H, tq, D = q.shape
    hkv, G = case["Hkv"], H // case["Hkv"]
    chosen = torch.full((B, hkv, tq, case["n"]), -1, dtype=torch.int32, device=q.device)
    for b in range(B):
        for r in range(tq):
            mine = lens[b] - tq + r
            some = min(lens[b] // BLOCK, mine // BLOCK + 1) if mine >= 0 else 0
            if some == 0:
                continue
            best = None
            for g in range(G):
                x = q[b, :, r].reshape(hkv, G, D)[:, g]
                most = x.abs().amax(dim=-1, keepdim=True)
                c = torch.round(127 * x / torch.where(most > 0, most, torch.ones_like(most))).long()[:, None]
                ends = s["bounds"][b, :, :some].long()
                dot = torch.maximum(c * ends[:, :, 0], c * ends[:, :, 1]).sum(dim=-1)
                step = (most / 127).float()
                score = (dot.double() * s["scales"][b, :, :some, 0].double()).float()
                score = (score.double() * step.double()).float()
                best = score if best is None else torch.maximum(best, score)
            order = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : case["n"]]
            chosen[b, :, r, : order.shape[1]] = order.sort(dim=-1).values.int()
    return chosen


def exact(case, seed):
    s = prepare(case, seed)
    dev = s["lens"].device
    if case["op"] in ("decode", "sparse"):
        B, H, tq, D = s["q"].shape
        hkv, G = case["Hkv"], H // case["Hkv"]
        blocks = _chosen_exactly(s) if case["op"] == "sparse" else None
        o = torch.zeros(B, H, tq, D, dtype=torch.float64, device=dev)
        lse = torch.full((B, H, tq), float("-inf"), dtype=torch.float64, device=dev)
        weight = s["weight"].double()
        for b in range(B):
            n = int(s["lens"][b])
            if n == 0:
                continue
            k, v = _held_exactly(s, b)
            got = torch.zeros(hkv, n, dtype=torch.float64, device=dev)
            for r in range(tq):
                sees = n - tq + r + 1
                if sees < 1:
                    continue
                use = torch.zeros(hkv, n, dtype=torch.bool, device=dev)
                if blocks is None:
                    use[:, :sees] = True
                else:
                    mark = torch.zeros(hkv, n // BLOCK + 1, dtype=torch.bool, device=dev)
                    chosen = blocks[b, :, r].long()
                    mark.scatter_(1, torch.where(chosen >= 0, chosen, torch.full_like(chosen, n // BLOCK)), True)
                    mark[:, n // BLOCK] = True  # the open block
                    use = mark.repeat_interleave(BLOCK, dim=1)[:, :n] & (torch.arange(n, device=dev) < sees)
                x = torch.einsum("hgd,htd->hgt", s["q"][b, :, r].double().reshape(hkv, G, D), k) / D**0.5
                x = x.masked_fill(~use[:, None], float("-inf"))
                all_of = torch.logsumexp(x, dim=-1)
                p = torch.exp(x - all_of[..., None]).nan_to_num(0.0)
                o[b, :, r] = torch.einsum("hgt,htd->hgd", p, v).reshape(H, D)
                lse[b, :, r] = all_of.reshape(H)
                got += p.sum(dim=1)
            closed = n // BLOCK
            weight[b, :, :closed] = got[:, : closed * BLOCK].reshape(hkv, closed, BLOCK).sum(dim=-1)
        out = {"o": o, "lse": lse}
        if case["op"] == "sparse":
            out["blocks"] = blocks
        elif case["weights"]:
            out["weight"] = weight
        return out
    if case["op"] == "append":
        k0, v0 = torch.zeros(2, case["B"], case["Hkv"], s["back"], case["D"], dtype=torch.float64, device=dev)
        scales, recent = s["scales"].double(), [s["recent_k"].clone(), s["recent_v"].clone()]
        for b in range(case["B"]):
            n, m = int(s["lens"][b]), int(s["new"][b])
            start, closed = int(s["starts"][b]), n // BLOCK
            for side, (x, ring, out) in enumerate(((s["k"], s["recent_k"], k0), (s["v"], s["recent_v"], v0))):
                old = [p % RING for p in range(start, n - m)]
                tokens = torch.cat([ring[b][:, old], x[b, :, :m]], dim=1).double()  # positions start .. n - 1
                whole = (closed * BLOCK - start) // BLOCK
                if whole > 0:
                    block = tokens[:, : whole * BLOCK].reshape(case["Hkv"], whole, BLOCK, -1)
                    step = block.abs().amax(dim=(2, 3)) / 127
                    scales[b, :, start // BLOCK : closed, side] = step
                    unit = torch.where(step > 0, step, torch.ones_like(step))[:, :, None, None]
                    # 127 x / most itself, so that what lies half-way between two codes stays there
                    most = block.abs().amax(dim=(2, 3), keepdim=True)
                    code = torch.round(127 * block / torch.where(most > 0, most, torch.ones_like(most)))
                    tokens = torch.cat([(code * unit).flatten(1, 2), tokens[:, whole * BLOCK :]], dim=1)
                there = min(s["back"], n - start)
                out[b, :, :there] = tokens[:, :there]
                for p in range(max(n - m, (closed - 1) * BLOCK, 0), n):
                    recent[side][b, :, p % RING] = x[b, :, p - (n - m)]
        return {"k": k0, "v": v0, "scales": scales, "bounds": None, "weight": None, "recent_k": recent[0].double(), "recent_v": recent[1].double()}
    B, hkv, keep, D = case["B"], case["Hkv"], case["keep"], case["D"]
    if B * hkv > 600:
        return None
    k, v = torch.zeros(2, B, hkv, keep * BLOCK, D, dtype=torch.float64, device=dev)
    for b in range(B):
        closed = int(s["lens"][b]) // BLOCK
        held = _held_exactly(s, b)
        for h in range(hkv):
            w = s["weight"][b, h, :closed].double().tolist()
            free = list(range(case["sink"], max(case["sink"], closed - case["recent"])))
            must = sorted(set(range(closed)) - set(free))
            free = [j for j in free if j < closed]
            some = sorted(free, key=lambda j: (-w[j], j))[: max(0, min(keep, closed) - len(must))]
            for i, j in enumerate(sorted(must + some)):
                k[b, h, i * BLOCK : (i + 1) * BLOCK] = held[0][h, j * BLOCK : (j + 1) * BLOCK]
                v[b, h, i * BLOCK : (i + 1) * BLOCK] = held[1][h, j * BLOCK : (j + 1) * BLOCK]
            n, after = int(s["lens"][b]), min(keep, closed)
            rest = min(keep * BLOCK, after * BLOCK + n % BLOCK) - after * BLOCK
            if rest > 0:
                k[b, h, after * BLOCK : after * BLOCK + rest] = held[0][h, closed * BLOCK : closed * BLOCK + rest]
                v[b, h, after * BLOCK : after * BLOCK + rest] = held[1][h, closed * BLOCK : closed * BLOCK + rest]
    return {"lens": None, "kept": None, "k": k, "v": v, "scales": None, "bounds": None, "weight": None, "recent_k": None, "recent_v": None}
