"""The 8-bit block cache in plain numpy, in 64 bits, written from its
definition (include/attn.h): a list of tokens for each sequence, quantised
block by block, and the attention over what is held.  Shares no code with the
library.

Error bounds of the attention (see ``bounds``).  With x = the exact value:

* scores: products of a bf16 query and an 8-bit code are exact, the D of them
  are summed in float32, each addition off by at most one unit 2^-23 of the
  sum of their absolute values (tensor cores may truncate), and three more
  float32 roundings scale the sum:
      es = (D + 3) 2^-23 * max_j sum_d |q_d k_jd| * scale  (+ 2^-38 max|q| ...)
  the last part for query values below 2^-31 of the row's largest.
* weights: exp2 of a float32 difference, off by 2^-22 relatively (ex2.approx:
  2 units) and by the difference's own rounding, 2^-24 of its size, which is
  at most 2 max|s| log2(e); P then is rounded to f16, 2^-11, in the products
  with the values only.
      ew = 2 es + 2^-21 + 2^-22 max|s|
* o: |do| <= 2^-8 |o| (bf16 output) + (ew + 2^-11 + n 2^-23) sum_j p_j |v_j|,
  n = 64 additions in a block and one a block in the accumulators; where a
  long row's sum of n terms is split over many warps its error grows with the
  longest chain only, so n = 64 + 2 * blocks / 8 covers every split.
* lse: es + 2^-21 + (|lse| + 1) 2^-22 * 4, and a block's weight the relative
  error of its terms: 2 ew + n 2^-23.
"""
from __future__ import annotations

import numpy as np
import torch

BLOCK, RING = 64, 128


def bf16(x):
    """Rounds to bf16, as float64."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def quantise(x):
    """codes [64, D] (0 .. 255) and the float32 scale of one block, [64, D] float64 (bf16 values)."""
    if not np.all(np.isfinite(x)):
        return np.full(x.shape, 128, np.uint8), np.float32(np.nan)
    most = np.max(np.abs(x))
    if most == 0:
        return np.full(x.shape, 128, np.uint8), np.float32(0)
    return (128 + np.rint(127 * x / most)).astype(np.uint8), np.float32(most) / np.float32(127)


class Sequence:
    """One sequence and key head: its tokens in bf16, and what is held of them."""

    def __init__(self, k, v):
        """k, v: [n, D] float64 arrays of bf16 values."""
        self.k, self.v = k, v
        n = len(k)
        self.closed = n // BLOCK
        self.k_codes, self.v_codes, self.scales = [], [], []
        hk, hv = [], []
        for j in range(self.closed):
            at = slice(j * BLOCK, (j + 1) * BLOCK)
            kc, ks = quantise(k[at])
            vc, vs = quantise(v[at])
            self.k_codes.append(kc)
            self.v_codes.append(vc)
            self.scales.append((ks, vs))
            hk.append((kc.astype(np.float64) - 128) * np.float64(ks))
            hv.append((vc.astype(np.float64) - 128) * np.float64(vs))
        D = k.shape[1]
        self.held_k = np.concatenate(hk + [k[self.closed * BLOCK:]]).reshape(n, D)
        self.held_v = np.concatenate(hv + [v[self.closed * BLOCK:]]).reshape(n, D)

    def bounds(self):
        c = np.stack(self.k_codes).astype(np.int64) - 128
        return np.stack([c.min(axis=1), c.max(axis=1)], axis=1).astype(np.int8)


def attend(q, k, v, use, scale):
    """One query row: o, lse and weights over the tokens where `use`; and the bounds' ingredients."""
    s = (k @ q) * scale
    a = (np.abs(k) @ np.abs(q)) * scale
    if not use.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(len(k)), 0.0, 0.0, np.zeros(v.shape[1])
    m = s[use].max()
    p = np.where(use, np.exp(np.where(use, s - m, 0)), 0)
    total = p.sum()
    p /= total
    vu = np.where(use[:, None], v, 0)
    return p @ vu, m + np.log(total), p, a[use].max(), np.abs(s[use]).max(), p @ np.abs(vu)


def tolerances(D, blocks, scale, q, k, a_max, s_max, o, lse, pv):
    """(bound on |do| per channel, bound on |d lse|, relative bound on a weight)."""
    es = (D + 3) * 2.0**-23 * a_max + D * 2.0**-38 * np.abs(q).max() * (np.abs(k).max() if k.size else 0) * scale
    ew = 2 * es + 2.0**-21 + 2.0**-22 * s_max
    n = (64 + 2 * blocks / 8) * 2.0**-23
    return 2.0**-8 * np.abs(o) + (ew + 2.0**-11 + n) * pv + 1e-30, es + 2.0**-21 + 4 * (abs(lse) + 1) * 2.0**-22, 2 * ew + n


def scores(seq, q_heads, closed):
    """The float32 score of each of the first `closed` blocks for the query heads [G, D] of a group."""
    if closed == 0:
        return np.zeros(0, np.float32)
    lo, hi = (x.astype(np.int64) for x in np.moveaxis(seq.bounds()[:closed], 1, 0))
    best = np.full(closed, -np.inf, np.float32)
    for q in q_heads:
        most = np.abs(q).max()
        c = np.rint(127 * q / most).astype(np.int64) if most > 0 else np.zeros(len(q), np.int64)
        dot = np.maximum(c * lo, c * hi).sum(axis=1)
        ks = np.array([s[0] for s in seq.scales[:closed]], np.float32)
        best = np.maximum(best, (dot.astype(np.float32) * ks) * (np.float32(most) / np.float32(127)))
    return best


def best_of(score, n):
    """The places of the n largest, ties to the lowest, ascending, -1 behind them."""
    order = sorted(range(len(score)), key=lambda j: (-float(score[j]), j))[:n]
    return sorted(order) + [-1] * (n - len(order))
