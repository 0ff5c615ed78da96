"""The paged 8-bit cache's operators in float64 on the CPU, token by token, and the
bounds that the GPU's results are held to. Shares no code with the library.

Bounds (u = a rounding's largest relative error: float32 2^-24, f16 2^-11, bf16 2^-8,
e4m3 2^-4):
  rotation in float32: cos and sin within 2^-23 of the true ones, two products and a sum
      rounded: an error of at most (|x_i| + |x_j|) (2^-23 + 2 * 2^-24) =: (|x_i| + |x_j|) 2^-22.
  decode: a score is a float32 sum of 128 products, off by at most 128 * 2^-23 times the
      sum A of their magnitudes (a matrix instruction may cut where it does not round:
      2^-23 a step). q goes in as the sum of four e4m3 terms, each the rounded rest of the
      ones before, 2^4 apart: what is left after the last is half its smallest step, 2^-10 / 2^12
      with the largest value scaled to at least 2^7: 2^-29 max|q| an element. Then the score is scaled
      (three roundings) and, like the row's reference, taken as a power of two: p is off by
      a relative 2 ((128 * 2^-23 + 4 * 2^-24) A + 2^-29 max|q| sum|k|) + 2^-21. P is rounded
      to f16 for the product with V: 2^-11. It goes in as four e4m3 terms in the same way, scaled
      to 2^8 at a reference that is at most the row's largest p: what is left is at most
      2^-10 / 2^12 / 2^8 = 2^-30 of that largest p, and f16's own smallest step, 2^-25 / 2^8, is
      less. Where a tile's pages have different value scales, a key's P takes the ratio of its
      scale to the tile's largest, u (one more rounding of 2^-24), and the rest counts against
      u |v8| instead of |v| = scale |v8|. The sum l has the same error as p. Then the
      output's rounding to bf16. With S = sum p |v|, U = (largest p) * sum u |v8| (tile by tile
      its own u; sum |v| where the scales are one):
      |o - ref| <= 2^-8 |ref| + S (2^-11 + 4 (129 * 2^-23 A + 2^-29 max|q| sum|k|) + 2^-20) + 2^-30 U.
"""

from __future__ import annotations

import math

import numpy as np
import torch

D = 128


def _e4m3_table():
    t = np.empty(256)
    for b in range(256):
        s, e, m = (-1.0 if b & 128 else 1.0), (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            t[b] = np.nan
        elif e == 0:
            t[b] = s * m * 2.0 ** -9
        else:
            t[b] = s * (1 + m / 8) * 2.0 ** (e - 7)
    return t


E4M3 = _e4m3_table()


def round_e4m3(x):
    """Nearest e4m3 value, ties to even, of |x| <= 448; NaN where not finite."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.maximum(np.frexp(np.abs(np.where(np.isfinite(x), x, 1.0)))[1] - 1, -6)
        step = np.ldexp(1.0, e - 3)
        y = np.rint(x / step) * step
    return np.where(np.isfinite(x), y, np.nan)


def half_step_e4m3(x):
    e = np.maximum(np.frexp(np.abs(x))[1] - 1, -6)
    return np.ldexp(0.5, e - 3)


def bytes_of(t):
    return t.detach().contiguous().view(torch.uint8).cpu().numpy()


def values_of(t):
    return E4M3[bytes_of(t)]


def least_scale(amax):
    e = -100
    if amax > 0:
        e = max(-100, math.frexp(amax)[1] - 10)
        while amax > 448.0 * 2.0 ** e:
            e += 1
        while e > -100 and amax <= 448.0 * 2.0 ** (e - 1):
            e -= 1
    return 2.0 ** e


def rotated(x, pos, inv_freq, interleaved):
    """(rotated rows, bound of a float32 rotation's error): x [..., 128] float64."""
    y, tol = x.copy(), np.zeros_like(x)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = float(pos) * float(inv_freq[i])
        c, s = math.cos(ang), math.sin(ang)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        tol[..., a] = tol[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * 2.0 ** -22
    return y, tol


class RefCache:
    """Copies of a cache's tensors (values, not bytes) that append() changes as the
    operator is defined to. ``exact`` holds, for every element that an append wrote, the
    value before its rounding (NaN elsewhere) and ``tol`` its float32 error."""

    def __init__(self, k_pages, v_pages, k_scale, v_scale, table):
        self.val = [values_of(k_pages), values_of(v_pages)]
        self.scale = [k_scale.double().cpu().numpy().copy(), v_scale.double().cpu().numpy().copy()]
        self.table = table.cpu().numpy()
        self.exact = [np.full_like(x, np.nan) for x in self.val]
        self.tol = [np.zeros_like(x) for x in self.val]
        self.page = k_pages.shape[2]
        self.n_pages = k_pages.shape[0]

    def append(self, k, v, lens, cu=None, inv_freq=None, interleaved=False, q=None, max_new=None):
        f64 = lambda t: None if t is None else t.detach().double().cpu().numpy()  # noqa: E731
        k, v, q, freq = f64(k), f64(v), f64(q), f64(inv_freq)
        q_out = None if q is None else np.full_like(q, np.nan)
        q_tol = None if q is None else np.zeros_like(q)
        page = self.page
        for b, n in enumerate(lens):
            first, m = (b, 1) if cu is None else (cu[b], cu[b + 1] - cu[b])
            if m <= 0 or n < m or (max_new is not None and m > max_new):
                continue
            start = n - m
            for slot in range(start // page, (n - 1) // page + 1):
                lo, hi = max(start, slot * page), min(n, (slot + 1) * page)
                rows = [first + p - start for p in range(lo, hi)]
                if q is not None:
                    for p, r in zip(range(lo, hi), rows):
                        q_out[r], q_tol[r] = rotated(q[r], p, freq, interleaved)
                pid = int(self.table[b, slot]) if slot < self.table.shape[1] else -1
                if not 0 <= pid < self.n_pages:
                    continue
                for w, src in enumerate((k, v)):
                    new = [(src[r], np.zeros_like(src[r])) for r in rows]
                    if w == 0:
                        new = [rotated(src[r], p, freq, interleaved)
                               for p, r in zip(range(lo, hi), rows)]
                    for h in range(src.shape[1]):
                        xs = np.stack([x[h] for x, _ in new])
                        fin = np.abs(xs[np.isfinite(xs)])
                        s = least_scale(fin.max() if fin.size else 0.0)
                        used = lo - slot * page
                        if used:
                            old = self.scale[w][pid, h]
                            s = max(s, old)
                            kept = self.val[w][pid, h, :used]
                            self.val[w][pid, h, :used] = round_e4m3(kept * (old / s))
                        self.scale[w][pid, h] = s
                        at = (pid, h, slice(used, used + len(rows)))
                        self.exact[w][at] = xs / s
                        self.tol[w][at] = np.stack([t[h] for _, t in new]) / s
                        self.val[w][at] = round_e4m3(xs / s)
        return q_out, q_tol

    def check(self, k_pages, v_pages, k_scale, v_scale):
        """The cache's tensors against this one: scales and values equal, but that an
        element next to a tie may fall on either side of it."""
        for w, (pages, scale) in enumerate(((k_pages, k_scale), (v_pages, v_scale))):
            assert np.array_equal(scale.double().cpu().numpy(), self.scale[w], equal_nan=True), "scales"
            got, want = values_of(pages), self.val[w]
            assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN places"
            off = (got != want) & ~np.isnan(want)
            if off.any():
                x, t = self.exact[w][off], self.tol[w][off]
                assert np.isfinite(x).all(), "an element that no append wrote has changed"
                assert (np.abs(got[off] - x) <= half_step_e4m3(x) + t).all(), "rounding"
                assert off.mean() < 1e-3


def sequence(cache_tensors, table, b, n):
    """K, V [Hkv, n, 128] float64 of sequence b."""
    return _sequence(cache_tensors, table, b, n)[:2]


def _sequence(cache_tensors, table, b, n):
    """K, V, and |v8| times the largest value scale of the key's 128-key tile."""
    k_pages, v_pages, k_scale, v_scale = cache_tensors
    page = k_pages.shape[2]
    ids = table[b, :-(-n // page)].long().cpu().numpy()
    out = []
    for pages, scale in ((k_pages, k_scale), (v_pages, v_scale)):
        x = values_of(pages[torch.as_tensor(ids, device=pages.device)]
                      if pages.dtype == torch.uint8 else
                      pages.view(torch.uint8)[torch.as_tensor(ids, device=pages.device)])
        s = scale.double().cpu().numpy()[ids]                       # [pages, Hkv]
        per = 128 // page
        tops = np.maximum.reduceat(np.abs(s), np.arange(0, len(ids), per), axis=0)
        u = np.repeat(tops, per, axis=0)[:len(ids)]
        for y in (x * s[:, :, None, None], np.abs(x) * u[:, :, None, None]):
            out.append(y.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, D)[:, :n])
    return out[0], out[2], out[3]


def decode_bound(q, K, V, ref, keep_keys, coarse=None):
    """|o - ref| bound of one query head: q [128], K, V [n, 128], keep_keys [n] bool,
    coarse: u |v8| [n, 128] (|V| when None)."""
    k = K[keep_keys]
    A = (np.abs(k) @ np.abs(q)).max() / math.sqrt(D)
    B = 2.0 ** -29 * np.abs(q).max() * np.abs(k).sum(-1).max() / math.sqrt(D)
    s = (k @ q) / math.sqrt(D)
    p = np.exp(s - s.max())
    p /= p.sum()
    v = np.abs(V[keep_keys])
    S = p @ v
    U = p.max() * (v if coarse is None else coarse[keep_keys]).sum(0)
    return 2.0 ** -8 * np.abs(ref) + S * (2.0 ** -11 + 4 * (129 * 2.0 ** -23 * A + B) + 2.0 ** -20) \
        + 2.0 ** -30 * U
