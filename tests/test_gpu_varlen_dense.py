"""mala_fwd_varlen at tau = 0 (exact attention) over packed chunks, against the oracle:
every legal tile is kept, whatever its scores."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
from tests.parity import TOL, as_f64, rel_l2

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import mass_adaptive_causal_b200 as mala  # noqa: E402


def test_varlen_without_skipping_keeps_every_tile():
    lens = [(180, 180), (27, 27), (400, 1000), (1, 129), (300, 940)]  # (new queries, all keys)
    H, Hkv = 4, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    q = rand(sum(a for a, _ in lens), H, 128) * 3  # far-apart scores: a threshold would skip
    k, v = (rand(sum(b for _, b in lens), Hkv, 128) for _ in range(2))
    cq, ck = (np.cumsum([0] + [x[i] for x in lens]) for i in range(2))
    dev = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    mq, mk = max(a for a, _ in lens), max(b for _, b in lens)
    O, LSE, kept, bits = mala.mala_fwd_varlen(q, k, v, dev(cq), dev(ck), mq, mk, tau=0.0, trace=True)
    mala.mala_check()
    for b, (lq, lk) in enumerate(lens):
        koff = -(-(lk - lq) // 128)
        nbq = -(-lq // 128)
        assert kept[b, :, :nbq].tolist() == [[koff + i + 1 for i in range(nbq)]] * H
        for h in range(H):
            ref = oracle.fwd_chunk(as_f64(q[cq[b]:cq[b + 1], h]), as_f64(k[ck[b]:ck[b + 1], h // 2]),
                                   as_f64(v[ck[b]:ck[b + 1], h // 2]), tile=128, tau=0.0)
            assert rel_l2(as_f64(O[cq[b]:cq[b + 1], h]), ref["O"]) <= TOL["bf16"]["O"]
            assert rel_l2(as_f64(LSE[h, cq[b]:cq[b + 1]]), ref["LSE"]) <= TOL["bf16"]["LSE"]


def test_varlen_without_skipping_shows_a_tile_of_nan_keys():
    """A tile whose keys are all NaN (a page that is not there, read back from a cache) is kept
    like any other: it shows in the rows and heads that see it, and every older tile counts."""
    lens = [(200, 700), (90, 90), (1, 400)]
    H, Hkv = 4, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    q = rand(sum(a for a, _ in lens), H, 128)
    k, v = (rand(sum(b for _, b in lens), Hkv, 128) for _ in range(2))
    cq, ck = (np.cumsum([0] + [x[i] for x in lens]) for i in range(2))
    dev = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (dev(cq), dev(ck), max(a for a, _ in lens), max(b for _, b in lens))
    clean, _ = mala.mala_fwd_varlen(q, k, v, *args, tau=0.0)
    off = 500  # of sequence 0; its key tiles are aligned to its query blocks
    koff = -(-off // 128)
    lo = off + 128 * (2 - koff)
    k[ck[0] + lo: ck[0] + lo + 128, 1] = float("nan")
    O, LSE, kept, bits = mala.mala_fwd_varlen(q, k, v, *args, tau=0.0, trace=True)
    mala.mala_check()
    assert torch.isnan(O[:200, 2:]).all() and torch.isnan(LSE[2:, :200]).all()
    assert torch.equal(O[:200, :2], clean[:200, :2]) and torch.equal(O[200:], clean[200:])
    assert kept[0, :, :2].tolist() == [[koff + 1, koff + 2]] * H


@pytest.mark.parametrize("G", [1, 3])
def test_varlen_without_skipping_over_many_lengths(G):
    """Caches that end anywhere in a tile, odd and even numbers of query blocks, single tokens;
    outputs against the oracle, and a sequence alone against the packed call bit for bit."""
    lens = [(1, 1), (128, 128), (129, 300), (257, 257), (1, 2049), (2, 128), (385, 1153), (0, 70),
            (640, 641), (127, 2000)]
    Hkv = 2
    H = G * Hkv
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    q = rand(sum(a for a, _ in lens), H, 128)
    k, v = (rand(sum(b for _, b in lens), Hkv, 128) for _ in range(2))
    cq, ck = (np.cumsum([0] + [x[i] for x in lens]) for i in range(2))
    dev = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    mq, mk = max(a for a, _ in lens), max(b for _, b in lens)
    O, LSE = mala.mala_fwd_varlen(q, k, v, dev(cq), dev(ck), mq, mk, tau=0.0)
    mala.mala_check()
    for b, (lq, lk) in enumerate(lens):
        if not lq:
            continue
        qs, ks = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        o, lse = mala.mala_fwd_varlen(q[qs].contiguous(), k[ks].contiguous(), v[ks].contiguous(),
                                      dev([0, lq]), dev([0, lk]), lq, lk, tau=0.0)
        assert torch.equal(o, O[qs]) and torch.equal(lse, LSE[:, qs])
        for h in range(H):
            ref = oracle.fwd_chunk(as_f64(q[qs, h]), as_f64(k[ks, h // G]), as_f64(v[ks, h // G]),
                                   tile=128, tau=0.0)
            assert rel_l2(as_f64(O[qs, h]), ref["O"]) <= TOL["bf16"]["O"]
            assert rel_l2(as_f64(LSE[h, qs]), ref["LSE"]) <= TOL["bf16"]["LSE"]
    mala.mala_check()
