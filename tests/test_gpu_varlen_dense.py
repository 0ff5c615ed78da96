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
