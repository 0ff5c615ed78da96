"""The paged 8-bit cache on the GPU: append, decode and gather against float64
(tests/paged_ref.py, and the oracle for the decode rule), at the sizes, masks, strides
and contents where they can go wrong, and used together. The bounds are derived in
tests/paged_ref.py."""

from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
from tests import paged_ref as R
from tests.parity import as_f64, compare_decode_keep, rel_l2

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import mass_adaptive_causal_b200 as mala  # noqa: E402

f8, bf16, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.int32
LAYOUTS = ["plain", "token_major", "interleaved_kv"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def new_pool(n, Hkv, page, layout="plain"):
    """k, v pages full of NaN bytes (as memory that nothing has written may be), scales NaN."""
    u8 = dict(dtype=torch.uint8, device="cuda")
    if layout == "plain":
        k, v = (torch.full((n, Hkv, page, 128), 0x7f, **u8) for _ in range(2))
    elif layout == "token_major":
        k, v = (torch.full((n, page, Hkv, 128), 0x7f, **u8).transpose(1, 2) for _ in range(2))
    else:
        both = torch.full((n, 2, Hkv, page, 128), 0xff, **u8)
        k, v = both[:, 0], both[:, 1]
    s = torch.full((2, n, Hkv), float("nan"), device="cuda")
    return k.view(f8), v.view(f8), s[0].contiguous(), s[1].contiguous()


def table_for(lens, page, n_pages, g, spare=2):
    """Pages from all over the pool; entries past a sequence's last page are no pages."""
    width = max(-(-n // page) for n in lens) + spare
    order = torch.randperm(n_pages, device="cuda", generator=g).int()
    t = torch.empty((len(lens), width + 3), dtype=i32, device="cuda")[:, :width]
    t[:, 0::2], t[:, 1::2] = -7, 1 << 30
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        t[b, :m] = order[at:at + m]
        at += m
    return t


def pages_needed(lens, page):
    return sum(-(-n // page) for n in lens)


def filled(lens, Hkv, page, layout, seed, peak=True, pow2=True):
    """A cache with content for sequences of these lengths; rows behind a sequence stay NaN."""
    g = gen(seed)
    n_pages = pages_needed(lens, page) + 3
    k, v, ks, vs = new_pool(n_pages, Hkv, page, layout)
    t = table_for(lens, page, n_pages, g)
    for b, n in enumerate(lens):
        for s in range(-(-n // page)):
            pid, rows = int(t[b, s]), min(page, n - s * page)
            x = torch.randn((2, Hkv, rows, 128), device="cuda", generator=g).clamp(-4, 4) * 100
            k.view(torch.uint8)[pid, :, :rows] = x[0].to(f8).view(torch.uint8)
            v.view(torch.uint8)[pid, :, :rows] = x[1].to(f8).view(torch.uint8)
        ids = t[b, :-(-n // page)].long()
        e = torch.randint(-9, -4, (2, len(ids), Hkv), device="cuda", generator=g)
        if peak:  # a few pages with much larger or smaller values
            e += 6 * (torch.rand(e.shape, device="cuda", generator=g) < 0.1).long()
        sc = torch.exp2(e.float())
        if not pow2:
            sc *= 1 + torch.rand(e.shape, device="cuda", generator=g)
        ks[ids], vs[ids] = sc[0], sc[1] * 8
    return k, v, ks, vs, t


def check_decode(tensors, lens, q, o, tau, per_head, kept=None, bits=None, skip=()):
    k, v, ks, vs, t = tensors
    Hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    qn, on = as_f64(q), as_f64(o)
    compared = 0
    for b, n in enumerate(lens):
        if b in skip:
            continue
        if n <= 0:
            assert (on[b] == 0).all() and (kept is None or int(kept[b].abs().sum()) == 0)
            assert bits is None or int(bits[b].abs().sum()) == 0
            continue
        K, V, coarse = R._sequence((k, v, ks, vs), t, b, n)
        ref = oracle.decode(qn[b], K, V, tau=tau, per_head=per_head, want_margin=True)
        nt = oracle.n_blocks(n, 128)
        for h in range(q.shape[1]):
            unit = h if per_head else h // G
            if bits is not None:
                gk = mala.unpack_bits(bits[b], 32 * bits.shape[2])[unit]
                assert not gk[nt:].any()
                if compare_decode_keep(gk[:nt], ref["keep"][unit], ref["margin"][unit]):
                    continue
                assert int(kept[b, unit]) == int(ref["keep"][unit].sum())
            keys = np.repeat(ref["keep"][unit].astype(bool), 128)[:n]
            tol = R.decode_bound(qn[b, h], K[h // G], V[h // G], ref["o"][h], keys, coarse[h // G])
            assert (np.abs(on[b, h] - ref["o"][h]) <= tol).all(), (b, h, n)
            compared += 1
    return compared


# ---------------------------------------------------------------------------- decode
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_decode_lengths_and_layouts(page, layout):
    lens = [1, 0, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1000, 2049]
    Hkv, G = 2, 4
    tensors = filled(lens, Hkv, page, layout, 100 + page)
    q = (torch.randn((len(lens), Hkv * G, 128), device="cuda", generator=gen(1)) * 0.5).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    for tau in (1.0, 0.0):
        o, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=tau, trace=True)
        mala.mala_check()
        assert check_decode(tensors, lens, q, o, tau, False, kept, bits) >= 0.9 * 18 * Hkv * G


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("per_head", [False, True])
def test_decode_groups(G, per_head):
    lens = [700, 129, 3000]
    Hkv = 3
    tensors = filled(lens, Hkv, 32, "plain", 200 + G, pow2=False)
    q = torch.randn((3, Hkv * G, 128), device="cuda", generator=gen(G)).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    for tau in (1.0, 0.05):
        o, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=tau, per_head=per_head, trace=True)
        mala.mala_check()
        assert check_decode(tensors, lens, q, o, tau, per_head, kept, bits) >= 0.9 * 9 * G


@pytest.mark.parametrize("B,Hkv,n,tau", [(1, 1, 40000, 1.0), (1, 8, 9000, 1.0), (2, 1, 70001, 0.0),
                                          (40, 2, 3000, 1.0), (3, 2, 20000, 1e-4)])
def test_decode_long_and_many(B, Hkv, n, tau):
    """Few and many groups, long contexts: however the work is split. Keys of the sequence's
    own query stand out, so that tiles are kept here and there."""
    g = gen(n)
    lens = [n - 37 * i for i in range(B)]
    page = 64
    tensors = filled(lens, Hkv, page, "plain", n, peak=False)
    k, v, ks, vs, t = tensors
    G = 4
    q = (torch.randn((B, Hkv * G, 128), device="cuda", generator=g) * 0.4).to(bf16)
    for b, m in enumerate(lens):
        for pos in torch.randint(0, m, (9,), generator=g, device="cuda").tolist():
            pid = int(t[b, pos // page])
            x = q[b].float().view(Hkv, G, 128)[:, pos % G]
            k.view(torch.uint8)[pid, :, pos % page] = (x * 400).clamp(-448, 448).to(f8).view(torch.uint8)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    o, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=tau, trace=True)
    mala.mala_check()
    pick = sorted(set([0, B // 2, B - 1]))
    for b in pick:
        assert check_decode((k, v, ks, vs, t[b:b + 1]), [lens[b]], q[b:b + 1], o[b:b + 1], tau,
                            False, kept[b:b + 1], bits[b:b + 1]) >= 0.7 * Hkv * G


def test_decode_max_seqlen_bounds_and_odd_values():
    """Looser and exact bounds of the length give the same answer; explicit scale; q = 0; one key
    that takes all the mass; scores far apart; a large q."""
    lens = [300, 300, 300, 300, 1]
    tensors = filled(lens, 2, 16, "plain", 7)
    k = tensors[0]
    q = torch.randn((5, 6, 128), device="cuda", generator=gen(3))
    q[0] = 0
    q[1] *= 1e4
    q[2] *= 1e-30
    q = q.to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    a = mala.mala_decode_paged(q, cache, sl, tau=1.0)
    b = mala.mala_decode_paged(q, cache, sl, tau=1.0, max_seqlen=300)
    out = torch.empty_like(q)
    assert mala.mala_decode_paged(q, cache, sl, tau=1.0, max_seqlen=100000, out=out) is out
    c = mala.mala_decode_paged(q, cache, sl, tau=1.0, scale=1 / math.sqrt(128))
    mala.mala_check()
    assert torch.equal(out, a) or rel_l2(as_f64(out), as_f64(a)) < 2e-3
    assert rel_l2(as_f64(b), as_f64(a)) < 2e-3 and torch.equal(c, a)
    check_decode(tensors, lens, q, a, 1.0, False, skip=(1,))
    # q = 1e4 * N(0, 1): one key has all the mass, to within exp(-100)
    K, V = R.sequence(tensors[:4], tensors[4], 1, 300)
    qn, on = as_f64(q), as_f64(a)
    for h in range(6):
        s = K[h // 3] @ qn[1, h] / math.sqrt(128)
        top = np.sort(s)[-2:]
        if top[1] - top[0] > 100:
            assert (np.abs(on[1, h] - V[h // 3][s.argmax()]) <= 2.0 ** -8 * np.abs(on[1, h])).all()


def test_decode_nan_stays_in_its_head_and_shows():
    lens = [400, 400]
    tensors = filled(lens, 2, 64, "plain", 11)
    k, v, ks, vs, t = tensors
    q = (torch.randn((2, 4, 128), device="cuda", generator=gen(5)) * 0.3).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    clean = mala.mala_decode_paged(q, cache, sl, tau=0.25)
    k.view(torch.uint8)[int(t[0, 1]), 1, 3, 100] = 0x7f  # an old key of sequence 0, head 1
    for tau in (0.25, 0.0):
        o = mala.mala_decode_paged(q, cache, sl, tau=tau)
        mala.mala_check()
        assert torch.isnan(o[0, 2:]).all()
        assert not torch.isnan(o[0, :2]).any() and not torch.isnan(o[1]).any()
        if tau:
            assert torch.equal(o[0, :2], clean[0, :2]) and torch.equal(o[1], clean[1])


def test_decode_pages_outside_the_pool_and_lengths_beyond_the_bound():
    lens = [300, 200, 260, 0]
    tensors = filled(lens, 2, 32, "plain", 13)
    t = tensors[4]
    q = torch.randn((4, 4, 128), device="cuda", generator=gen(6)).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    good = mala.mala_decode_paged(q, cache, sl, tau=0.0)
    mala.mala_check()
    saved = int(t[0, 4])
    for bad in (-1, tensors[0].shape[0], 2 ** 31 - 1):
        t[0, 4] = bad
        for tau in (0.0, 1.0):
            o = mala.mala_decode_paged(q, cache, sl, tau=tau)
            with pytest.raises(mala.MalaError, match="MALA_ERR_BAD_PAGE"):
                mala.mala_check()
            assert torch.isnan(o[0]).all() and not torch.isnan(o[1:]).any()
            if tau == 0.0:
                assert torch.equal(o[1:], good[1:])
    t[0, 4] = saved
    o = mala.mala_decode_paged(q, cache, sl, tau=0.0, max_seqlen=256)  # lengths 300 and 260
    with pytest.raises(mala.MalaError, match="MALA_ERR_BAD_PAGE"):
        mala.mala_check()
    assert torch.isnan(o[0]).all() and torch.isnan(o[2]).all()
    assert not torch.isnan(o[1]).any() and (o[3] == 0).all()
    sl[1] = 10 ** 9  # far beyond the table
    o = mala.mala_decode_paged(q, cache, sl, tau=0.0)
    with pytest.raises(mala.MalaError, match="MALA_ERR_BAD_PAGE"):
        mala.mala_check()
    assert torch.isnan(o[1]).all() and torch.equal(o[0], good[0])
    mala.mala_check()  # reported once
    sl[1] = -5
    assert (mala.mala_decode_paged(q, cache, sl, tau=0.0)[1] == 0).all()
    mala.mala_check()


def test_decode_pages_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes, its last and first pages in one sequence."""
    Hkv, page = 8, 128
    n_pages = (2 ** 32) // (Hkv * page * 128) + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    k = torch.empty((n_pages, Hkv, page, 128), dtype=torch.uint8, device="cuda").view(f8)
    v = torch.empty((n_pages, Hkv, page, 128), dtype=torch.uint8, device="cuda").view(f8)
    ks, vs = (torch.ones((n_pages, Hkv), device="cuda") for _ in range(2))
    t = torch.tensor([[n_pages - 1, 0, n_pages - 2, n_pages // 2 + 3]], dtype=i32, device="cuda")
    n, H = 4 * page, 2 * Hkv
    g = gen(17)
    x = torch.randn((n, 2 * Hkv + H, 128), device="cuda", generator=g).to(bf16)
    lens = torch.tensor([n], dtype=i32, device="cuda")
    cache = mala.PagedCache(k, v, ks, vs, t)
    cu = torch.tensor([0, n], dtype=i32, device="cuda")
    mala.mala_cache_append(cache, x[:, :Hkv], x[:, Hkv:2 * Hkv], lens, cu_seqlens=cu)
    K, V = mala.mala_cache_gather(cache, cu, n, n)
    q = x[-1:, 2 * Hkv:].contiguous()
    o = mala.mala_decode_paged(q, cache, lens, tau=0.0)
    mala.mala_check()
    small = t[0].long()
    ref = R.RefCache(*(torch.zeros((4, Hkv, page, 128), dtype=torch.uint8),) * 2,
                     *(torch.ones(4, Hkv),) * 2, torch.arange(4)[None])
    ref.append(x[:, :Hkv], x[:, Hkv:2 * Hkv], [n], [0, n])
    ref.check(k.view(torch.uint8)[small], v.view(torch.uint8)[small], ks[small], vs[small])
    kv = [(ref.val[w] * ref.scale[w][:, :, None, None]).transpose(1, 0, 2, 3).reshape(Hkv, -1, 128)
          for w in range(2)]
    assert np.array_equal(as_f64(K), kv[0].transpose(1, 0, 2))
    assert np.array_equal(as_f64(V), kv[1].transpose(1, 0, 2))
    r = oracle.decode(as_f64(q)[0], kv[0], kv[1], tau=0.0)
    for h in range(H):
        tol = R.decode_bound(as_f64(q)[0, h], kv[0][h // 2], kv[1][h // 2], r["o"][h],
                             np.ones(n, bool))
        assert (np.abs(as_f64(o)[0, h] - r["o"][h]) <= tol).all()


@pytest.mark.parametrize("per_head", [False, True])
def test_decode_statistics_in_several_stretches(per_head):
    """A cache long enough that the rule is replayed in stretches (eight heads: 1280 tiles at a
    time), with keys of the sequence's queries here and there."""
    n, page, G = 200_003, 128, 8
    tensors = filled([n], 1, page, "plain", 71, peak=False)
    k, _, _, _, t = tensors
    g = gen(72)
    q = (torch.randn((1, G, 128), device="cuda", generator=g) * 0.4).to(bf16)
    for i, pos in enumerate(torch.randint(0, n, (24,), generator=g, device="cuda").tolist()):
        x = q[0, i % G].float()
        k.view(torch.uint8)[int(t[0, pos // page]), 0, pos % page] = \
            (x * 400).clamp(-448, 448).to(f8).view(torch.uint8)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor([n], dtype=i32, device="cuda")
    o, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=0.5, per_head=per_head, trace=True)
    mala.mala_check()
    assert int(kept.min()) > 1
    assert check_decode(tensors, [n], q, o, 0.5, per_head, kept, bits) >= 0.7 * G


def test_decode_a_length_above_the_bound_within_its_tile():
    lens = [300, 299, 300]
    tensors = filled(lens, 1, 32, "plain", 73)
    q = torch.randn((3, 2, 128), device="cuda", generator=gen(74)).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    for tau in (1.0, 0.0):
        o = mala.mala_decode_paged(q, cache, sl, tau=tau, max_seqlen=299)
        with pytest.raises(mala.MalaError, match="MALA_ERR_BAD_PAGE"):
            mala.mala_check()
        assert torch.isnan(o[0]).all() and torch.isnan(o[2]).all() and not torch.isnan(o[1]).any()


def test_decode_a_nan_value_shows_only_in_heads_that_keep_its_tile():
    """per_head: a value that is NaN in a tile that one head keeps and the others skip."""
    n, page = 1000, 64
    tensors = list(filled([n], 1, page, "plain", 75, peak=False))
    k, v, ks, vs, t = tensors
    q = (torch.randn((1, 4, 128), device="cuda", generator=gen(76)) * 0.3).to(bf16)
    ks[:] = 2.0 ** -6
    u8 = k.view(torch.uint8)
    pid = int(t[0, 1])
    u8[pid, 0, 5] = (q[0, 2].float() * 1500).clamp(-448, 448).to(f8).view(torch.uint8)  # tile 0, head 2
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor([n], dtype=i32, device="cuda")
    clean, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=900.0, per_head=True, trace=True)
    keeps = [bool(int(bits[0, h, 0]) & 1) for h in range(4)]
    assert keeps[2] and not all(keeps)
    v.view(torch.uint8)[pid, 0, 9, 17] = 0x7f
    o = mala.mala_decode_paged(q, cache, sl, tau=900.0, per_head=True)
    mala.mala_check()
    for h in range(4):
        assert bool(torch.isnan(o[0, h, 17])) == keeps[h]
        rest = [i for i in range(128) if i != 17]
        assert torch.equal(o[0, h, rest], clean[0, h, rest])


def rule_with_nan(qn, K, tau, per_head):
    """The rule read literally, in float64: a tile is skipped only where every head's test says
    so, and a NaN says nothing of the kind. keep and the tests' margin, [units, nt]"""
    Hq, Hkv = qn.shape[0], K.shape[0]
    G, n = Hq // Hkv, K.shape[1]
    nt = -(-n // 128)
    units = Hq if per_head else Hkv
    keep, margin = np.zeros((units, nt), bool), np.full((units, nt), np.inf)
    thr = math.log(tau) - math.log(n)
    for u in range(units):
        heads = [u] if per_head else list(range(u * G, (u + 1) * G))
        scores = K[heads[0] // G] @ qn[heads].T / math.sqrt(128)
        lse = np.full(len(heads), -np.inf)
        for t in range(nt - 1, -1, -1):
            s = scores[t * 128:(t + 1) * 128]
            m = s.max(0)
            if t < nt - 1:
                margin[u, t] = (m - lse - thr).max()
                if (m - lse < thr).all():
                    continue
            keep[u, t] = True
            lse = np.log(np.exp(lse - m) + np.exp(s - m).sum(0)) + m
    return keep, margin


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("nt,Hkv,G,at", [(160, 2, 4, 3), (160, 2, 4, 40), (160, 2, 4, 70),
                                         (160, 2, 4, 150), (1563, 2, 8, 100), (1563, 2, 8, 1500)])
def test_decode_a_nan_score_ends_the_skipping(nt, Hkv, G, at, per_head):
    """One NaN in a tile in the middle of a head's keys: that tile and all older ones are kept,
    wherever it stands among the words and stretches that the rule is replayed in."""
    n, page = 128 * nt - 5, 64
    tensors = filled([n], Hkv, page, "plain", 90 + at, peak=False)
    k, _, _, _, t = tensors
    q = (torch.randn((1, Hkv * G, 128), device="cuda", generator=gen(91)) * 0.3).to(bf16)
    pos = (nt - 1 - at) * 128 + 50
    k.view(torch.uint8)[int(t[0, pos // page]), 1, pos % page, 7] = 0x7f
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor([n], dtype=i32, device="cuda")
    o, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=300.0, per_head=per_head, trace=True)
    mala.mala_check()
    K, _ = R.sequence(tensors[:4], t, 0, n)
    want, margin = rule_with_nan(as_f64(q)[0], K, 300.0, per_head)
    got = mala.unpack_bits(bits[0], 32 * bits.shape[2])[:, :nt].astype(bool)
    assert want[0].mean() < 0.9
    compared = 0
    for u in range(want.shape[0]):
        assert int(kept[0, u]) == got[u].sum()
        if u >= want.shape[0] // 2:
            assert got[u, :nt - at].all()
        compared += not compare_decode_keep(got[u], want[u], margin[u])
    assert compared >= 0.7 * want.shape[0]
    assert not torch.isnan(o[0, :G]).any() and torch.isnan(o[0, G:]).all()


def test_decode_queries_that_are_not_finite_and_of_all_sizes():
    lens = [500]
    tensors = filled(lens, 1, 16, "plain", 77, peak=False)
    q = torch.randn((1, 8, 128), device="cuda", generator=gen(78))
    q[0, 1, 3] = float("inf")
    q[0, 3, 100] = float("nan")
    q[0, 4] = q[0, 4] * 2.0 ** -120
    q[0, 5, 1:] *= 2.0 ** -18  # one value far above the rest
    q[0, 6] = 0
    q = q.to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    o = mala.mala_decode_paged(q, cache, sl, tau=0.0)
    mala.mala_check()
    assert torch.isnan(o[0, [1, 3]]).all()
    K, V, coarse = R._sequence(tensors[:4], tensors[4], 0, 500)
    qn, on = as_f64(q), as_f64(o)
    for h in (0, 2, 4, 5, 6, 7):
        ref = oracle.decode(qn[0, h:h + 1], K, V, tau=0.0)["o"][0]
        tol = R.decode_bound(qn[0, h], K[0], V[0], ref, np.ones(500, bool), coarse[0])
        assert (np.abs(on[0, h] - ref) <= tol).all(), h


@pytest.mark.parametrize("tau", [0.0, 1.0])
@pytest.mark.parametrize("G", [4, 7])
def test_decode_probabilities_hold_sixteen_bits(G, tau):
    """Keys in pairs whose values cancel: an output is the difference of two probabilities near
    each other, far below their sum, so that its own rounding hides nothing of theirs.

    The bound of tests/paged_ref.py with 2^-16 in the place of 2^-11: a probability p in [2^e,
    2^(e+1)) goes in as four e4m3 terms; the first leaves at most half its step, 2^(e-4), which goes
    on rounded to f16, by at most 2^(e-16); the other three hold those eleven bits (four
    and a sign each), down to 2^-30 of the row's largest. Scores of about 2^-8, so that their own
    part of the bound, 4 * 129 * 2^-23 A, is below 2^-16."""
    B, Hkv, page, n = 64, 2, 16, 2
    g = gen(88)
    k, v, ks, vs = new_pool(B, Hkv, page)
    x = torch.randn((B, Hkv, 2, 128), device="cuda", generator=g).clamp(-4, 4)
    y = torch.randn((B, Hkv, 1, 128), device="cuda", generator=g).clamp(-4, 4)
    k.view(torch.uint8)[:, :, :2] = (100 * x).to(f8).view(torch.uint8)
    v.view(torch.uint8)[:, :, :2] = (100 * torch.cat([y, -y], 2)).to(f8).view(torch.uint8)
    ks[:], vs[:] = 2.0 ** -7, 2.0 ** -7
    t = torch.arange(B, dtype=i32, device="cuda")[:, None]
    q = (torch.randn((B, Hkv * G, 128), device="cuda", generator=g) * 0.004).to(bf16)
    cache = mala.PagedCache(k, v, ks, vs, t)
    o = mala.mala_decode_paged(q, cache, torch.full((B,), n, dtype=i32, device="cuda"), tau=tau)
    mala.mala_check()
    qn, on = as_f64(q), as_f64(o)
    for b in range(B):
        K, V = R.sequence((k, v, ks, vs), t, b, n)
        for h in range(Hkv * G):
            kk, vv = K[h // G], V[h // G]
            s = kk @ qn[b, h] / math.sqrt(128)
            p = np.exp(s - s.max())
            p /= p.sum()
            ref, S = p @ vv, p @ np.abs(vv)
            A = (np.abs(kk) @ np.abs(qn[b, h])).max() / math.sqrt(128)
            rest = 2.0 ** -29 * np.abs(qn[b, h]).max() * np.abs(kk).sum(-1).max() / math.sqrt(128)
            tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -30 * p.max() * np.abs(vv).sum(0) \
                + S * (2.0 ** -16 + 4 * (129 * 2.0 ** -23 * A + rest) + 2.0 ** -20)
            assert (np.abs(on[b, h] - ref) <= tol).all(), (b, h)


@pytest.mark.parametrize("page", [16, 64])
def test_decode_pages_of_very_different_scales(page):
    lens = [700, 130]
    tensors = filled(lens, 2, page, "plain", 79, peak=False)
    vs = tensors[3]
    vs *= torch.exp2(torch.randint(-12, 13, vs.shape, device="cuda", generator=gen(80)).float())
    vs[int(tensors[4][0, 1])] = 0.0
    q = torch.randn((2, 6, 128), device="cuda", generator=gen(81)).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    for tau in (1.0, 0.0):
        o, kept, bits = mala.mala_decode_paged(q, cache, sl, tau=tau, trace=True)
        mala.mala_check()
        assert check_decode(tensors, lens, q, o, tau, False, kept, bits) >= 0.9 * 12


def test_decode_beside_a_prefill_on_another_stream():
    """Both kernels want tensor memory; whichever an SM runs first, both end."""
    g = gen(82)
    lens = [2000] * 8
    tensors = filled(lens, 4, 64, "plain", 83)
    q = torch.randn((8, 16, 128), device="cuda", generator=g).to(bf16)
    cache = mala.PagedCache(*tensors)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    Q, K, V = (torch.randn((1, 8, 4096, 128), device="cuda", generator=g).to(bf16) for _ in range(3))
    want = mala.mala_decode_paged(q, cache, sl, tau=1.0)
    O, _ = mala.mala_fwd(Q, K, V, tau=1.0)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    outs, fwd = [], []
    for _ in range(5):
        with torch.cuda.stream(other):
            fwd.append(mala.mala_fwd(Q, K, V, tau=1.0)[0])
        outs.append(mala.mala_decode_paged(q, cache, sl, tau=1.0))
    torch.cuda.synchronize()
    mala.mala_check()
    assert all(torch.equal(x, want) for x in outs) and all(torch.equal(x, O) for x in fwd)


@pytest.mark.parametrize("B,G", [(148, 4), (8, 4), (148, 8)])
def test_decode_blocks_that_skip_tiles_whose_values_they_loaded(B, G):
    """Short caches under a threshold that skips most tiles: a block has asked for the values of
    all its tiles, and may only end when they are there. Values far from the L2 and a copy that
    takes the memory's rate make them late; the next blocks use the same shared memory at once."""
    g = gen(86)
    Hkv, page, rows = 4, 64, 16
    lens = [65 + 13 * (b % 40) for b in range(B)]  # up to 5 tiles: one or two to a block
    base = filled(lens[:40], Hkv, page, "plain", 87, peak=False)
    n_pages = base[0].shape[0]
    # the values of `rows` copies of the pool, each used once, and keys that stay in the L2
    big = [x.view(torch.uint8).repeat(rows, 1, 1, 1).view(f8) for x in base[:2]]
    scales = [x.repeat(rows, 1) for x in base[2:4]]
    q = (torch.randn((B, Hkv * G, 128), device="cuda", generator=g) * 0.2).to(bf16)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    t40 = base[4].clamp(0, n_pages - 1)
    tables = [(t40 + r * n_pages).repeat(4, 1)[:B].contiguous() for r in range(rows)]
    caches = [mala.PagedCache(*big, *scales, t) for t in tables]
    want, kept, _ = mala.mala_decode_paged(q, caches[0], sl, tau=1e4, max_seqlen=640, trace=True)
    torch.cuda.synchronize()
    tiles = Hkv * sum(-(-n // 128) for n in lens)
    assert int(kept.sum()) < 0.75 * tiles  # most of the older tiles are skipped
    noise = torch.empty((2, 1 << 28), dtype=torch.uint8, device="cuda")
    other = torch.cuda.Stream()
    outs = []
    for cache in caches:
        with torch.cuda.stream(other):
            noise[1].copy_(noise[0])
        for _ in range(4):  # blocks of one call follow those of the one before
            outs.append(mala.mala_decode_paged(q, cache, sl, tau=1e4, max_seqlen=640))
    torch.cuda.synchronize()
    mala.mala_check()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("per_head", [False, True])
def test_decode_bounds_of_millions_of_tokens(per_head):
    """Short sequences under a table that could hold millions of tokens: the statistics' room
    follows the bound; beyond it the call is refused, but for exact attention."""
    lens, page = [700, 129], 128
    k, v, ks, vs, t = filled(lens, 2, page, "plain", 84)
    wide = torch.full((2, 40000), -1, dtype=i32, device="cuda")
    wide[:, :t.shape[1]] = t
    q = torch.randn((2, 16, 128), device="cuda", generator=gen(85)).to(bf16)
    sl = torch.tensor(lens, dtype=i32, device="cuda")
    small = mala.PagedCache(k, v, ks, vs, t)
    large = mala.PagedCache(k, v, ks, vs, wide)
    want = mala.mala_decode_paged(q, small, sl, tau=1.0, per_head=per_head, max_seqlen=700)
    for bound in (100_000, 1_000_000, 3_000_000):
        o, kept, bits = mala.mala_decode_paged(q, large, sl, tau=1.0, per_head=per_head,
                                               max_seqlen=bound, trace=True)
        mala.mala_check()
        assert check_decode((k, v, ks, vs, t), lens, q, o, 1.0, per_head, kept, bits) >= 0.9 * 32
        assert rel_l2(as_f64(o), as_f64(want)) < 2e-3
    with pytest.raises(mala.MalaError, match="TOO_LARGE"):
        mala.mala_decode_paged(q, large, sl, tau=1.0, per_head=per_head)  # 5.1 million tokens
    o = mala.mala_decode_paged(q, large, sl, tau=0.0, per_head=per_head)
    mala.mala_check()
    assert check_decode((k, v, ks, vs, t), lens, q, o, 0.0, per_head) == 32


# ---------------------------------------------------------------------------- append
def projection(T, Hq, Hkv, g, size=1.0):
    x = torch.randn((T, Hq + 2 * Hkv, 128), device="cuda", generator=g) * size
    x *= torch.where(torch.rand((Hq + 2 * Hkv, 128), device="cuda", generator=g) < 0.05, 8.0, 1.0)
    x = x.to(bf16)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def check_q(q_out, want, tol):
    got = as_f64(q_out)
    rows = ~np.isnan(want)
    assert (np.abs(got - want)[rows] <= (2.0 ** -8 * np.abs(want) + tol * (1 + 2.0 ** -8))[rows]).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, False), (96, True), (0, False)])
def test_append_prompts_chunks_and_steps(page, layout, rot, inter):
    """Three calls on one cache: prompts of many lengths, chunks behind them, single tokens."""
    g = gen(page + rot)
    Hq, Hkv = 6, 2
    first = [1, 2, page - 1, page, page + 1, 3 * page + 5, 300, 0]
    chunk = [5, 0, 2, page, 2 * page - 1, 1, 130, 0]
    final = [a + b + 1 if a + b else 0 for a, b in zip(first, chunk)]
    n_pages = pages_needed(final, page) + 2
    k_pages, v_pages, ks, vs = new_pool(n_pages, Hkv, page, layout)
    t = table_for(final, page, n_pages, g)
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    ref = R.RefCache(k_pages, v_pages, ks, vs, t)
    freq = (1e4 ** (-torch.arange(rot // 2, device="cuda") / (rot // 2 or 1))).float() if rot else None
    lens = [0] * 8
    for step, (news, size) in enumerate(((first, 0.1), (chunk, 1.0), (None, 3.0))):
        if news is None:  # one token each; the last sequence is an unused slot
            lens, cu, T = final, None, 8
        else:
            lens = [a + b for a, b in zip(lens, news)]
            cu = np.concatenate([[0], np.cumsum(news)]).tolist()
            T = cu[-1] + 4  # rows behind the last sequence
        q, k, v = projection(T, Hq, Hkv, g, size)
        sl = torch.tensor(lens, dtype=i32, device="cuda")
        cut = None if cu is None else torch.tensor(cu, dtype=i32, device="cuda")
        q_out = torch.full((T, Hq, 128), 777.0, dtype=bf16, device="cuda")
        mala.mala_cache_append(cache, k, v, sl, cu_seqlens=cut, inv_freq=freq, interleaved=inter,
                               q=q, q_out=q_out, max_new=None if news is None else max(news))
        mala.mala_check()
        want, tol = ref.append(k, v, lens, cu, freq, inter, q)
        ref.check(k_pages, v_pages, ks, vs)
        check_q(q_out, want, tol)
        assert (q_out[torch.tensor(np.isnan(want[:, 0, 0]))] == 777.0).all()


@pytest.mark.parametrize("page,B,total,Hkv,G,rot,inter,in_place", [
    (16, 24, 480, 8, 4, 64, False, True),    # all eight heads to a block, rows of one warp
    (16, 10, 400, 8, 8, 32, True, False),    # 3 + 3 + 2 heads
    (32, 30, 700, 7, 5, 96, False, False),   # seven heads and 35 queries' heads, more than 32
    (64, 40, 1000, 8, 8, 32, False, True),   # two warps to a row group; 64 queries' heads
    (64, 24, 900, 5, 3, 32, True, True),     # 3 + 2 heads
    (128, 50, 1500, 8, 2, 32, False, False),  # four warps
    (128, 28, 1400, 3, 8, 16, True, True),   # 2 + 1 heads
    (128, 50, 1500, 8, 0, 32, True, False),  # no queries
])
def test_append_blocks_of_several_heads(page, B, total, Hkv, G, rot, inter, in_place):
    """Calls whose (page, sequence) blocks would fill the chip, so that a block takes several heads
    one after the other: the next unit's rows come while the last one's are stored, the page's
    maxima go through the same shared memory again, and the last block of a page may have fewer
    heads. A chunk of small tokens, then one of large ones behind it (scales grow in the middle of
    pages), runs of 0 to 2 pages; the bound of the new tokens is that of all sequences together."""
    g = gen(1000 * page + Hkv)
    rng = np.random.default_rng(page + Hkv)
    Hq = G * Hkv
    chunks = []
    for _ in range(2):
        news = rng.choice([0, 1, 5, page - 1, page, page + 3, 2 * page + 1], B)
        while news.sum() > total:
            news[rng.integers(B)] //= 2
        chunks.append(news.tolist())
    final = np.sum(chunks, 0).tolist()
    n_pages = pages_needed(final, page) + 2
    k_pages, v_pages, ks, vs = new_pool(n_pages, Hkv, page, "token_major")
    t = table_for(final, page, n_pages, g)
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    freq = (1e4 ** (-torch.arange(rot // 2, device="cuda") / (rot // 2))).float()
    lens = [0] * B
    for news, size in zip(chunks, (0.05, 2.0)):
        lens = [a + b for a, b in zip(lens, news)]
        cu = np.concatenate([[0], np.cumsum(news)]).tolist()
        q, k, v = projection(total, Hq, Hkv, g, size)
        given = q.clone()
        # from the cache as it lies there: what an earlier chunk left next to a tie may have fallen
        # on either side of it, and is now rounded again from there
        ref = R.RefCache(k_pages, v_pages, ks, vs, t)
        out = None
        if G:
            out = q if in_place else torch.full((total, Hq, 128), 777.0, dtype=bf16, device="cuda")
        mala.mala_cache_append(cache, k, v, torch.tensor(lens, dtype=i32, device="cuda"),
                               cu_seqlens=torch.tensor(cu, dtype=i32, device="cuda"), inv_freq=freq,
                               interleaved=inter, q=q if G else None, q_out=out)
        mala.mala_check()
        want, tol = ref.append(k, v, lens, cu, freq, inter, given if G else None)
        ref.check(k_pages, v_pages, ks, vs)
        if G:
            check_q(out, want, tol)
            rest = torch.tensor(np.isnan(want[:, 0, 0]))
            assert torch.equal(out[rest], given[rest] if in_place else torch.full_like(given[rest], 777))


@pytest.mark.parametrize("B,Hkv,G,rot,inter,in_place", [
    (20, 8, 4, 128, False, True), (20, 8, 8, 64, True, False), (7, 40, 0, 128, True, False),
    (33, 5, 3, 0, False, True), (3, 1, 1, 96, False, False)])
def test_append_up_to_two_tokens_each(B, Hkv, G, rot, inter, in_place):
    """A draft token beside the newest one: none, one or two new tokens, within a page and across
    its end, growing and shrinking, in blocks of some of the heads."""
    g = gen(B + Hkv)
    page, Hq = 16, G * Hkv
    lens = [int(x) for x in np.random.default_rng(B).integers(0, 3 * page, B)]
    lens[0], lens[1], lens[2] = page - 1, page, 0
    n_pages = pages_needed([n + 10 for n in lens], page)
    k_pages, v_pages, ks, vs = new_pool(n_pages, Hkv, page, "interleaved_kv")
    t = table_for([n + 10 for n in lens], page, n_pages, g)
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    freq = (1e4 ** (-torch.arange(rot // 2, device="cuda") / (rot // 2 or 1))).float() if rot else None
    _, k, v = projection(max(sum(lens), 1), 0, Hkv, g)
    mala.mala_cache_append(cache, k, v, torch.tensor(lens, dtype=i32, device="cuda"), inv_freq=freq,
                           cu_seqlens=torch.tensor([0, *np.cumsum(lens)], dtype=i32, device="cuda"),
                           interleaved=inter)
    for step, size in enumerate((0.3, 6.0, 1.0)):
        news = [(b + step) % 3 for b in range(B)]
        lens = [a + b for a, b in zip(lens, news)]
        cu = np.concatenate([[0], np.cumsum(news)]).tolist()
        T = cu[-1]
        q, k, v = projection(T, Hq, Hkv, g, size)
        given = q.clone()
        ref = R.RefCache(k_pages, v_pages, ks, vs, t)
        out = mala.mala_cache_append(cache, k, v, torch.tensor(lens, dtype=i32, device="cuda"),
                                     cu_seqlens=torch.tensor(cu, dtype=i32, device="cuda"), max_new=2,
                                     inv_freq=freq, interleaved=inter, q=q if G else None,
                                     q_out=q if G and in_place else None)
        mala.mala_check()
        want, tol = ref.append(k, v, lens, cu, freq, inter, given if G else None)
        ref.check(k_pages, v_pages, ks, vs)
        if G:
            check_q(out, want, tol)


def test_append_scales_grow_and_hold():
    """Tokens of growing, shrinking, zero, tiny, huge and non-finite values into one page."""
    page = 32
    k_pages, v_pages, ks, vs = new_pool(2, 1, page)
    t = torch.tensor([[1]], dtype=i32, device="cuda")
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    ref = R.RefCache(k_pages, v_pages, ks, vs, t)
    g = gen(3)
    sizes = [0.0, 1e-38, 1e-3, 1.0, 1e3, 1e-2, 1e37, 1.0, 448.0, 0.0]
    for i, size in enumerate(sizes):
        x = (torch.randn((2, 1, 1, 128), device="cuda", generator=g).clamp(-2, 2) * size).to(bf16)
        if i == 5:
            x[0, 0, 0, 3], x[0, 0, 0, 4], x[1, 0, 0, 5] = float("inf"), float("nan"), -float("inf")
        if i == 8:
            x[:] = 448.0  # the largest value of its scale exactly
        n = torch.tensor([i + 1], dtype=i32, device="cuda")
        mala.mala_cache_append(cache, x[0], x[1], n)
        mala.mala_check()
        ref.append(x[0], x[1], [i + 1])
        ref.check(k_pages, v_pages, ks, vs)


def test_append_far_positions():
    """Angles of positions where float32 products have lost them."""
    page, n = 128, 500_000
    width = -(-n // page)
    k_pages, v_pages, ks, vs = new_pool(3, 2, page)
    t = torch.full((1, width), 99, dtype=i32, device="cuda")
    t[0, -3:] = torch.tensor([2, 0, 1], dtype=i32)
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    ref = R.RefCache(k_pages, v_pages, ks, vs, t)
    m = (n - 1) % page + 1 + 150
    q, k, v = projection(m, 4, 2, gen(9))
    freq = (5e5 ** (-torch.arange(64, device="cuda") / 64)).float()
    lens, cu = [n], [0, m]
    q_out = mala.mala_cache_append(cache, k, v, torch.tensor(lens, dtype=i32, device="cuda"),
                                   cu_seqlens=torch.tensor(cu, dtype=i32, device="cuda"),
                                   inv_freq=freq, q=q)
    mala.mala_check()
    want, tol = ref.append(k, v, lens, cu, freq, False, q)
    check_q(q_out, want, tol)
    # the first page's rows before the new tokens were NaN bytes with a NaN scale:
    # they stay NaN, and the page's scale is the new tokens'
    ref.check(k_pages, v_pages, ks, vs)


def test_append_in_place_queries_and_one_row_views():
    g = gen(21)
    k_pages, v_pages, ks, vs = new_pool(4, 1, 16)
    t = torch.tensor([[0, 1], [2, 3]], dtype=i32, device="cuda")
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    q, k, v = projection(2, 3, 1, g)
    freq = torch.rand(64, device="cuda", generator=g)
    sl = torch.tensor([17, 4], dtype=i32, device="cuda")
    ref = R.RefCache(k_pages, v_pages, ks, vs, t)
    want, tol = ref.append(k, v, [17, 4], None, freq, False, q)
    other = mala.mala_cache_append(cache, k, v, sl, inv_freq=freq, q=q)
    same = mala.mala_cache_append(cache, k, v, sl, inv_freq=freq, q=q, q_out=q)
    mala.mala_check()
    assert same is q and torch.equal(other, q)
    check_q(q, want, tol)
    # a page table's second page of sequence 0: rows before position 17 were never written
    assert int(ks.isnan().sum()) == 2


def test_append_what_does_not_fit_is_left_out():
    g = gen(22)
    page = 16
    k_pages, v_pages, ks, vs = new_pool(6, 2, page)
    t = torch.tensor([[0, 1], [2, 55], [3, 4], [5, 5]], dtype=i32, device="cuda")
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    q, k, v = projection(60, 2, 2, g)

    def call(lens, cu, max_new=60):
        ref = R.RefCache(k_pages, v_pages, ks, vs, t)
        mala.mala_cache_append(cache, k, v, torch.tensor(lens, dtype=i32, device="cuda"),
                               cu_seqlens=torch.tensor(cu, dtype=i32, device="cuda"),
                               max_new=max_new)
        ok = True
        try:
            mala.mala_check()
        except mala.MalaError as e:
            assert e.code == 6
            ok = False
        return ref, ok

    ref, ok = call([20, 20, 20, 0], [0, 20, 40, 60, 60])  # sequence 1's second page is no page
    ref.append(k, v, [20, 20, 20, 0], [0, 20, 40, 60, 60])
    assert not ok
    ref.check(k_pages, v_pages, ks, vs)
    ref, ok = call([20, 3, 20, 0], [0, 5, 10, 12, 12])  # sequence 1 has more new tokens than length
    ref.append(k, v, [20, 3, 20, 0], [0, 5, 10, 12, 12])
    assert not ok
    ref.check(k_pages, v_pages, ks, vs)
    ref, ok = call([20, 16, 32, 0], [0, 5, 10, 26, 26], max_new=8)  # sequence 2: 16 > 8
    ref.append(k, v, [20, 16, 32, 0], [0, 5, 10, 26, 26], max_new=8)
    assert not ok
    ref.check(k_pages, v_pages, ks, vs)
    for cu in ([-3, 0, 0, 0, 0], [0, 0, 0, 100, 100], [0, 61, 61, 61, 61]):  # rows that are not there
        ref, ok = call([20, 16, 32, 0], cu)
        assert not ok
        ref.check(k_pages, v_pages, ks, vs)
    ref, ok = call([33, 0, 0, 0], [0, 5, 5, 5, 5])  # past the table: position 32
    ref.append(k, v, [33, 0, 0, 0], [0, 5, 5, 5, 5])
    assert not ok
    ref.check(k_pages, v_pages, ks, vs)
    ref, ok = call([0, -4, 0, 0], [0, 5, 9, 9, 9])  # unused slots: nothing, and nothing to report
    assert ok
    ref.check(k_pages, v_pages, ks, vs)


# ---------------------------------------------------------------------------- gather
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_gather(page, layout):
    lens = [1, 0, page, page - 1, page + 1, 700, 129]
    Hkv = 3
    tensors = filled(lens, Hkv, page, layout, 300 + page)
    cache = mala.PagedCache(*tensors)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1]) + 5
    out = tuple(torch.full((total, Hkv, 128), 55.0, dtype=bf16, device="cuda") for _ in range(2))
    K, V = mala.mala_cache_gather(cache, torch.tensor(cu, dtype=i32, device="cuda"), max(lens),
                                  total, out=out)
    mala.mala_check()
    assert K is out[0] and V is out[1]
    for b, n in enumerate(lens):
        if n:
            for got, want in zip((K, V), R.sequence(tensors[:4], tensors[4], b, n)):
                assert np.array_equal(as_f64(got[cu[b]:cu[b + 1]]), want.transpose(1, 0, 2))
    assert (K[cu[-1]:] == 55.0).all() and (V[cu[-1]:] == 55.0).all()


def test_gather_refusals_on_the_device():
    lens = [40, 20, 50]
    tensors = filled(lens, 2, 16, "plain", 31)
    t = tensors[4]
    cache = mala.PagedCache(*tensors)
    total = 110

    def call(cu, max_seqlen):
        out = tuple(torch.full((total, 2, 128), 55.0, dtype=bf16, device="cuda") for _ in range(2))
        mala.mala_cache_gather(cache, torch.tensor(cu, dtype=i32, device="cuda"), max_seqlen, total,
                               out=out)
        with pytest.raises(mala.MalaError, match="MALA_ERR_BAD_PAGE"):
            mala.mala_check()
        return out

    K, V = call([0, 40, 60, 110], 45)  # the third is longer than the bound
    assert (K[60:] == 55.0).all() and not (K[:60] == 55.0).all(-1).any()
    K, V = call([0, 40, 60, 120], 60)  # rows past the end
    assert (V[60:] == 55.0).all()
    t[1, 1] = -1
    K, V = call([0, 40, 60, 110], 50)
    assert torch.isnan(K[56:60]).all() and torch.isnan(V[56:60]).all()
    assert not torch.isnan(K[:56]).any() and not torch.isnan(K[60:]).any()


# ---------------------------------------------------------------------------- together
def test_serving_run_matches_the_prefill_and_decode_over_a_whole_cache():
    """Prompts in two chunks (append, gather, mala_fwd_varlen), then steps (append, decode):
    decode's keep sets and outputs against mala_decode over the same values as a contiguous
    bf16 cache, the prefill's last row against a decode of the same query."""
    g = gen(41)
    Hq, Hkv, page = 8, 2, 32
    prompts = [300, 45, 1000]
    B, steps = 3, 4
    final = [n + steps for n in prompts]
    n_pages = pages_needed(final, page)
    k_pages, v_pages, ks, vs = new_pool(n_pages, Hkv, page)
    t = table_for(final, page, n_pages, g)
    cache = mala.PagedCache(k_pages, v_pages, ks, vs, t)
    freq = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float()
    done = [0] * B
    for part in (0.6, 1.0):
        news = [round(part * n) - d for n, d in zip(prompts, done)]
        done = [d + m for d, m in zip(done, news)]
        cu = torch.tensor([0, *np.cumsum(news)], dtype=i32, device="cuda")
        cu_k = torch.tensor([0, *np.cumsum(done)], dtype=i32, device="cuda")
        lens = torch.tensor(done, dtype=i32, device="cuda")
        q, k, v = projection(sum(news), Hq, Hkv, g)
        q = mala.mala_cache_append(cache, k, v, lens, cu_seqlens=cu, max_new=max(news),
                                   inv_freq=freq, q=q)
        K, V = mala.mala_cache_gather(cache, cu_k, max(done), sum(done))
        O, LSE = mala.mala_fwd_varlen(q, K, V, cu, cu_k, max(news), max(done), tau=0.0)
        last = (cu[1:] - 1).long()
        o = mala.mala_decode_paged(q[last].contiguous(), cache, lens, tau=0.0)
        mala.mala_check()
        assert rel_l2(as_f64(O[last]), as_f64(o)) <= 4e-3  # both within 2e-3 of the formula
    for _ in range(steps):
        done = [d + 1 for d in done]
        lens += 1
        q, k, v = projection(B, Hq, Hkv, g)
        q = mala.mala_cache_append(cache, k, v, lens, inv_freq=freq, q=q)
        for tau in (1.0, 0.0):
            o, kept, bits = mala.mala_decode_paged(q, cache, lens, tau=tau, trace=True)
            mala.mala_check()
            for b, n in enumerate(done):
                K, V = (torch.tensor(x).to(bf16).cuda()[None].contiguous()
                        for x in R.sequence((k_pages, v_pages, ks, vs), t, b, n))
                o2, kept2, bits2 = mala.mala_decode(q[b:b + 1].contiguous(), K, V, tau=tau, trace=True)
                mala.mala_check()
                assert torch.equal(kept2[0], kept[b])
                assert torch.equal(bits2[0], bits[b, :, :bits2.shape[2]])
                assert rel_l2(as_f64(o[b]), as_f64(o2[0])) <= 4e-3


def test_steps_in_a_graph_and_on_two_streams():
    """A captured step (lengths + 1, append, decode) replayed against eager calls; two captured
    graphs of two caches replayed at once on two streams."""
    def setup(seed):
        g = gen(seed)
        Hq, Hkv, page, lens = 8, 2, 16, [30, 1, 500, 0]
        room = [n + 20 for n in lens]
        n_pages = pages_needed(room, page)
        k, v, ks, vs = new_pool(n_pages, Hkv, page)
        t = table_for(room, page, n_pages, g, spare=0)
        cache = mala.PagedCache(k, v, ks, vs, t)
        T = sum(lens)
        _, kk, vv = projection(T, Hq, Hkv, g)
        sl = torch.tensor(lens, dtype=i32, device="cuda")
        freq = torch.rand(64, device="cuda", generator=g)
        mala.mala_cache_append(cache, kk, vv, sl, cu_seqlens=torch.tensor(
            [0, *np.cumsum(lens)], dtype=i32, device="cuda"), inv_freq=freq)
        x = torch.randn((4, Hq + 2 * Hkv, 128), device="cuda", generator=g).to(bf16)
        used = (sl > 0).int()

        def step():
            sl.add_(used)  # the unused slot stays at 0
            q = mala.mala_cache_append(cache, x[:, 8:10], x[:, 10:], sl, inv_freq=freq, q=x[:, :8])
            return mala.mala_decode_paged(q, cache, sl, tau=1.0)
        return step, x, g, (k, v, ks, vs, sl)

    eager, xe, ge, se = setup(51)
    steps, graphs, outs, states, inputs = [], [], [], [], []
    for _ in range(2):
        step, x, g, st = setup(51)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o = step()
        graphs.append((graph, s))
        steps.append(step)  # keeps the cache and its page table, which the graph reads
        outs.append(o)
        states.append(st)
        inputs.append(x)
    torch.cuda.synchronize()
    for _ in range(12):
        fresh = torch.randn(xe.shape, device="cuda", generator=ge).to(bf16)
        want = None
        xe.copy_(fresh)
        want = eager()
        for x in inputs:
            x.copy_(fresh)
        torch.cuda.synchronize()
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, st in zip(outs, states):
            assert torch.equal(o, want)
            for a, b in zip(st, se):
                if a.dtype == f8:
                    a, b = a.view(torch.uint8), b.view(torch.uint8)
                assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a,
                                   b.nan_to_num(7.0) if b.is_floating_point() else b)
    mala.mala_check()


def test_a_page_shared_by_two_sequences_is_read_by_both():
    lens = [96, 90]
    tensors = list(filled([96], 2, 32, "plain", 61))
    t = tensors[4]
    tensors[4] = torch.stack([t[0], t[0]])[:, :3].contiguous()
    q = torch.randn((1, 4, 128), device="cuda", generator=gen(8)).to(bf16).repeat(2, 1, 1)
    cache = mala.PagedCache(*tensors)
    o = mala.mala_decode_paged(q, cache, torch.tensor(lens, dtype=i32, device="cuda"), tau=0.0)
    mala.mala_check()
    assert check_decode(tensors, lens, q, o, 0.0, False) == 8
