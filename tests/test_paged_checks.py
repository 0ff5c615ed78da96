"""The paged cache's calls without a GPU: what the binding and the C entry points
refuse, on the host, before anything is launched, and what the binding passes on."""

import ctypes

import pytest
import torch

import mass_adaptive_causal_b200 as mala

bf16, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from mass_adaptive_causal_b200 import build
    build.build()
    return mala.lib()


def pool(n=6, Hkv=2, page=16, d=128):
    return torch.zeros((n, Hkv, page, d), dtype=f8)


def make(n=6, Hkv=2, page=16, B=3, width=4, **kw):
    t = dict(k_pages=pool(n, Hkv, page), v_pages=pool(n, Hkv, page),
             k_scale=torch.ones(n, Hkv), v_scale=torch.ones(n, Hkv),
             page_table=torch.zeros((B, width), dtype=i32))
    t.update(kw)
    return mala.PagedCache(**t)


def test_cache_construction():
    c = make()
    assert (c.Hkv, c.page_size, c.max_seqlen, c.sequences) == (2, 16, 64, 3)
    nhd = torch.zeros((6, 16, 2, 128), dtype=f8).transpose(1, 2)      # [page][token][head][d]
    both = torch.zeros((6, 2, 2, 16, 128), dtype=f8)                  # [page][k or v]...
    c = make(k_pages=nhd, v_pages=both[:, 1])
    assert c._struct.k_stride_token == 256 and c._struct.k_stride_head == 128
    assert c._struct.v_stride_page == 2 * 2 * 16 * 128
    wide = torch.zeros((3, 9), dtype=i32)[:, :4]
    assert make(page_table=wide)._struct.table_stride == 9
    for kw, msg in (
            (dict(k_pages=pool().view(torch.uint8)), "float8"),
            (dict(k_pages=pool()[0]), "float8"),
            (dict(v_pages=pool(n=5)), "one shape"),
            (dict(k_pages=pool(page=24), v_pages=pool(page=24)), "page_size"),
            (dict(k_pages=pool(d=64), v_pages=pool(d=64)), "page_size"),
            (dict(k_scale=torch.ones(6, 3)), "shape"),
            (dict(v_scale=torch.ones(6, 2).double()), "must be"),
            (dict(k_scale=torch.ones(2, 6).t()), "contiguous"),
            (dict(page_table=torch.zeros((3, 4), dtype=torch.int64)), "int32"),
            (dict(page_table=torch.zeros((4, 3), dtype=i32).t()), "rows"),
            (dict(page_table=torch.zeros((1, 4), dtype=i32).expand(3, 4)), "overlap"),
            (dict(page_table=torch.zeros((3, 0), dtype=i32)), "empty"),
            (dict(k_pages=torch.zeros((6, 2, 16, 256), dtype=f8)[..., ::2]), "contiguous"),
            (dict(k_pages=pool()[:1].expand(6, 2, 16, 128)), "multiples of 16"),
            (dict(k_pages=torch.zeros(6 * 2 * 16 * 128 + 1, dtype=f8)[1:].view(6, 2, 16, 128)),
             "aligned"),
            (dict(v_pages=pool().to("meta")), "device")):
        with pytest.raises(ValueError, match=msg):
            make(**kw)
    with pytest.raises(AttributeError):
        make().k_pages = pool()


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    ready = mala._paged_ready
    monkeypatch.setattr(mala, "_lib", r)
    monkeypatch.setattr(mala, "_paged_ready", lambda c: ready(c, require_cuda=False))
    monkeypatch.setattr(mala, "_paged_stream", lambda stream, index: None)
    return r


def test_a_cache_off_the_gpu_is_refused():
    c = make()
    with pytest.raises(ValueError, match="CUDA"):
        mala.mala_decode_paged(torch.zeros((3, 4, 128), dtype=bf16), c, torch.zeros(3, dtype=i32))
    with pytest.raises(TypeError, match="PagedCache"):
        mala.mala_cache_gather((1, 2), torch.zeros(2, dtype=i32), 1, 1)


def test_append_marshals_and_refuses(rec):
    c = make()
    qkv = torch.zeros((3, 8, 128), dtype=bf16)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    lens = torch.ones(3, dtype=i32)
    freq = torch.ones(32)
    out = mala.mala_cache_append(c, k, v, lens, inv_freq=freq, q=q)
    name, a = rec.calls[-1]
    assert name == "mala_cache_append" and out.shape == (3, 4, 128) and out.is_contiguous()
    assert a[0] == c._ref
    assert list(a[1:4]) == [k.data_ptr(), 1024, 128] and list(a[4:7]) == [v.data_ptr(), 1024, 128]
    assert list(a[7:10]) == [q.data_ptr(), 1024, 128]
    assert list(a[10:13]) == [out.data_ptr(), 512, 128]
    assert list(a[13:]) == [None, lens.data_ptr(), 3, 3, 1, 4, freq.data_ptr(), 64, 0, None]
    assert mala.mala_cache_append(c, k, v, lens) is None
    assert rec.calls[-1][1][7:13] == (None, 0, 0, None, 0, 0) and rec.calls[-1][1][19] is None
    cu = torch.tensor([0, 1, 3], dtype=i32)
    assert mala.mala_cache_append(c, k, v, lens[:2], cu_seqlens=cu, q=q, q_out=q,
                                  interleaved=True) is q
    assert list(rec.calls[-1][1][13:]) == [cu.data_ptr(), lens.data_ptr(), 2, 3, 3, 4, None, 0, 1,
                                           None]
    ok = dict(cache=c, k=k, v=v, seq_lens=lens, inv_freq=freq, q=q)
    n = len(rec.calls)
    for kw, msg in (
            (dict(k=k[:2]), "one new token"),
            (dict(k=k.float()), "bf16"),
            (dict(v=v[:, :1]), "shape"),
            (dict(v=v[..., :64]), "shape"),
            (dict(k=torch.zeros((3, 2, 256), dtype=bf16)[..., ::2]), "contiguous"),
            (dict(k=torch.zeros(3 * 260, dtype=bf16).as_strided((3, 2, 128), (260, 128, 1))),
             "multiples of 8"),
            (dict(q=qkv[:, :3]), "multiple"),
            (dict(q_out=torch.zeros((3, 2, 128), dtype=bf16)), "shape"),
            (dict(q_out=torch.zeros((1, 4, 128), dtype=bf16).expand(3, 4, 128)), "overlap"),
            (dict(q=None, q_out=q), "without q"),
            (dict(seq_lens=lens.long()), "int32"),
            (dict(seq_lens=torch.ones(4, dtype=i32)), "page table"),
            (dict(cu_seqlens=torch.zeros(3, dtype=i32)), "entries"),
            (dict(cu_seqlens=torch.zeros(4, dtype=i32), max_new=-1), "negative"),
            (dict(inv_freq=torch.ones(12)), "multiple of 16"),
            (dict(inv_freq=torch.ones(72)), "multiple of 16"),
            (dict(inv_freq=freq.double()), "float32"),
            (dict(q=qkv[:, :4].to("meta")), "bf16"),
            (dict(q_out=qkv[:, :4].transpose(0, 1)), "shape")):
        with pytest.raises(ValueError, match=msg):
            mala.mala_cache_append(**{**ok, **kw})
    assert len(rec.calls) == n


def test_decode_marshals_and_refuses(rec):
    c = make()
    q = torch.zeros((3, 4, 128), dtype=bf16)
    lens = torch.zeros(3, dtype=i32)
    o, kept, bits = mala.mala_decode_paged(q, c, lens, tau=0.5, per_head=True, trace=True)
    name, a = rec.calls[-1]
    assert name == "mala_decode_paged" and kept.shape == (3, 4) and bits.shape == (3, 4, 1)
    assert list(a[:7]) == [c._ref, q.data_ptr(), o.data_ptr(), lens.data_ptr(), 3, 4, 64]
    assert a[7] == 0.5 and a[9] == 1
    assert mala.mala_decode_paged(q[:2], c, lens[:2], max_seqlen=5000, trace=True)[2].shape == \
        (2, 2, 2)
    n = len(rec.calls)
    for kw, msg in ((dict(q=q.float()), "bf16"), (dict(q=q[:, :, :64]), "contiguous"),
                    (dict(q=q[:, :3].contiguous()), "multiple"),
                    (dict(q=q[:2]), "entries"), (dict(seq_lens=lens.long()), "int32"),
                    (dict(max_seqlen=0), "positive"), (dict(out=q[:2]), "shape"),
                    (dict(out=q.float()), "must be"),
                    (dict(q=torch.zeros((4, 4, 128), dtype=bf16),
                          seq_lens=torch.zeros(4, dtype=i32)), "page table")):
        with pytest.raises(ValueError, match=msg):
            mala.mala_decode_paged(**{**dict(q=q, cache=c, seq_lens=lens), **kw})
    assert len(rec.calls) == n


def test_gather_marshals_and_refuses(rec):
    c = make()
    cu = torch.tensor([0, 5, 5, 9], dtype=i32)
    k, v = mala.mala_cache_gather(c, cu, max_seqlen=5, total=9)
    assert k.shape == v.shape == (9, 2, 128) and k.dtype == bf16
    assert rec.calls[-1][1] == (c._ref, k.data_ptr(), v.data_ptr(), cu.data_ptr(), 3, 5, 9, None)
    assert mala.mala_cache_gather(c, cu, 5, 9, out=(v, k))[0] is v
    n = len(rec.calls)
    for kw, msg in ((dict(cu_seqlens_k=cu.long()), "int32"), (dict(total=-1), "negative"),
                    (dict(out=(k, k[:8])), "shape"), (dict(out=(k.float(), v)), "must be"),
                    (dict(cu_seqlens_k=torch.zeros(5, dtype=i32)), "page table"),
                    (dict(cu_seqlens_k=torch.zeros(1, dtype=i32)), "batch")):
        with pytest.raises(ValueError, match=msg):
            mala.mala_cache_gather(**{**dict(cache=c, cu_seqlens_k=cu, max_seqlen=5, total=9), **kw})
    assert len(rec.calls) == n


def test_bounds_beyond_32_bits_are_refused(rec):
    """They would wrap on their way into the library: 2**32 + 100 into a bound of 100."""
    c = make()
    q, kv = torch.zeros((3, 4, 128), dtype=bf16), torch.zeros((3, 2, 128), dtype=bf16)
    lens, cu = torch.ones(3, dtype=i32), torch.tensor([0, 1, 2, 3], dtype=i32)
    for big in (2 ** 31, 2 ** 32 + 100, 2 ** 63):
        for call in (lambda: mala.mala_decode_paged(q, c, lens, max_seqlen=big),
                     lambda: mala.mala_cache_append(c, kv, kv, lens, cu_seqlens=cu, max_new=big),
                     lambda: mala.mala_cache_gather(c, cu, big, 3),
                     lambda: mala.mala_cache_gather(c, cu, 3, big)):
            with pytest.raises(ValueError, match="2\\*\\*31"):
                call()
    assert not rec.calls
    mala.mala_decode_paged(q, c, lens, max_seqlen=2 ** 31 - 1)
    assert rec.calls[-1][1][6] == 2 ** 31 - 1


# ------------------------------------------------------------------ the C entry points
def struct(**kw):
    f = dict(k_pages=256, v_pages=256, k_scale=256, v_scale=256, page_table=256,
             k_stride_page=4096, k_stride_head=2048, k_stride_token=128, v_stride_page=4096,
             v_stride_head=2048, v_stride_token=128, table_stride=4, num_pages=6, page_size=16,
             max_pages=4, Hkv=2, d=128)
    f.update(kw)
    return mala._CacheStruct(**f)


def test_c_cache_checks(lib):
    def call(s):
        return lib.mala_cache_gather(ctypes.addressof(s) if s else None, 256, 256, 256, 1, 0, 0,
                                     None)
    assert call(struct()) == 0  # nothing to do
    assert call(None) == 1
    for kw in (dict(k_pages=None), dict(v_scale=None), dict(page_table=None), dict(k_pages=264),
               dict(k_scale=258), dict(page_table=257), dict(num_pages=0), dict(max_pages=0),
               dict(Hkv=0), dict(Hkv=70000), dict(k_stride_page=0), dict(k_stride_head=64),
               dict(v_stride_token=-128), dict(v_stride_token=136), dict(table_stride=3),
               dict(max_pages=1 << 30, table_stride=1 << 30), dict(k_stride_page=1 << 41)):
        assert call(struct(**kw)) == 1, kw
    for kw in (dict(d=64), dict(page_size=24), dict(page_size=256), dict(page_size=8)):
        assert call(struct(**kw)) == 2, kw
    assert call(struct(num_pages=1, k_stride_page=0)) == 0  # a stride that is not used


def test_c_append_checks(lib):
    c = struct()

    def call(k=256, kt=256, q=None, qo=None, qt=512, cu=256, lens=256, batch=2, total=3, new=2,
             Hq=4, freq=256, rot=64, inter=0):
        return lib.mala_cache_append(ctypes.addressof(c), k, kt, 128, 256, 256, 128, q, qt, 128, qo,
                                     512, 128, cu, lens, batch, total, new, Hq, freq, rot, inter,
                                     None)
    assert call(total=0) == 0 and call(new=0) == 0
    for kw in (dict(k=None), dict(k=264), dict(kt=100), dict(q=256), dict(q=256, qo=250),
               dict(q=256, qo=256, qt=4), dict(q=256, qo=256, Hq=3), dict(q=256, qo=256, Hq=0),
               dict(lens=None), dict(lens=257), dict(cu=None), dict(freq=None), dict(batch=0),
               dict(batch=70000), dict(total=-1), dict(new=-1), dict(inter=2)):
        assert call(**kw) == 1, kw
    assert call(rot=24) == 2 and call(rot=144) == 2 and call(rot=-16) == 2


def test_c_decode_checks(lib):
    c = struct()

    def call(q=256, o=256, lens=256, batch=2, Hq=4, n=0, tau=1.0, ph=0, kept=None, bits=None):
        return lib.mala_decode_paged(ctypes.addressof(c), q, o, lens, batch, Hq, n, tau, 0.0, ph,
                                     kept, bits, None)
    for kw in (dict(q=None), dict(o=None), dict(lens=None), dict(q=264), dict(o=8), dict(lens=258),
               dict(kept=2), dict(bits=2), dict(batch=0), dict(batch=70000), dict(Hq=0),
               dict(Hq=3), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")),
               dict(ph=2)):
        assert call(**kw) == 1, kw
    assert call(Hq=18) == 2  # nine query heads per key/value head


def test_c_gather_checks(lib):
    c = struct()

    def call(k=256, v=256, cu=256, batch=1, n=4, total=4):
        return lib.mala_cache_gather(ctypes.addressof(c), k, v, cu, batch, n, total, None)
    for kw in (dict(k=None), dict(v=None), dict(k=264), dict(cu=None), dict(cu=254), dict(batch=0),
               dict(batch=70000), dict(n=-1), dict(total=-1)):
        assert call(**kw) == 1, kw
    assert call(total=0) == 0 and call(n=0) == 0
