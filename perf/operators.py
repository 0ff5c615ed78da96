"""The serving cache's operators: what a pass of each does, its plain form and its exact answer.

Three operators around one data structure, a paged key/value cache in 8 bits (e4m3, one float32
scale per page and key/value head):

* ``append`` -- new tokens' keys (rotated by position) and values into the pages, queries rotated;
* ``decode`` -- one step of MALA decode attention over the pages;
* ``gather`` -- the pages of some sequences back as packed bf16 keys and values for a prefill.

``own`` false: the plain forms, elementary torch operations in float32. ``own`` true: the calls of
``mass_adaptive_causal_b200``.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128        # head dimension
TILE = 128     # keys per tile of the decode rule
E4M3_MAX = 448.0
MIN_EXP = -100


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one chat user, a short context: the latency of a step
        dict(name="decode_1x1000", op="decode", B=1, Hq=32, Hkv=8, len=1000, ragged=0, empty=0,
             page=16, tau=1.0, per_head=False),
        # continuous batching: lengths from a few tokens to 16K, one slot of the batch unused
        dict(name="decode_ragged_24x16k", op="decode", B=24, Hq=32, Hkv=8, len=16384, ragged=5,
             empty=1, page=64, tau=1.0, per_head=False),
        # ordinary batch, exact attention (tau = 0 keeps every tile)
        dict(name="decode_16x8k_dense", op="decode", B=16, Hq=32, Hkv=8, len=8192, ragged=0,
             empty=0, page=64, tau=0.0, per_head=False),
        # eight query heads per cached head, each deciding alone
        dict(name="decode_8x32k_per_head", op="decode", B=8, Hq=64, Hkv=8, len=32767, ragged=0,
             empty=0, page=128, tau=1.0, per_head=True),
        # the repository's long decode workload, with its cache in pages of 8 bits
        dict(name="decode_16x128k", op="decode", B=16, Hq=32, Hkv=8, len=131072, ragged=0,
             empty=0, page=64, tau=1.0, per_head=False),
        # long contexts, exact attention, small pages, no grouping of heads beyond four
        dict(name="decode_4x128k_dense", op="decode", B=4, Hq=32, Hkv=8, len=131072, ragged=0,
             empty=0, page=32, tau=0.0, per_head=False),
        # one decode step's tokens of a small batch (a fused projection's rows, q rotated too)
        dict(name="append_step_16", op="append", B=16, Hq=32, Hkv=8, len=2000, ragged=3, new=1,
             page=64, rot=128, interleaved=False, with_q=True),
        # one decode step of a large batch, small pages
        dict(name="append_step_256", op="append", B=256, Hq=32, Hkv=8, len=300, ragged=4, new=1,
             page=16, rot=128, interleaved=False, with_q=True),
        # chunks of several prompts, half of the head rotated in adjacent pairs, queries elsewhere
        dict(name="append_chunks_12", op="append", B=12, Hq=16, Hkv=4, len=3000, ragged=7,
             new=2048, page=32, rot=64, interleaved=True, with_q=False),
        # whole prompts at once
        dict(name="append_prompt_4x8k", op="append", B=4, Hq=32, Hkv=8, len=8192, ragged=0,
             new=8192, page=128, rot=128, interleaved=False, with_q=True),
        # a few caches read back for the next chunk of their prompts
        dict(name="gather_9x4k", op="gather", B=9, Hkv=4, len=4096, ragged=6, page=16),
        # long caches read back
        dict(name="gather_4x128k", op="gather", B=4, Hkv=8, len=131072, ragged=0, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "append", "gather"])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    ragged = rng.choice([0, rng.randrange(1, 1000), rng.randrange(1, 1000)])
    if op == "decode":
        G = rng.randrange(1, 9)
        L = _log_int(rng, 1, 131072)
        B = _log_int(rng, 1, max(1, min(128, 16 * 131072 * 8 // (L * Hkv))))
        return dict(op="decode", B=B, Hq=G * Hkv, Hkv=Hkv, len=L, ragged=ragged,
                    empty=rng.choice([0, 0, 1]) if B > 1 and ragged else 0, page=page,
                    tau=rng.choice([0.0, 0.25, 1.0, 1.0]), per_head=rng.random() < 0.3)
    if op == "append":
        G = rng.randrange(1, 9)
        new = rng.choice([1, _log_int(rng, 1, 8192)])
        L = new + _log_int(rng, 1, 2000)
        B = _log_int(rng, 1, max(1, min(256, 4 * 8192 // new, 262144 // L)))
        return dict(op="append", B=B, Hq=G * Hkv, Hkv=Hkv, len=L, ragged=ragged, new=new,
                    page=page, rot=rng.choice([32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, with_q=rng.random() < 0.7)
    L = _log_int(rng, 1, 131072)
    return dict(op="gather", B=_log_int(rng, 1, max(1, min(64, 4 * 131072 * 8 // (L * Hkv)))),
                Hkv=Hkv, len=L, ragged=ragged, page=page)


def lens_of(case):
    """Cache lengths (new tokens included) of a case's sequences: all ``len``, or spread over
    1..len on a log scale with the first one full; ``empty`` slots at the end hold nothing."""
    if not case["ragged"]:
        lens = [case["len"]] * case["B"]
    else:
        r = random.Random(case["ragged"])
        lens = [case["len"]] + [_log_int(r, 1, case["len"]) for _ in range(case["B"] - 1)]
    for i in range(case.get("empty", 0)):
        lens[-1 - i] = 0
    return lens


def news_of(case):
    """New tokens of each sequence: at most ``new``, and no more than its length."""
    r = random.Random(case["ragged"] + 1)
    return [min(n, case["new"] if not case["ragged"] else _log_int(r, 1, case["new"]))
            for n in lens_of(case)]


def work(case):
    lens = lens_of(case)
    T, page = sum(lens), case["page"]
    pages = sum(-(-n // page) for n in lens)
    Hkv = case["Hkv"]
    if case["op"] == "decode":
        live = sum(n > 0 for n in lens)
        qo = case["B"] * case["Hq"] * D * 4
        k = T * Hkv * D + pages * (4 * Hkv + 4)
        if case["tau"] == 0.0:  # every key and every value
            return {"bytes": 2 * k - 4 * pages + qo, "flops": 4 * D * T * case["Hq"]}
        # every key, and at least the newest tile's values
        newest = sum(min(n, (n - 1) % TILE + 1) for n in lens)
        return {"bytes": k + newest * Hkv * D + 4 * Hkv * live + qo,
                "flops": 2 * D * case["Hq"] * (T + newest)}
    if case["op"] == "append":
        new = sum(news_of(case))
        touched = sum((n - 1) // page - (n - m) // page + 1 for n, m in zip(lens, news_of(case)))
        q = new * case["Hq"] * D * 4 if case["with_q"] else 0
        rotated = new * (Hkv + (case["Hq"] if case["with_q"] else 0)) * case["rot"]
        return {"bytes": new * Hkv * D * 2 * 3 + q + touched * (8 * Hkv + 4),
                "flops": 3 * rotated + 2 * new * Hkv * D * 2}
    return {"bytes": T * Hkv * D * 2 * 3 + pages * (8 * Hkv + 4), "flops": 2 * T * Hkv * D}


# ------------------------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """The least power of two s >= 2^MIN_EXP with amax <= 448 s (448 = 1.75 * 2^8)."""
    f, e = torch.frexp(amax.double())            # amax = f * 2^e, f in [0.5, 1)
    e = torch.where(f > 0.875, e + 1, e) - 9
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(f), e)


def _to_pages(x, page):
    """[H, L, D] float32 -> e4m3 [pages, H, page, D] and its scales [pages, H]."""
    H, L, _ = x.shape
    n = -(-L // page)
    x = torch.nn.functional.pad(x, (0, 0, 0, n * page - L)).view(H, n, page, D).transpose(0, 1)
    s = _pow2_scale(x.abs().amax((2, 3))).float()
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _ar1(shape, L, rho, g):
    """Latent x_t = rho x_{t-1} + sqrt(1 - rho^2) e_t along a length-L axis: [*shape, L, D]."""
    x = torch.randn((*shape, L, D), device="cuda", generator=g)
    x[..., 1:, :] *= math.sqrt(1 - rho * rho)
    step = 1
    while step < min(L, 1024):
        y = x.clone()
        y[..., step:, :].add_(x[..., :-step, :], alpha=rho ** step)
        x, step = y, step * 2
    return x


def _cache(case, g, fill):
    """A pool with some spare pages, its scales, and a table that gives each sequence pages from
    all over it. ``fill(b, length)`` makes a sequence's keys and values, [Hkv, length, D]."""
    lens, page, Hkv = lens_of(case), case["page"], case["Hkv"]
    counts = [-(-n // page) for n in lens]
    total = sum(counts) + 3
    order = torch.randperm(total, device="cuda", generator=g)
    k8 = torch.zeros((total, Hkv, page, D), dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    ks = torch.ones((total, Hkv), device="cuda")
    vs = torch.ones((total, Hkv), device="cuda")
    width = max(1, max(counts))
    table = torch.zeros((case["B"], width), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        if n:
            ids = order[at:at + counts[b]]
            at += counts[b]
            table[b, :counts[b]] = ids.int()
            for x, pool, scales in zip(fill(b, n), (k8, v8), (ks, vs)):
                x8, s = _to_pages(x, page)
                pool[ids] = x8.view(torch.uint8)
                scales[ids] = s
    f8 = torch.float8_e4m3fn
    return dict(k_pages=k8.view(f8), v_pages=v8.view(f8), k_scale=ks, v_scale=vs, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    """Inputs with the structure long-context attention meets: keys that drift slowly (AR(1)), a
    sink at position 0, keys that other queries and this step's queries single out."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, Hkv = lens_of(case), case["Hkv"]
    s = dict(case=case)
    rho = 0.98
    c = math.sqrt(1 - rho * rho)
    u = torch.randn(D, device="cuda", generator=g)
    u = u / u.norm()
    if case["op"] == "decode":
        G = case["Hq"] // Hkv
        q = torch.zeros((case["B"], Hkv, G, D), device="cuda")

        def fill(b, n):
            x = _ar1((Hkv,), n, rho, g)
            k = 2.5 * x
            k[:, 0] += 6.0 * u
            qb = 2.5 * (rho * x[:, -1:] + c * torch.randn((Hkv, G, D), device="cuda", generator=g))
            q[b] = qb + 1.5 * u
            aim = lambda y: 2.5 * math.sqrt(D) * y / y.norm(dim=-1, keepdim=True)  # noqa: E731

            def places(count):  # distinct positions in [1, n - 256), one from each equal stretch
                cell = (n - 257) // count
                at = torch.rand((Hkv, count), device="cuda", generator=g) * cell
                return 1 + cell * torch.arange(count, device="cuda") + at.long().clamp(max=cell - 1)

            if n > 300:
                i = torch.randint(258, n, (Hkv, n // 128), device="cuda", generator=g)
                h = torch.arange(Hkv, device="cuda")[:, None]
                k[h, places(n // 128)] = aim(2.5 * x[h, i] + 1.5 * u)
                k[h, places(4 * G)] = aim(q[b].repeat(1, 4, 1))
            return k, torch.randn((Hkv, n, D), device="cuda", generator=g)

        s.update(_cache(case, g, fill))
        s["q"] = q.view(case["B"], case["Hq"], D).bfloat16()
        s["max_len"] = max(lens)
    elif case["op"] == "append":
        def fill(b, n):
            # earlier tokens, of a size that the new ones sometimes exceed
            size = torch.rand((2, Hkv, 1, 1), device="cuda", generator=g) * 3 + 0.5
            x = torch.randn((2, Hkv, n, D), device="cuda", generator=g) * size
            return x[0], x[1]

        s.update(_cache(case, g, fill))
        new = news_of(case)
        T = sum(new)
        heads = (case["Hq"] if case["with_q"] else 0) + 2 * Hkv
        qkv = torch.randn((T, heads, D), device="cuda", generator=g)
        qkv *= torch.where(torch.rand(heads, D, device="cuda", generator=g) < 0.03, 6.0, 1.0)
        qkv = qkv.bfloat16()  # rows of a fused projection: q, k, v are views of it
        hq = heads - 2 * Hkv
        s.update(q=qkv[:, :hq] if hq else None, k=qkv[:, hq:hq + Hkv], v=qkv[:, hq + Hkv:])
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if case["new"] > 1 else None
        s["max_new"] = max(new)
        s["total"] = T
        half = case["rot"] // 2
        s["inv_freq"] = (500000.0 ** (-torch.arange(half, device="cuda") / half)).float()
    else:
        def fill(b, n):
            x = torch.randn((2, Hkv, n, D), device="cuda", generator=g)
            return 2.5 * x[0], x[1]

        s.update(_cache(case, g, fill))
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["max_len"], s["total"] = max(lens), cu[-1]
    if own:
        import mass_adaptive_causal_b200 as mala
        s["cache"] = mala.PagedCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                     s["table"])
    return s


# ------------------------------------------------------------------------------------ a pass
def run(s):
    case = s["case"]
    if own:
        import mass_adaptive_causal_b200 as mala
        if case["op"] == "decode":
            return mala.mala_decode_paged(s["q"], s["cache"], s["lens"], tau=case["tau"],
                                          per_head=case["per_head"], max_seqlen=s["max_len"])
        if case["op"] == "append":
            q = mala.mala_cache_append(s["cache"], s["k"], s["v"], s["lens"], cu_seqlens=s["cu"],
                                       max_new=s["max_new"], inv_freq=s["inv_freq"],
                                       interleaved=case["interleaved"], q=s["q"])
            return q, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
        return mala.mala_cache_gather(s["cache"], s["cu"], max_seqlen=s["max_len"],
                                      total=s["total"])
    return {"decode": _plain_decode, "append": _plain_append, "gather": _plain_gather}[case["op"]](s)


def _values(pages, scale, ids):
    """float32 values of the pages ``ids`` [...]: [..., Hkv, page, D]."""
    x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    return x * scale[ids][..., None, None]


def _plain_decode(s):
    case, lens, q = s["case"], s["lens"].long(), s["q"]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    G, ids = Hq // Hkv, s["table"].long()
    seq = lambda x: x.transpose(1, 2).reshape(B, Hkv, -1, D)  # noqa: E731
    k = seq(_values(s["k_pages"], s["k_scale"], ids))
    L = k.shape[2]
    x = torch.matmul(q.view(B, Hkv, G, D).float(), k.transpose(2, 3)) / math.sqrt(D)
    del k
    pos = torch.arange(L, device=q.device)
    x = x.masked_fill(pos >= lens.view(B, 1, 1, 1), -math.inf)
    if case["tau"] > 0:
        nt = -(-L // TILE)
        x = torch.nn.functional.pad(x, (0, nt * TILE - L), value=-math.inf)
        tiles = x.view(B, Hkv, G, nt, TILE)
        mt = tiles.amax(-1)
        lt = (tiles - mt.clamp(min=-1e30)[..., None]).exp().sum(-1)
        bound = (math.log(case["tau"]) - torch.log(lens.clamp(min=1).float())).view(B, 1, 1)
        newest = ((lens - 1) // TILE).view(B, 1, 1)
        m = torch.full_like(mt[..., 0], -1e30)
        l = torch.zeros_like(m)
        keep = torch.zeros_like(mt, dtype=torch.bool)
        for t in range(nt - 1, -1, -1):  # the rule is a recurrence over the tiles, newest first
            want = mt[..., t] - m - l.log() >= bound
            if not case["per_head"]:
                want = want.any(-1, keepdim=True).expand_as(want)
            want = (want & (newest > t)) | (newest == t)
            m2 = torch.where(want, torch.maximum(m, mt[..., t]), m)
            l = torch.where(want, l * (m - m2).exp() + lt[..., t] * (mt[..., t] - m2).exp(), l)
            m = m2
            keep[..., t] = want
        x = tiles.masked_fill(~keep[..., None], -math.inf).view(B, Hkv, G, nt * TILE)[..., :L]
    p = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p, seq(_values(s["v_pages"], s["v_scale"], ids)))
    return o.view(B, Hq, D).to(q.dtype)


def _rotated(x, pos, case, inv_freq):
    """float32 rows [T, H, D] rotated by their positions [T]."""
    angle = pos.double()[:, None, None] * inv_freq.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    x, rot = x.float(), case["rot"]
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_append(s):
    case, lens = s["case"], s["lens"].long()
    page, ids = case["page"], s["table"].long()
    if s["cu"] is None:
        n, seq = torch.ones_like(lens), torch.arange(case["B"], device=lens.device)
        first = seq
    else:
        n, first = (s["cu"][1:] - s["cu"][:-1]).long(), s["cu"][:-1].long()
        seq = torch.repeat_interleave(n, output_size=s["total"])
    start = lens - n
    pos = start[seq] + torch.arange(s["total"], device=lens.device) - first[seq]
    dest, row = ids[seq, pos // page], pos % page
    k = _rotated(s["k"], pos, case, s["inv_freq"])
    q = None if s["q"] is None else _rotated(s["q"], pos, case, s["inv_freq"]).to(s["q"].dtype)
    has, used = ids.gather(1, (start // page)[:, None])[:, 0], start % page
    for x, pages, scale in ((k, s["k_pages"], s["k_scale"]),
                            (s["v"].float(), s["v_pages"], s["v_scale"])):
        pages = pages.view(torch.uint8)
        finite = x.isfinite()
        amax = torch.full_like(scale, -1.0)
        amax.index_reduce_(0, dest, x.abs().where(finite, 0.0).amax(-1), "amax")
        old = torch.zeros_like(scale)
        old[has] = torch.where((used > 0)[:, None], scale[has], 0.0)
        new = torch.maximum(_pow2_scale(amax).float(), old)
        earlier = pages[has].view(torch.float8_e4m3fn).float()   # [B, Hkv, page, D]
        earlier = earlier * (old[has] / new[has])[..., None, None]
        held = (torch.arange(page, device=lens.device) < used[:, None])[:, None, :, None]
        pages[has] = torch.where(held, earlier.to(torch.float8_e4m3fn).view(torch.uint8),
                                 pages[has])
        scale.copy_(torch.where(amax >= 0, new, scale))
        x = x.where(finite, math.nan) / new[dest][..., None]
        pages[dest, :, row] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return q, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _plain_gather(s):
    case, cu = s["case"], s["cu"].long()
    seq = torch.repeat_interleave(cu[1:] - cu[:-1], output_size=s["total"])
    pos = torch.arange(s["total"], device=cu.device) - cu[seq]
    ids, row = s["table"].long()[seq, pos // case["page"]], pos % case["page"]
    out = []
    for pages, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
        x = pages.view(torch.uint8)[ids, :, row].view(torch.float8_e4m3fn).float()
        out.append((x * scale[ids][..., None]).bfloat16())
    return tuple(out)


# ------------------------------------------------------------------------------------ 64 bits
def _round_e4m3(x):
    """The nearest e4m3 value, ties to even, of |x| <= 448 (float64); the rest is NaN."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.ldexp(torch.ones_like(x), e.int()) > x.abs(), e - 1, e).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(x), (e - 3).int())
    return torch.where(x.abs() <= 448, torch.round(x / step) * step, math.nan)


def _exact_decode(s):
    case = s["case"]
    Hkv, G, page = case["Hkv"], case["Hq"] // case["Hkv"], case["page"]
    o = torch.zeros((case["B"], case["Hq"], D), dtype=torch.float64, device="cuda")
    lens = lens_of(case)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        kv = []
        for pages, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            x = x * scale[ids].double()[:, :, None, None]
            kv.append(x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n])
        score = torch.einsum("hgd,hld->hgl", s["q"][b].double().view(Hkv, G, D), kv[0]) / D ** 0.5
        keep = torch.ones((Hkv, G, n), dtype=torch.bool, device="cuda")
        if case["tau"] > 0:
            bound = math.log(case["tau"]) - math.log(n)
            edges = list(range(0, n, TILE))
            top = torch.stack([score[..., t:t + TILE].amax(-1) for t in edges], -1).cpu()
            mass = torch.stack([score[..., t:t + TILE].logsumexp(-1) for t in edges], -1).cpu()
            lse = mass[..., -1].clone()          # log of the kept mass; the newest tile is kept
            kept = torch.ones((Hkv, G, len(edges)), dtype=torch.bool)
            for t in range(len(edges) - 2, -1, -1):
                w = top[..., t] - lse >= bound
                if not case["per_head"]:
                    w = w.any(-1, keepdim=True).expand_as(w)
                kept[..., t] = w
                lse = torch.where(w, torch.logaddexp(lse, mass[..., t]), lse)
            keep = kept.cuda().repeat_interleave(TILE, -1)[..., :n]
        p = torch.softmax(score.masked_fill(~keep, -math.inf), -1)
        o[b] = torch.einsum("hgl,hld->hgd", p, kv[1]).reshape(-1, D)
    return o


def _exact_append(s):
    case, lens, new = s["case"], lens_of(s["case"]), news_of(s["case"])
    page, Hkv, rot = case["page"], case["Hkv"], case["rot"]
    where = torch.tensor([p for n, m in zip(lens, new) for p in range(n - m, n)], device="cuda")
    seq = torch.tensor([b for b, m in enumerate(new) for _ in range(m)], device="cuda")
    at = (torch.arange(rot // 2, device="cuda"), torch.arange(rot // 2, rot, device="cuda"))
    if case["interleaved"]:
        at = (torch.arange(0, rot, 2, device="cuda"), torch.arange(1, rot, 2, device="cuda"))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       where.double()[:, None] * s["inv_freq"].double()[None])[:, None]

    def spin(x):
        y = x.double().clone()
        z = torch.complex(y[..., at[0]], y[..., at[1]]) * turn
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    out = [None if s["q"] is None else spin(s["q"])]
    owner = s["table"].long()[seq, where // page]
    scales = []
    for x, pages, scale in ((spin(s["k"]), s["k_pages"], s["k_scale"]),
                            (s["v"].double(), s["v_pages"], s["v_scale"])):
        val = pages.view(torch.uint8).view(torch.float8_e4m3fn).double()
        sc = scale.double()
        need = torch.zeros_like(sc)
        need.scatter_reduce_(0, owner[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        e = torch.ceil(torch.log2(need / 448)).clamp(min=MIN_EXP)
        e = e - 1  # log2 may be off by one next to a whole number: the least e that holds
        for _ in range(2):
            low = torch.ldexp(torch.full_like(sc, 448.0), e.int()) < need
            e = torch.where(low, e + 1, e).clamp(min=MIN_EXP)
        least = torch.ldexp(torch.ones_like(sc), e.int())
        fresh = torch.zeros(sc.shape[0], dtype=torch.bool, device="cuda")
        fresh[owner] = True
        first = torch.zeros_like(fresh)
        for b, (n, m) in enumerate(zip(lens, new)):
            if m and (n - m) % page:
                i = int(s["table"][b, (n - m) // page])
                first[i] = True
                grown = torch.maximum(least[i], sc[i])
                u = (n - m) % page
                val[i, :, :u] = _round_e4m3(val[i, :, :u] * (sc[i] / grown)[:, None, None])
        sc = torch.where(first[:, None], torch.maximum(least, sc),
                         torch.where(fresh[:, None], least, sc))
        val[owner, :, where % page] = _round_e4m3(x / sc[owner][..., None])
        out.append(val)
        scales.append(sc)
    return tuple(out + scales)


def _exact_gather(s):
    case = s["case"]
    page, out = case["page"], []
    for pages, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
        rows = []
        for b, n in enumerate(lens_of(case)):
            ids = s["table"][b, :-(-n // page)].long()
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            x = x * scale[ids].double()[:, :, None, None]
            rows.append(x.transpose(1, 2).reshape(-1, case["Hkv"], D)[:n])
        out.append(torch.cat(rows))
    return tuple(out)


def exact(case, seed):
    """The operators' definitions in float64, sequence by sequence."""
    s = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "gather": _exact_gather}[case["op"]](s)
