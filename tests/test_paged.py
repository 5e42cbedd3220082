"""The paged-cache operators (append_kv, attend_paged, decode_attend) against their
definitions in 64 bits, and their refusals."""
import ctypes
import math

import pytest
import torch

import block_sparse_long_up_gb300 as up
from block_sparse_long_up_gb300.paged import _CKv, _CLogits

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ refusals (no GPU)

@pytest.fixture(scope="module")
def L():
    up.build()
    return up.lib()


def _cache(**kw):
    a = dict(k=256, v=256, pos=256, table=256, lens=256, pages=64, B=2, maxp=8, page=128, Hk=2,
             d=64, dtype=0)
    a.update(kw)
    return ctypes.byref(_CKv(a["k"], a["v"], a["pos"], a["table"], a["lens"], a["pages"], a["B"],
                             a["maxp"], a["page"], a["Hk"], a["d"], a["dtype"]))


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
              (dict(k=264), 1), (dict(v=258), 1), (dict(pages=0), 1), (dict(pages=-1), 1),
              (dict(pages=1 << 31), 1), (dict(B=-1), 1), (dict(maxp=0), 1), (dict(page=0), 1),
              (dict(page=24), 1), (dict(page=-16), 1), (dict(Hk=0), 1), (dict(d=96), 2),
              (dict(d=0), 2), (dict(dtype=2), 2), (dict(pos=258), 1),
              (dict(Hk=1 << 14, page=1 << 18), 1)]


def _append(L, cache=None, q=256, qs=512, k=256, ks=128, v=256, vs=128, pos=256, A=1, axes=None,
            f=256, rot=64, flags=0, cu=256, T=10, Hq=8, out=512):
    return L.up_append_kv(q, qs, k, ks, v, vs, pos, A, axes, f, rot, flags, cu, T, Hq,
                          cache or _cache(), out, None)


def _attend(L, cache=None, q=256, cu=256, T=10, Hq=8, lg=(0.1, 0.0, None, None), vis=None, out=256,
            lse=256, ws=256, wsb=1 << 40):
    return L.up_attend_paged(q, cu, T, Hq, cache or _cache(), ctypes.byref(_CLogits(*lg)), vis, out,
                             lse, ws, wsb, None)


def _decode(L, cache=None, q=256, Hq=8, lg=(0.1, 0.0, None, None), start=None, out=256, lse=256,
            ws=256, wsb=1 << 40):
    return L.up_decode_attend(q, Hq, cache or _cache(), ctypes.byref(_CLogits(*lg)), start, out,
                              lse, ws, wsb, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, code):
    c = _cache(**bad)
    big = max(1, bad.get("Hk", 2)) * 64
    assert _append(L, cache=c, ks=big, vs=big) == code
    assert _attend(L, cache=c, Hq=max(1, bad.get("Hk", 4))) == code
    assert _decode(L, cache=c, Hq=max(1, bad.get("Hk", 4))) == code


def test_append_refusals(L):
    for bad in (dict(k=None), dict(v=None), dict(pos=None), dict(cu=None), dict(q=None),
                dict(out=None), dict(f=None), dict(rot=8), dict(rot=80), dict(rot=-16),
                dict(flags=2), dict(T=-1), dict(T=1 << 31), dict(Hq=-1), dict(A=0), dict(qs=504),
                dict(ks=120), dict(vs=120), dict(qs=516), dict(ks=132), dict(k=264), dict(q=264),
                dict(out=264), dict(out=256, qs=520), dict(pos=257), dict(axes=258)):
        assert _append(L, **bad) == 1, bad
    assert L.up_append_kv(*[None] * 1, 0, None, 0, None, 0, None, 1, None, None, 0, 0, None, 0, 0,
                          None, None, None) == 1  # no cache
    assert _append(L, T=0) == 0  # nothing to do


def test_attend_refusals(L):
    for call in (_attend, _decode):
        for bad in (dict(q=None), dict(out=None), dict(q=264), dict(out=264), dict(lse=258),
                    dict(Hq=0), dict(Hq=7), dict(Hq=-8), dict(lg=(math.inf, 0.0, None, None)),
                    dict(lg=(math.nan, 0.0, None, None)), dict(lg=(0.1, -1.0, None, None)),
                    dict(lg=(0.1, math.inf, None, None)), dict(lg=(0.1, 1e-7, None, None)),
                    dict(lg=(0.1, 0.0, 256, None)),
                    dict(lg=(0.1, 0.0, 256, 256), cache=_cache(pos=None))):
            assert call(L, **bad) == 1, bad
        assert call(L, Hq=64) == 2  # 32 query heads on a KV head
        for bad in (dict(ws=None), dict(ws=272), dict(wsb=0)):
            assert call(L, **bad) == 3, bad
    assert _attend(L, cu=None) == 1 and _attend(L, T=-1) == 1 and _attend(L, T=1 << 31) == 1
    assert _attend(L, T=1 << 29) == 1  # rows past 32 bits
    assert _attend(L, vis=260) == 1 and _decode(L, start=258) == 1
    assert _attend(L, T=0) == 0 and _decode(L, cache=_cache(B=0)) == 0


def test_workspace_sizes(L):
    assert up.attend_paged_workspace(1000, 4, 8, 2, 64) > 0
    assert up.decode_attend_workspace(4, 8, 2, 64) > 0
    for bad in ((8, 3, 64), (8, 2, 96), (64, 2, 64), (0, 2, 64), (8, 0, 64)):
        assert up.attend_paged_workspace(1000, 4, *bad) == 0
        assert up.decode_attend_workspace(4, *bad) == 0
    assert up.attend_paged_workspace(-1, 4, 8, 2, 64) == 0
    assert up.decode_attend_workspace(-1, 8, 2, 64) == 0


def test_python_refuses_host_tensors():
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        up.PagedKV(kp, kp, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        up.PagedKV(kp.float(), kp.float(), torch.zeros(1, 4, dtype=torch.int32),
                   torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        up.PagedKV(None, kp, None, None)


# ------------------------------------------------------------------ a cache and its oracle

class Made:
    """A cache of shuffled pages. Slots past a sequence's length and pages that nobody
    names hold NaN; with slack, table rows are longer than needed and end in -1."""

    def __init__(self, lens, Hk, d, page, dtype, seed=0, poison=True, extra=3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.lens, self.Hk, self.d, self.page = g, lens, Hk, d, page
        dt = self.dt = DT[dtype]
        B = len(lens)
        need = [-(-kv // page) for _, kv in lens]
        maxp, n = max(need + [1]) + 1, sum(need) + extra
        order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((B, maxp), -1, dtype=torch.int32, device="cuda")
        self.kp = torch.randn(n, Hk, page, d, generator=g, device="cuda").to(dt)
        self.vp = torch.randn(n, Hk, page, d, generator=g, device="cuda").to(dt)
        self.pp = torch.zeros(n, page, dtype=torch.int32, device="cuda")
        at, used = 0, torch.zeros(n, page, dtype=torch.bool, device="cuda")
        for s, (_, kv) in enumerate(lens):
            self.table[s, :need[s]] = order[at:at + need[s]]
            p = (torch.randint(1, 4, (need[s] * page,), generator=g, device="cuda").cumsum(0)
                 if kv else torch.zeros(0, device="cuda"))
            self.pp[order[at:at + need[s]].long()] = p.view(-1, page).to(torch.int32)
            i = torch.arange(kv, device="cuda")
            used[self.table[s].long()[i // page], i % page] = True
            at += need[s]
        if poison:
            self.kp.masked_fill_(~used[:, None, :, None], math.nan)
            self.vp.masked_fill_(~used[:, None, :, None], math.nan)
        self.kv_lens = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
        self.cu = torch.tensor([0] + [n for n, _ in lens], dtype=torch.int32, device="cuda").cumsum(
            0, dtype=torch.int32)
        self.T = sum(n for n, _ in lens)
        self.cache = up.PagedKV(self.kp, self.vp, self.table, self.kv_lens, self.pp)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(self.dt)

    def tokens(self, s, x):
        """x's rows (per slot) of sequence s, in order."""
        kv = self.lens[s][1]
        i = torch.arange(kv, device="cuda")
        return x[self.table[s].long()[i // self.page], ..., i % self.page, :] if x.dim() == 4 else \
            x[self.table[s].long()[i // self.page], i % self.page]


def oracle(m, q, lo, hi, scale, softcap=0.0, slopes=None, q_pos=None):
    """(out, sum of weight * |value|, lse, largest |logit|) in 64 bits."""
    T, Hq, d = q.shape
    g = Hq // m.Hk
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    big, t0 = 1.0, 0
    for s, (n, kv) in enumerate(m.lens):
        if n and kv:
            k, v = m.tokens(s, m.kp).double(), m.tokens(s, m.vp).double()  # [kv, Hk, d]
            place, i = m.tokens(s, m.pp).double(), torch.arange(kv, device="cuda")
            rows = slice(t0, t0 + n)
            seen = (i >= lo[rows, None]) & (i < hi[rows, None])
            for h in range(Hq):
                z = q[rows, h].double() @ k[:, h // g].T * scale
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                if slopes is not None:
                    z = z - slopes[h].double() * (q_pos[rows].double()[:, None] - place).abs()
                z = z.masked_fill(~seen, -math.inf)
                if bool(seen.any()):
                    big = max(big, float(z[seen].abs().max()))
                l = torch.logsumexp(z, 1)
                w = torch.where(seen.any(1, keepdim=True), torch.exp(z - l[:, None]), torch.zeros_like(z))
                # a value that a row may not see has no weight there
                out[rows, h], mag[rows, h], lse[rows, h] = w @ v[:, h // g], w @ v[:, h // g].abs(), l
        t0 += n
    return out, mag, lse, big


def check(m, got, lse, want):
    """Every weight may be rounded to the cache's type once and the result once (half a
    step each); products, exponentials and sums in 32 bits are off by a few 2^-24 of the
    largest logit (in the exponent, so relative to the result) and 2^-22 for the
    exponential; 2^-12 covers them at the logits used here."""
    out, mag, ref, big = want
    half = torch.finfo(m.dt).eps / 2
    assert big < 200
    tol = half * (mag + out.abs()) + 2.0 ** -12 * mag + torch.finfo(m.dt).tiny
    err = (got.double() - out).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())
    empty = ref == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert bool((got[empty] == 0).all())
    e = (lse.double() - ref)[~empty].abs()
    assert e.numel() == 0 or float(e.max()) <= 2.0 ** -18 * (big + 16), float(e.max())


HEADS = [(4, 4), (8, 2), (12, 4), (16, 1), (32, 8)]
DECODE_LENS = [[1], [2, 0, 1], [15, 16, 17], [127, 128, 129, 5], [255, 256, 257], [1000, 3, 4099],
               [9001], [33] * 40]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", DECODE_LENS, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_lengths(d, dtype, lens):
    i = DECODE_LENS.index(lens)
    Hq, Hk = HEADS[(i + d // 64) % len(HEADS)]
    page = [16, 128, 48, 64, 256][(i + d) % 5]
    m = Made([(1, kv) for kv in lens], Hk, d, page, dtype, seed=i)
    q = m.normal(len(lens), Hq, d) * 2
    out, lse = up.decode_attend(q, m.cache)
    lo = torch.zeros(len(lens), dtype=torch.long, device="cuda")
    assert up.get_device_error() == 0  # a sequence without a cached token has an empty row
    check(m, out, lse, oracle(m, q, lo, m.kv_lens.long(), d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", HEADS + [(5, 1), (14, 2)])
@pytest.mark.parametrize("kind", ["cap", "bias", "window", "all"])
def test_decode_logits(kind, Hq, Hk):
    lens = [700, 1, 130, 2500]
    m = Made([(1, kv) for kv in lens], Hk, 128, 32, "bf16", seed=Hq)
    q = m.normal(4, Hq, 128) * 4
    kw, lo = {}, torch.zeros(4, dtype=torch.int32, device="cuda")
    if kind in ("cap", "all"):
        kw["softcap"] = 15.0
    if kind in ("bias", "all"):
        kw["slopes"] = torch.linspace(0.002, 0.02, Hq, device="cuda")
        kw["q_pos"] = torch.tensor([1500, 3, 200, 4000], dtype=torch.int32, device="cuda")
    if kind in ("window", "all"):  # negative, past the end (empty), inside, at the last slot
        lo = torch.tensor([-5, 1, 77, 2499], dtype=torch.int32, device="cuda")
        # what the query does not see has no effect
        at = m.table[2].long()[torch.arange(77, device="cuda") // 32]
        m.kp[at, :, torch.arange(77, device="cuda") % 32] = math.nan
        m.vp[at, :, torch.arange(77, device="cuda") % 32] = math.inf
        kw["kv_start"] = lo
    out, lse = up.decode_attend(q, m.cache, scale=0.07, **kw)
    assert up.get_device_error() == 0
    kw.pop("kv_start", None)
    m.kp.nan_to_num_(0.0), m.vp.nan_to_num_(0.0, 0.0, 0.0)
    check(m, out, lse, oracle(m, q, lo.long(), m.kv_lens.long(), 0.07, **kw))


ATTEND = [  # (new, cached) of every sequence
    [(1, 1)], [(3, 3)], [(64, 64)], [(129, 129)], [(1, 300), (0, 40), (7, 7)], [(200, 777)],
    [(33, 128), (31, 129), (128, 127 + 128)], [(257, 513), (2, 2), (0, 0), (5, 1025)], [(600, 600)],
    [(40, 5000)]]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", ATTEND, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_lengths(d, dtype, lens):
    i = ATTEND.index(lens)
    Hq, Hk = HEADS[(i + d // 64) % len(HEADS)]
    m = Made(lens, Hk, d, [16, 128, 48, 64, 256, 384][(i + d) % 6], dtype, seed=i)
    q = m.normal(m.T, Hq, d) * 2
    out, lse = up.attend_paged(q, m.cu, m.cache)
    assert up.get_device_error() == 0
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).cuda()
    check(m, out, lse, oracle(m, q, torch.zeros_like(own), own + 1, d ** -0.5))


def masks(kind, lens, seed):
    g = torch.Generator().manual_seed(seed)
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in lens])
    end = torch.cat([torch.full((n,), kv) for n, kv in lens])
    lo, hi = torch.zeros_like(own), own + 1
    if kind == "window":
        lo = own - 49
    elif kind == "docs":
        lo = own // 150 * 150
    elif kind == "prefix":
        hi = torch.maximum(hi, torch.full_like(hi, 333))
    elif kind == "ragged":  # any ranges: empty, reversed, outside, one slot
        lo = (torch.rand(own.shape, generator=g) * (end + 80)).long() - 40
        hi = lo + (torch.rand(own.shape, generator=g) * 400).long() - 60
        lo[::7], hi[::7] = -(1 << 31), (1 << 31) - 1
    return torch.stack([lo, hi], 1).to(torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d,dtype", [(8, 2, 64, "bf16"), (32, 8, 128, "bf16"), (12, 4, 128, "fp16"),
                                           (16, 1, 256, "fp16"), (3, 3, 256, "bf16"), (5, 1, 64, "fp16")])
@pytest.mark.parametrize("kind", ["window", "docs", "prefix", "ragged"])
@pytest.mark.parametrize("logits", ["plain", "cap", "bias", "both"])
def test_attend_masks(logits, kind, Hq, Hk, d, dtype):
    lens = [(150, 700), (1, 1), (70, 70), (300, 1100)]
    m = Made(lens, Hk, d, 64 if d < 256 else 16, dtype, seed=3)
    q = m.normal(m.T, Hq, d) * 3
    vis = masks(kind, lens, 5)
    kw = {}
    if logits in ("cap", "both"):
        kw["softcap"] = 12.0
    if logits in ("bias", "both"):
        kw["slopes"] = torch.linspace(0.03, 0.001, Hq, device="cuda")
        kw["q_pos"] = torch.randint(0, 2000, (m.T,), generator=m.g, device="cuda", dtype=torch.int32)
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, **kw)
    assert up.get_device_error() == 0
    check(m, out, lse, oracle(m, q, vis[:, 0].long(), vis[:, 1].long(), d ** -0.5, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_growing_logits(d):
    """Keys whose logits grow along the sequence: the running maximum moves at every tile."""
    m = Made([(100, 900)], 2, d, 128, "bf16", seed=1)
    ramp = torch.linspace(0.0, 60.0, 900, device="cuda")
    u = torch.ones(d, device="cuda") * d ** -0.5
    i = torch.arange(900, device="cuda")
    m.kp[m.table[0].long()[i // 128], :, i % 128] += (ramp[:, None] * u).to(m.dt)[:, None]
    q = (m.normal(100, 8, d).float() * 0.3 + u * d ** 0.5).to(m.dt)
    out, lse = up.attend_paged(q, m.cu, m.cache)
    own = torch.arange(800, 900, device="cuda")
    check(m, out, lse, oracle(m, q, torch.zeros_like(own), own + 1, d ** -0.5))
    o1, l1 = up.decode_attend(q[-1:].contiguous(), m.cache)
    check(m, o1, l1, tuple(x[-1:] if torch.is_tensor(x) else x
                           for x in oracle(m, q, torch.zeros_like(own), own + 1, d ** -0.5)))


@pytest.mark.gpu
def test_decode_equals_attend_of_one():
    m = Made([(1, kv) for kv in (5, 300, 4097)], 8, 128, 64, "bf16", seed=2)
    q = m.normal(3, 32, 128)
    a, la = up.attend_paged(q, m.cu, m.cache)
    b, lb = up.decode_attend(q, m.cache)
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -6 and torch.allclose(la, lb, atol=1e-4)


@pytest.mark.gpu
def test_bad_pages_and_lengths():
    """A page outside the pool reads as zeros; a length that cannot be leaves its sequence out."""
    m = Made([(4, 200), (4, 100), (4, 90)], 2, 64, 32, "bf16", seed=4, poison=False)
    q = m.normal(m.T, 8, 64)
    m.table[0, 1] = m.kp.shape[0]
    m.table[0, 2] = -7
    m.kv_lens[1] = 3            # fewer than its new tokens
    m.kv_lens[2] = 10 ** 6      # more than its pages
    out, lse = up.attend_paged(q, m.cu, m.cache)
    assert up.get_device_error() == 0x48
    z = Made([(4, 200), (4, 100), (4, 90)], 2, 64, 32, "bf16", seed=4, poison=False)
    z.table[0, 1:3] = z.table[0, 0]
    z.kp = torch.cat([z.kp, torch.zeros_like(z.kp[:1])])
    z.vp = torch.cat([z.vp, torch.zeros_like(z.vp[:1])])
    z.table[0, 1:3] = z.kp.shape[0] - 1
    z.pp = torch.cat([z.pp, torch.zeros_like(z.pp[:1])])
    own = torch.arange(196, 200, device="cuda").repeat(3)
    lo, hi = torch.zeros_like(own), own + 1
    hi[4:] = 0
    check(m, out, lse, oracle(z, q, lo, hi, 64 ** -0.5))
    out, lse = up.decode_attend(q[:3].contiguous(), m.cache)
    assert up.get_device_error() == 0x48
    z.lens = [(1, kv) for _, kv in z.lens]
    want = oracle(z, q[:3], torch.zeros(3, device="cuda"), torch.tensor([200, 3, 0], device="cuda"), 64 ** -0.5)
    check(m, out, lse, want)
    k = m.normal(m.T, 2, 64)
    before = m.kp.clone()
    m.table[0, 6] = 1 << 20
    up.append_kv(None, k, k, torch.zeros(m.T, dtype=torch.int32, device="cuda"), m.cu, m.cache, None)
    assert up.get_device_error() == 0x48
    assert torch.equal(m.kp, before)


@pytest.mark.gpu
def test_bad_cu_seqlens_stay_in_bounds():
    m = Made([(4, 200), (4, 100)], 2, 64, 32, "bf16", seed=4)
    q = m.normal(8, 8, 64)
    k = m.normal(8, 2, 64)
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    for cu in ([0, 4, 6], [3, 5, 8], [0, 9, 8], [-4, 4, 8], [0, 0, 0], [0, 4, 1 << 30]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        up.attend_paged(q, cu, m.cache)
        assert up.get_device_error() != 0
        up.append_kv(None, k, k, pos, cu, m.cache, None)
        up.get_device_error()


def rope(x, pos, inv_freq, axes, interleaved):
    half = inv_freq.numel()
    x = x.double().clone()
    pos = pos.view(-1, x.shape[0]).double()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = (pos[0 if axes is None else int(axes[i])] * inv_freq[i].double())[:, None]
        x[..., a], x[..., b] = x[..., a] * t.cos() - x[..., b] * t.sin(), x[..., b] * t.cos() + x[..., a] * t.sin()
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 5000), (1, 16), (1, 17)], [(37, 100), (0, 50), (300, 300)],
                                  [(2500, 2600)]], ids=str)
@pytest.mark.parametrize("Hq,Hk,d,dtype,rot,inter,A", [
    (8, 2, 64, "bf16", 64, False, 1), (32, 8, 128, "bf16", 128, False, 3), (16, 2, 256, "fp16", 64, True, 1),
    (4, 4, 128, "fp16", 32, False, 2), (12, 4, 64, "bf16", 16, True, 3), (0, 3, 256, "bf16", 256, True, 1),
    (8, 1, 128, "bf16", 0, False, 1)])
def test_append(Hq, Hk, d, dtype, rot, inter, A, lens):
    m = Made(lens, Hk, d, [16, 64, 48][len(lens) % 3], dtype, seed=6, poison=False)
    x = m.normal(m.T, (max(Hq, 1) + 2 * Hk) * d)
    q = x[:, :Hq * d].view(m.T, Hq, d) if Hq else None
    k = x[:, -2 * Hk * d:-Hk * d].view(m.T, Hk, d)
    v = x[:, -Hk * d:].view(m.T, Hk, d)
    pos = torch.randint(-5, 1 << 22, (A, m.T), generator=m.g, device="cuda", dtype=torch.int32)
    f = (10000.0 ** -(torch.arange(0, rot, 2, device="cuda") / max(rot, 1))).float() if rot else None
    axes = torch.randint(0, A, (rot // 2,), generator=m.g, device="cuda", dtype=torch.int32) if A > 1 else None
    kp, vp, pp = m.kp.clone(), m.vp.clone(), m.pp.clone()
    got = up.append_kv(q, k, v, pos if A > 1 else pos[0], m.cu, m.cache, f, axes=axes, interleaved=inter)
    assert up.get_device_error() == 0
    f = torch.zeros(0, device="cuda") if f is None else f
    # one rounding of the result; the angle is off by at most 2^-22 radians (its value in
    # 32 bits) and the two products by 2^-22 of the pair's size
    half = torch.finfo(m.dt).eps / 2

    def near(y, src):
        want = rope(src, pos, f, axes, inter)
        size = src.double().abs().amax(-1, keepdim=True)
        assert bool(((y.double() - want).abs() <= half * want.abs() + 2.0 ** -20 * size).all())
        assert torch.equal(y[..., 2 * f.numel():], src[..., 2 * f.numel():])

    if Hq:
        near(got, q)
    else:
        assert got is None
    t0 = 0
    for s, (n, kv) in enumerate(lens):
        i = torch.arange(kv - n, kv, device="cuda")
        at, row = m.table[s].long()[i // m.page], i % m.page
        if n:
            ks = torch.zeros_like(k)
            ks[t0:t0 + n] = m.kp[at, :, row]
            want = rope(k, pos, f, axes, inter)[t0:t0 + n]
            size = k[t0:t0 + n].double().abs().amax(-1, keepdim=True)
            assert bool(((m.kp[at, :, row].double() - want).abs() <= half * want.abs() + 2.0 ** -20 * size).all())
            assert torch.equal(m.vp[at, :, row], v[t0:t0 + n])
            assert torch.equal(m.pp[at, row], pos[0, t0:t0 + n])
        kp[at, :, row], vp[at, :, row], pp[at, row] = m.kp[at, :, row], m.vp[at, :, row], m.pp[at, row]
        t0 += n
    # nothing else was written
    assert torch.equal(kp, m.kp) and torch.equal(vp, m.vp) and torch.equal(pp, m.pp)
    if Hq:  # in place
        qc = q.contiguous()
        assert up.append_kv(qc, k, v, pos if A > 1 else pos[0], m.cu, m.cache, f if rot else None, axes=axes,
                            interleaved=inter, q_out=qc) is qc
        assert torch.equal(qc, got)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^32."""
    page, Hk, d = 256, 8, 128
    n = (1 << 32) // (page * Hk * d) + 5
    kp = torch.empty(n, Hk, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    m = Made([(3, 500)], Hk, d, page, "bf16", seed=8, poison=False)
    far = torch.tensor([[n - 1, n - 3, -1]], dtype=torch.int32, device="cuda")
    pp = torch.zeros(n, page, dtype=torch.int32, device="cuda")
    kp[far[0, :2].long()], vp[far[0, :2].long()] = m.kp[m.table[0, :2].long()], m.vp[m.table[0, :2].long()]
    cache = up.PagedKV(kp, vp, far, m.kv_lens, pp)
    k, v = m.normal(3, Hk, d), m.normal(3, Hk, d)
    pos = torch.tensor([7, 8, 9], dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0] * 64, device="cuda")
    for c in (cache, m.cache):
        up.append_kv(None, k, v, pos, m.cu, c, f)
    for a, b in ((kp, m.kp), (vp, m.vp)):
        assert torch.equal(a[far[0, :2].long()], b[m.table[0, :2].long()])
    q = m.normal(3, 32, d)
    for x, y in zip(up.attend_paged(q, m.cu, cache), up.attend_paged(q, m.cu, m.cache)):
        assert torch.equal(x, y)
    q1 = q[:1].contiguous()
    for x, y in zip(up.decode_attend(q1, cache), up.decode_attend(q1, m.cache)):
        assert torch.equal(x, y)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_repeat_graph_and_side_stream():
    """The same bits again, from a captured graph and from another stream."""
    m = Made([(1, 3000), (1, 77)], 8, 128, 64, "bf16", seed=9)
    c = Made([(130, 2000), (64, 64)], 8, 128, 64, "bf16", seed=10)
    q, qc = m.normal(2, 32, 128), c.normal(c.T, 32, 128)
    k, v = m.normal(2, 8, 128), m.normal(2, 8, 128)
    pos = torch.tensor([2999, 76], dtype=torch.int32, device="cuda")
    f = 10000.0 ** -(torch.arange(0, 128, 2, device="cuda") / 128)

    def step(stream=None):
        y = up.append_kv(q, k, v, pos, m.cu, m.cache, f, stream=stream)
        return (y,) + up.decode_attend(y, m.cache, stream=stream) + up.attend_paged(qc, c.cu, c.cache, stream=stream)

    first = [x.clone() for x in step()]
    for x, y in zip(first, step()):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    side.synchronize()
    for x, y in zip(first, other):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for x in held:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(first, held):
        assert torch.equal(x, y)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_python_refusals_on_the_gpu():
    m = Made([(2, 20)], 2, 64, 16, "bf16")
    q, k = m.normal(2, 8, 64), m.normal(2, 2, 64)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        up.attend_paged(q.half(), m.cu, m.cache)
    with pytest.raises(ValueError):
        up.attend_paged(q.transpose(0, 1), m.cu, m.cache)
    with pytest.raises(ValueError):
        up.decode_attend(q, m.cache)  # two tokens, one sequence
    with pytest.raises(ValueError):
        up.attend_paged(q, m.cu, m.cache, slopes=torch.zeros(8, device="cuda"))
    with pytest.raises(up.UpError):
        up.attend_paged(m.normal(2, 7, 64), m.cu, m.cache)
    with pytest.raises(up.UpError):
        up.attend_paged(q, m.cu, m.cache, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        up.append_kv(q, k, k, pos[:1], m.cu, m.cache, None)
    with pytest.raises(ValueError):
        up.append_kv(q, k, k.transpose(1, 2).contiguous().transpose(1, 2), pos, m.cu, m.cache, None)
    with pytest.raises(up.UpError):
        up.append_kv(q, k, k, pos, m.cu, m.cache, torch.ones(4, device="cuda"))
    assert up.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [2.0, 30.0, 50.0, 400.0])
@pytest.mark.parametrize("d", [64, 256])
def test_caps_from_tight_to_wide(d, softcap):
    """The capped logit's short series, long series and general form."""
    m = Made([(70, 400), (3, 900)], 2, d, 64, "fp16", seed=11)
    q = m.normal(m.T, 8, d) * 5
    out, lse = up.attend_paged(q, m.cu, m.cache, softcap=softcap)
    own = torch.cat([torch.arange(330, 400), torch.arange(897, 900)]).cuda()
    zero = torch.zeros_like(own)
    want = oracle(m, q, zero, own + 1, d ** -0.5, softcap=softcap)
    check(m, out, lse, want)
    one = Made([(1, 400), (1, 900)], 2, d, 64, "fp16", seed=12)
    q = one.normal(2, 8, d) * 5
    out, lse = up.decode_attend(q, one.cache, softcap=softcap)
    check(one, out, lse, oracle(one, q, zero[:2], one.kv_lens.long(), d ** -0.5, softcap=softcap))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.02])
def test_any_scale(scale):
    m = Made([(140, 500)], 2, 128, 32, "bf16", seed=13)
    q = m.normal(140, 8, 128)
    own = torch.arange(360, 500).cuda()
    out, lse = up.attend_paged(q, m.cu, m.cache, scale=scale)
    check(m, out, lse, oracle(m, q, torch.zeros_like(own), own + 1, scale))
    out, lse = up.decode_attend(q[-1:].contiguous(), m.cache, scale=scale)
    check(m, out, lse, tuple(x[-1:] if torch.is_tensor(x) else x
                             for x in oracle(m, q, torch.zeros_like(own), own + 1, scale)))


@pytest.mark.gpu
def test_more_sequences_than_a_block_has_threads():
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 4, (1500,), generator=g).tolist()
    lens = [(a, a + b) for a, b in zip(n, torch.randint(0, 40, (1500,), generator=g).tolist())]
    m = Made(lens, 2, 64, 16, "bf16", seed=14)
    q = m.normal(m.T, 4, 64) * 2
    out, lse = up.attend_paged(q, m.cu, m.cache)
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).cuda()
    check(m, out, lse, oracle(m, q, torch.zeros_like(own), own + 1, 0.125))
    q = m.normal(1500, 4, 64) * 2
    out, lse = up.decode_attend(q, m.cache)
    assert up.get_device_error() == 0
    m.lens = [(1, kv) for _, kv in lens]
    check(m, out, lse, oracle(m, q, torch.zeros(1500, dtype=torch.long, device="cuda"), m.kv_lens.long(), 0.125))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d", [(32, 8, 128), (16, 2, 256), (24, 3, 64)])
def test_units_cut_by_shares(Hq, Hk, d):
    """Enough work for every SM: whole units, units cut in two and units without a token."""
    lens = [(700, 3000), (1, 20), (0, 64), (33, 2100), (1200, 1200)]
    m = Made(lens, Hk, d, 128, "bf16", seed=15)
    q = m.normal(m.T, Hq, d) * 2
    vis = masks("ragged", lens, 7)
    vis[300:420] = 0  # units that see nothing
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).cuda()
    for visible in (None, vis):
        out, lse = up.attend_paged(q, m.cu, m.cache, visible=visible)
        lo, hi = (torch.zeros_like(own), own + 1) if visible is None else vis.long().unbind(1)
        check(m, out, lse, oracle(m, q, lo, hi, d ** -0.5))
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_no_log_sum_asked_for():
    m = Made([(5, 300), (90, 90)], 2, 64, 32, "bf16", seed=16)
    q = m.normal(m.T, 8, 64)
    want, _ = up.attend_paged(q, m.cu, m.cache)
    L, out = up.lib(), torch.zeros_like(q)
    ws = torch.empty(up.attend_paged_workspace(m.T, 2, 8, 2, 64), dtype=torch.uint8, device="cuda")
    lg = ctypes.byref(_CLogits(0.125, 0.0, None, None))
    stream = torch.cuda.current_stream().cuda_stream
    assert L.up_attend_paged(q.data_ptr(), m.cu.data_ptr(), m.T, 8, m.cache.ref, lg, None, out.data_ptr(),
                             None, ws.data_ptr(), ws.numel(), stream) == 0
    assert torch.equal(out, want)
    want, _ = up.decode_attend(q[:2].contiguous(), m.cache)
    assert L.up_decode_attend(q.data_ptr(), 8, m.cache.ref, lg, None, out.data_ptr(), None, ws.data_ptr(),
                              ws.numel(), stream) == 0
    assert torch.equal(out[:2], want)


@pytest.mark.gpu
def test_expired_wait_stops_attention_cleanly():
    """A wait bound of a few cycles: the kernel gives up, reports the timeout and leaves
    the context usable."""
    m = Made([(600, 2000)], 8, 128, 64, "bf16", seed=17)
    q = m.normal(600, 32, 128)
    want = [x.clone() for x in up.attend_paged(q, m.cu, m.cache)]
    up.set_wait_limit(64)
    try:
        up.attend_paged(q, m.cu, m.cache)
        assert up.get_device_error() & 0x4
    finally:
        up.set_wait_limit(0)
    for x, y in zip(want, up.attend_paged(q, m.cu, m.cache)):
        assert torch.equal(x, y)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_example_runs_the_operators_together():
    """Prefill with dropped tokens and captured decode steps; twice the same tokens."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "sparse_prefill_decode.py")
    spec = importlib.util.spec_from_file_location("sparse_prefill_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    a = ex.main(["--prompt", "700", "333", "--steps", "6"])
    b = ex.main(["--prompt", "700", "333", "--steps", "6"])
    assert a == b and len(a) == 2 and all(len(t) == 6 for t in a)


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 48)])
def test_what_nobody_sees_may_be_anything(d, page, bias):
    """A window's old pages may be gone from the table and hold NaN, and so may the slots
    around the ranges that queries see."""
    lens = [(40, 700), (90, 1500)]
    m = Made(lens, 2, d, page, "bf16", seed=18)
    q = m.normal(m.T, 8, d) * 2
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).cuda()
    lo, hi = own - 333, own - 5
    vis = torch.stack([lo, hi], 1).to(torch.int32)
    kw = {}
    if bias:
        kw = dict(slopes=torch.linspace(0.01, 0.001, 8, device="cuda"),
                  q_pos=torch.cat([m.tokens(s, m.pp)[kv - n:] for s, (n, kv) in enumerate(lens)]).contiguous())
    want = oracle(m, q, lo.clamp(min=0), hi, d ** -0.5, **kw)
    t0 = 0
    for s, (n, kv) in enumerate(lens):
        first, end = int(lo[t0]), int(hi[t0 + n - 1])
        i = torch.cat([torch.arange(first), torch.arange(end, kv)]).cuda()
        at = m.table[s].long()[i // page]
        m.kp[at, :, i % page] = math.nan
        m.vp[at, :, i % page] = math.nan
        m.table[s, :first // page] = -1
        t0 += n
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, **kw)
    assert up.get_device_error() == 0
    check(m, out, lse, want)
    start = torch.tensor([700 - 300, 1500 - 300], dtype=torch.int32, device="cuda")
    m2 = Made([(1, 700), (1, 1500)], 2, d, page, "bf16", seed=18)
    q = m2.normal(2, 8, d)
    want = oracle(m2, q, start.long(), m2.kv_lens.long(), d ** -0.5)
    for s in range(2):
        m2.table[s, :int(start[s]) // page] = 1 << 30
    out, lse = up.decode_attend(q, m2.cache, kv_start=start)
    assert up.get_device_error() == 0
    check(m2, out, lse, want)


@pytest.mark.gpu
def test_a_cache_does_not_change_its_tensors():
    m = Made([(1, 20)], 2, 64, 16, "bf16")
    with pytest.raises(AttributeError):
        m.cache.kv_lens = m.kv_lens + 1
