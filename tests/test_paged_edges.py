"""The paged-cache operators at the edges of their ranges: logits of thousands, light weights,
ranges with gaps, tight caps, what must not reach a result, and a cache's identity."""
import copy
import math

import pytest
import torch

import block_sparse_long_up_gb300 as up
from block_sparse_long_up_gb300 import paged
from test_paged import Made, oracle


def check_at(m, got, lse, want, content=32.0, floor=0.0):
    """The result against 64 bits where logits are far from zero.  Each weight and the
    result are rounded to the cache's type (half a step each).  A logit of a key whose weight
    counts (2^-40 of the row's largest and more) lies within 28 of the largest one, which
    lies within the log of the keys' number of the log-sum; before its bias it is
    `content` at most.  The tensor cores add d / 16 times with 23 bits kept, the rest is a few
    roundings of 2^-24: 2^-18 of the logit's size in all, in the exponent.  `floor`: what
    the type's smallest steps leave of weights that are far below the largest."""
    out, mag, ref, _ = want
    assert torch.isfinite(got).all()
    empty = ref == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    near = torch.where(empty, torch.zeros_like(ref), ref).abs() + 28 + math.log(max(kv for _, kv in m.lens) + 1) + content
    half = torch.finfo(m.dt).eps / 2
    tol = half * (mag + out.abs()) + (2.0 ** -12 + 2.0 ** -18 * near[..., None]) * mag + floor + torch.finfo(m.dt).tiny
    err = (got.double() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    e = ((lse.double() - ref).abs() / (2.0 ** -18 * (near + 16)))[~empty]
    assert e.numel() == 0 or float(e.max()) <= 1.0, float(e.max())


# ------------------------------------------------------------------ logits far from zero

@pytest.mark.gpu
@pytest.mark.parametrize("steepest", [0.125, 0.5, 0.7])
@pytest.mark.parametrize("n,kv", [(40, 16384), (512, 16384), (3, 131072)])
@pytest.mark.parametrize("d,dtype", [(256, "fp16"), (256, "bf16"), (128, "fp16")])
def test_steep_biases_over_long_caches(d, dtype, n, kv, steepest):
    """Parts of a cut unit hold only keys whose biased logits are tens of thousands below the row's."""
    m = Made([(n, kv)], 2, d, 64, dtype, seed=n)
    q = m.normal(n, 16, d) * 2
    kw = dict(slopes=torch.linspace(steepest, steepest / 8, 16, device="cuda"),
              q_pos=m.tokens(0, m.pp)[kv - n:].contiguous())
    own = torch.arange(kv - n, kv, device="cuda")
    out, lse = up.attend_paged(q, m.cu, m.cache, **kw)
    check_at(m, out, lse, oracle(m, q, torch.zeros_like(own), own + 1, d ** -0.5, **kw))
    # rows that see only far keys
    vis = torch.stack([own * 0 + 5, own * 0 + 205], 1).to(torch.int32)
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, **kw)
    check_at(m, out, lse, oracle(m, q, vis[:, 0].long(), vis[:, 1].long(), d ** -0.5, **kw))
    one = dict(kw, q_pos=kw["q_pos"][-1:].contiguous())
    m.lens = [(1, kv)]
    out, lse = up.decode_attend(q[-1:].contiguous(), m.cache, **one)
    check_at(m, out, lse, oracle(m, q[-1:], own[-1:] * 0, own[-1:] + 1, d ** -0.5, **one))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_logits_of_thousands(d, dtype):
    """Logits of 6000 and -6000 with differences of a few, without a bias."""
    m = Made([(30, 700), (200, 1400)], 2, d, 64, dtype, seed=21)
    for s in range(2):
        i = torch.arange(m.lens[s][1], device="cuda")
        at, row = m.table[s].long()[i // 64], i % 64
        m.kp[at, :, row] = (15 + 0.1 * m.kp[at, :, row].float()).to(m.dt)
    size = torch.linspace(-25, 25, 16, device="cuda") * (256 / d) ** 0.5
    q = size.to(m.dt)[None, :, None].expand(m.T, 16, d).contiguous()
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in m.lens]).cuda()
    out, lse = up.attend_paged(q, m.cu, m.cache)
    check_at(m, out, lse, oracle(m, q, torch.zeros_like(own), own + 1, d ** -0.5))
    m.lens = [(1, 700), (1, 1400)]
    out, lse = up.decode_attend(q[:2].contiguous(), m.cache)
    check_at(m, out, lse, oracle(m, q[:2], own[:2] * 0, m.kv_lens.long(), d ** -0.5))


# ------------------------------------------------------------------ ranges with gaps

def gapped(kind, n, kv, seed):
    """First visible slot and end for n tokens: together they leave gaps."""
    t = torch.arange(n)
    if kind == "pair":        # neighbours see far-apart ranges
        lo = torch.where(t % 2 == 0, 0, kv // 2)
        hi = lo + 10
    elif kind == "halves":    # a gap between the first tokens and the last ones, most of them in units of their own
        lo = torch.where(t < n // 2, 3, 100)
        hi = torch.where(t < n // 2, 13, 110)
    elif kind == "islands":   # three islands across many key tiles, a token without a range between
        lo = torch.tensor([17, kv // 3, kv - 90])[t // 5 % 3] + t % 4
        hi = torch.where(t % 5 == 4, 0, lo + 40)
    else:                     # short ranges anywhere
        g = torch.Generator().manual_seed(seed)
        lo = torch.randint(-20, kv, (n,), generator=g)
        hi = lo + torch.randint(0, 30, (n,), generator=g)
    return lo, hi


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["pair", "halves", "islands", "any"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,page", [(8, 2, 64, 16), (8, 2, 128, 64), (16, 2, 256, 48), (2, 2, 128, 256), (12, 4, 64, 384)])
def test_gaps_between_ranges_may_hold_anything(Hq, Hk, d, page, bias, kind):
    """Slots that no token sees hold NaN, pages of such slots are gone from the table."""
    lens = [(40, 700), (1, 5), (300, 1500)]
    m = Made(lens, Hk, d, page, "bf16", seed=23)
    q = m.normal(m.T, Hq, d) * 2
    lo, hi = (torch.cat(x).cuda() for x in zip(*(gapped(kind, n, kv, 3) for n, kv in lens)))
    kw = {}
    if bias:
        kw = dict(slopes=torch.linspace(0.01, 0.001, Hq, device="cuda"),
                  q_pos=torch.cat([m.tokens(s, m.pp)[kv - n:] for s, (n, kv) in enumerate(lens)]).contiguous())
    want = oracle(m, q, lo, hi, d ** -0.5, **kw)
    t0 = 0
    for s, (n, kv) in enumerate(lens):
        i = torch.arange(-(-kv // page) * page, device="cuda")
        seen = ((i >= lo[t0:t0 + n, None]) & (i < hi[t0:t0 + n, None].clamp(max=kv))).any(0)
        at, row = m.table[s].long()[i // page], i % page
        m.kp[at[~seen], :, row[~seen]] = math.nan
        m.vp[at[~seen], :, row[~seen]] = math.nan
        m.table[s, :-(-kv // page)].masked_fill_(~seen.view(-1, page).any(1), -1)
        t0 += n
    vis = torch.stack([lo, hi], 1).to(torch.int32)
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, **kw)
    assert up.get_device_error() == 0
    check_at(m, out, lse, want)


# ------------------------------------------------------------------ tight caps

@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e-6, 1e-4, 1e-3, 1.0, 1e30])
@pytest.mark.parametrize("scale", [0.088, 1.0, -0.088, 1e5])
@pytest.mark.parametrize("d", [64, 256])
def test_caps_far_below_the_scale(d, scale, softcap):
    """Queries of zero, queries whose logits are a part of the cap, and ordinary ones."""
    lens = [(130, 400), (3, 900)]
    m = Made(lens, 2, d, 64, "bf16", seed=24)
    size = torch.tensor([0.0, 0.3 * min(softcap, 1.0) / abs(scale) * d ** -0.5, min(1.0, 10 / abs(scale))], device="cuda")
    q = (m.normal(m.T, 8, d).float() * size[torch.arange(m.T, device="cuda") // 40 % 3, None, None]).to(m.dt)
    own = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).cuda()
    out, lse = up.attend_paged(q, m.cu, m.cache, scale=scale, softcap=softcap)
    check_at(m, out, lse, oracle(m, q, own * 0, own + 1, scale, softcap=softcap), content=800.0)
    m.lens = [(1, 400), (1, 900)]
    for t in (0, 45, 90):
        x = q[t:t + 2].contiguous()
        out, lse = up.decode_attend(x, m.cache, scale=scale, softcap=softcap)
        check_at(m, out, lse, oracle(m, x, own[:2] * 0, m.kv_lens.long(), scale, softcap=softcap), content=800.0)


def test_a_scale_is_read_at_every_call():
    """A 0-dim tensor may be the scale or the cap, and may change between calls."""
    for k in range(2):
        x = torch.tensor([0.5, 30.0])
        given = [x[0], x[1]]
        for a, b in ((0.5, 30.0), (0.25, 20.0)):
            x[0], x[1] = a, b
            lg = paged._logits(None, 1, 1, *given, None, None)._obj
            assert (lg.scale, lg.softcap) == (a, b)
    with pytest.raises(TypeError):
        paged._logits(None, 1, 1, "0.5", 0.0, None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [64, 512, 2000])
@pytest.mark.parametrize("below", [12.0, 14.5, 17.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_light_weights_of_fp16_count(d, below, kv):
    """One key carries nearly all the weight and its value is zero, so the output is the others',
    each with a weight of e^-12 to e^-17.  A weight keeps a half step of fp16 down to 2^-21 of
    the reference; below, 2^-32 of it each."""
    m = Made([(3, kv)], 2, d, 64, "fp16", seed=22)
    i = torch.arange(kv, device="cuda")
    at, row = m.table[0].long()[i // 64], i % 64
    m.kp[at, :, row] = 0
    m.kp[at[0], :, 0] = below * d ** -0.5
    m.vp[at, :, row] = (1024 * (m.vp[at, :, row].float().abs().clamp(max=1) + 0.5)).to(m.dt)
    m.vp[at[0], :, 0] = 0
    q = torch.ones(3, 8, d, dtype=m.dt, device="cuda")
    own = torch.arange(kv - 3, kv, device="cuda")
    out, lse = up.attend_paged(q, m.cu, m.cache)
    floor = kv * 2.0 ** -32 * 1536
    check_at(m, out, lse, oracle(m, q, own * 0, own + 1, d ** -0.5), floor=floor)
    m.lens = [(1, kv)]
    out, lse = up.decode_attend(q[:1].contiguous(), m.cache)
    check_at(m, out, lse, oracle(m, q[:1], own[:1] * 0, m.kv_lens.long(), d ** -0.5), floor=floor)


# ------------------------------------------------------------------ what must not reach a result

CAP = dict(softcap=30.0)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d", [(12, 4, 64), (14, 2, 128), (5, 1, 256)])
def test_rows_without_a_token_change_no_bit(Hq, Hk, d):
    """Where the group does not divide 128 a tile ends in rows that hold whatever was there before."""
    m = Made([(100, 600)], Hk, d, 64, "bf16", seed=25)
    q = m.normal(m.T, Hq, d) * 0.5
    before = m.normal(256, 8 * Hk, d)
    cu = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    results = []
    for size in (0.0, 60.0, 0.0, 60.0):
        up.attend_paged((before * size), cu, m.cache, visible=torch.tensor([[0, 600]] * 256, dtype=torch.int32, device="cuda"), **CAP)
        results.append(up.attend_paged(q, m.cu, m.cache, **CAP))
    assert all(same(results[0], r) for r in results[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d", [(8, 2, 64), (32, 8, 128), (16, 2, 256)])
def test_other_sequences_change_no_bit(Hq, Hk, d):
    """A sequence's results do not depend on the queries of the one behind it."""
    m = Made([(37, 300), (50, 400)], Hk, d, 64, "bf16", seed=26)
    q = m.normal(m.T, Hq, d) * 0.5
    loud = q.clone()
    loud[37:] *= 60
    a, b = (up.attend_paged(x, m.cu, m.cache, **CAP) for x in (q, loud))
    assert same([x[:37] for x in a], [x[:37] for x in b])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d", [(8, 2, 64), (32, 8, 128), (16, 2, 256)])
def test_unseen_slots_change_no_bit(Hq, Hk, d):
    """What is stored in a slot that no query sees, whatever its logit would be."""
    m = Made([(60, 700)], Hk, d, 64, "bf16", seed=27, poison=False)
    q = m.normal(m.T, Hq, d) * 0.5
    vis = torch.tensor([[150, 670]] * 60, dtype=torch.int32, device="cuda")
    start = torch.tensor([150], dtype=torch.int32, device="cuda")
    results = []
    for size in (0.0, 60.0, math.inf):
        for s in list(range(150)) + list(range(670, 704)):
            pg = int(m.table[0, s // 64])
            m.kp[pg, :, s % 64], m.vp[pg, :, s % 64] = size, size
        m.kv_lens[0] = 700
        a = up.attend_paged(q, m.cu, m.cache, visible=vis, **CAP)
        m.kv_lens[0] = 670
        results.append(a + up.decode_attend(q[:1].contiguous(), m.cache, kv_start=start, **CAP))
    assert same(results[0], results[1]) and same(results[0], results[2])


# ------------------------------------------------------------------ malformed batches

@pytest.mark.gpu
@pytest.mark.parametrize("cu,covered", [([0, 4, 6], range(6)), ([3, 5, 8], range(3, 8)), ([0, 9, 8], ()),
                                        ([-4, 4, 8], range(4, 8)), ([0, 0, 0], ()), ([0, 4, 1 << 30], range(4))])
@pytest.mark.parametrize("d", [64, 256])
def test_malformed_cu_seqlens(d, cu, covered):
    """Attention gives the rows of an empty mask; the append writes the tokens that lie in a
    range of the batch and nothing else.  Both report it."""
    m = Made([(4, 200), (4, 100)], 2, d, 32, "bf16", seed=29, poison=False)
    q, k, v = m.normal(8, 8, d), m.normal(8, 2, d), m.normal(8, 2, d)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, math.nan), torch.full((8, 8), math.nan, device="cuda")
    up.attend_paged(q, bad, m.cache, out=out, lse=lse)
    assert up.get_device_error() == 0x1
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    want = [x.clone() for x in (m.kp, m.vp, m.pp)]
    pos = torch.arange(100, 108, dtype=torch.int32, device="cuda")
    for t in covered:
        s = 0 if cu[0] <= t < cu[1] else 1
        slot = m.lens[s][1] - (cu[s + 1] - t)
        pg = int(m.table[s, slot // 32])
        want[0][pg, :, slot % 32], want[1][pg, :, slot % 32], want[2][pg, slot % 32] = k[t], v[t], pos[t]
    up.append_kv(None, k, v, pos, bad, m.cache, None)
    assert up.get_device_error() == 0x1
    assert all(torch.equal(x, y) for x, y in zip(want, (m.kp, m.vp, m.pp)))


# ------------------------------------------------------------------ a cache's identity

def test_a_cache_is_no_tuple():
    """No way around the constructor's checks (a replaced field would leave the addresses behind)."""
    assert not issubclass(up.PagedKV, tuple)
    for name in ("_replace", "_make"):
        assert not hasattr(up.PagedKV, name)


@pytest.mark.gpu
def test_copies_of_a_cache_hold_their_own_tensors():
    m = Made([(1, 20), (1, 70)], 2, 64, 16, "bf16", seed=28)
    q = m.normal(2, 8, 64)
    want = up.decode_attend(q, m.cache)
    shallow, deep = copy.copy(m.cache), copy.deepcopy(m.cache)
    assert shallow.k_pages is m.kp and deep.k_pages is not m.kp
    assert torch.equal(deep.kv_lens, m.kv_lens) and torch.equal(deep.pos_pages, m.pp)
    m.kp.zero_(), m.vp.zero_(), m.kv_lens.zero_()
    for x, y in zip(want, up.decode_attend(q, deep)):
        assert torch.equal(x, y)
    assert bool((up.decode_attend(q, shallow)[0] == 0).all())
    for name in ("k_pages", "kv_lens", "ref", "anything"):
        with pytest.raises(AttributeError):
            setattr(m.cache, name, None)
        with pytest.raises(AttributeError):
            delattr(m.cache, name)


# ------------------------------------------------------------------ ranges that hop

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chunks", "falling", "mixed"])
@pytest.mark.parametrize("Hq,Hk,d,page", [(8, 2, 64, 48), (32, 8, 128, 128), (16, 2, 256, 16)])
def test_ranges_that_hop(Hq, Hk, d, page, kind):
    """Ranges in any order that cover all between them, ranges that cover it from the last to the first,
    and a batch in which one sequence has gaps and the others have not; whole and cut units."""
    lens = [(700, 3000), (90, 1500), (333, 333)]
    m = Made(lens, Hk, d, page, "bf16", seed=30)
    q = m.normal(m.T, Hq, d) * 2
    g = torch.Generator().manual_seed(4)
    lo, hi = [], []
    for s, (n, kv) in enumerate(lens):
        size = 30 if kv > 1000 else 7
        chunks = -(-kv // size)
        at = torch.arange(n) % chunks if n >= chunks else torch.arange(n) * chunks // n
        size = size if n >= chunks else -(-kv // n) + size
        at = at * kv // chunks
        at = at.flip(0) if kind == "falling" else at[torch.randperm(n, generator=g)]
        if kind == "mixed" and s == 1:
            at = torch.where(at > kv // 2, at, at // 4)
        lo.append(at), hi.append(at + size + 3)
    lo, hi = torch.cat(lo).cuda(), torch.cat(hi).cuda()
    want = oracle(m, q, lo, hi, d ** -0.5)
    t0, gaps = 0, []
    for s, (n, kv) in enumerate(lens):
        i = torch.arange(-(-kv // page) * page, device="cuda")
        seen = ((i >= lo[t0:t0 + n, None]) & (i < hi[t0:t0 + n, None].clamp(max=kv))).any(0)
        gaps.append(not bool(seen[:kv].all()))
        at, row = m.table[s].long()[i // page], i % page
        m.kp[at[~seen], :, row[~seen]] = math.nan
        m.vp[at[~seen], :, row[~seen]] = math.nan
        m.table[s, :-(-kv // page)].masked_fill_(~seen.view(-1, page).any(1), -1)
        t0 += n
    assert gaps == [False, kind == "mixed", False]
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=torch.stack([lo, hi], 1).to(torch.int32))
    assert up.get_device_error() == 0
    check_at(m, out, lse, want)


# ------------------------------------------------------------------ caches that come from memory

@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 20])
@pytest.mark.parametrize("d,dtype", [(256, "bf16"), (256, "fp16"), (128, "bf16"), (64, "bf16")])
def test_few_tokens_over_a_long_cache_again_and_again(d, dtype, n):
    """Keys and values that are read once, from memory, in pages far apart: copies land late and
    out of order, and the products wait for them."""
    kv = 131072
    m = Made([(n, kv)], 2, d, 64, dtype, seed=31)
    q = m.normal(n, 16, d) * 2
    own = torch.arange(kv - n, kv, device="cuda")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = up.attend_paged(q, m.cu, m.cache)
    check_at(m, *first, oracle(m, q, own * 0, own + 1, d ** -0.5))
    for _ in range(30):
        flush.zero_()
        for x, y in zip(first, up.attend_paged(q, m.cu, m.cache)):
            assert torch.equal(x, y)
    assert up.get_device_error() == 0


def ring_gap(stages, parts, pieces, products, logits):
    """The ring of attention with one row tile a piece: keys a tile ahead of the values, `parts` stages a
    tile.  The keys' issuer knows the products up to step - products to be done, the values' issuer
    the logits up to step - logits, each its own tiles.  The first use of a stage whose use
    before its waiter does not know to be over, or None."""
    ring, step = [], {}
    for p, n in enumerate(pieces):
        for t in range(n):
            step[p, t] = len(step)
        for kind, t in [("k", 0)] + [x for t in range(n) for x in ([("k", t + 1)] if t + 1 < n else []) + [("v", t)]]:
            ring += [(kind, p, t)] * parts
    for i in range(stages, len(ring)):
        (kind, p, t), (was, pp, pt) = ring[i], ring[i - stages]
        behind = 0 if kind == was else products if kind == "k" else logits
        if step[pp, pt] > step[p, t] - behind:
            return ring[i], ring[i - stages]
    return None


@pytest.mark.parametrize("stages,parts", [(8, 1), (4, 1), (5, 2)])  # head_dim 64, 128, 256
def test_waiters_know_the_phase_before(stages, parts):
    """A parity tells a phase only to a waiter that knows the one before to be over.  The issuers wait
    for the products of two steps ago and for the step's logits before their stages."""
    import itertools
    lists = [p for k in (1, 2, 3) for p in itertools.product(range(1, 8), repeat=k)]
    assert all(ring_gap(stages, parts, p, 2, 0) is None for p in lists)
    # stages waited for first: the order that head_dim 256 must not have
    assert (parts == 1) == all(ring_gap(stages, parts, p, 3, 1) is None for p in lists)
