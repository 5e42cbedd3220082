"""Attention of sets of slots: windows with first tokens that stay visible (attend_paged and
decode_attend with sinks) and trees of drafted tokens (attend_tree), against their
definitions in 64 bits, and their refusals."""
import ctypes
import math

import pytest
import torch

import block_sparse_long_up_gb300 as up
from block_sparse_long_up_gb300.paged import _CLogits
from test_paged_edges import check_at
from test_paged import BAD_CACHES, HEADS, L, Made, _cache, check, masks  # noqa: F401 (L is a fixture)


# ------------------------------------------------------------------ refusals (no GPU)

def _attend(L, cache=None, q=256, cu=256, T=10, Hq=8, lg=(0.1, 0.0, None, None), vis=256, sinks=4, out=256,
            lse=256, ws=256, wsb=1 << 40):
    return L.up_attend_sinks(q, cu, T, Hq, cache or _cache(), ctypes.byref(_CLogits(*lg)), vis, sinks, out,
                             lse, ws, wsb, None)


def _decode(L, cache=None, q=256, Hq=8, lg=(0.1, 0.0, None, None), start=256, sinks=4, out=256, lse=256,
            ws=256, wsb=1 << 40):
    return L.up_decode_sinks(q, Hq, cache or _cache(), ctypes.byref(_CLogits(*lg)), start, sinks, out,
                             lse, ws, wsb, None)


def _tree(L, cache=None, q=256, cu=256, parents=256, T=10, Hq=8, lg=(0.1, 0.0, None, None), start=None, sinks=0,
          out=256, lse=256, ws=256, wsb=1 << 40):
    return L.up_attend_tree(q, cu, parents, T, Hq, cache or _cache(), ctypes.byref(_CLogits(*lg)), start, sinks,
                            out, lse, ws, wsb, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, code):  # noqa: F811
    for call in (_attend, _decode, _tree):
        assert call(L, cache=_cache(**bad), Hq=max(1, bad.get("Hk", 4))) == code


def test_refusals(L):  # noqa: F811
    for call in (_attend, _decode, _tree):
        for bad in (dict(q=None), dict(out=None), dict(q=264), dict(out=264), dict(lse=258), dict(Hq=0),
                    dict(Hq=7), dict(lg=(math.nan, 0.0, None, None)), dict(lg=(0.1, -1.0, None, None)),
                    dict(lg=(0.1, 1e-7, None, None)), dict(lg=(0.1, 0.0, 256, None)), dict(sinks=-1),
                    dict(lg=(0.1, 0.0, 256, 256), cache=_cache(pos=None))):
            assert call(L, **bad) == 1, bad
        assert call(L, Hq=64) == 2 and call(L, sinks=4097) == 2 and call(L, sinks=2 ** 31 - 1) == 2
        for bad in (dict(ws=None), dict(ws=272), dict(wsb=0)):
            assert call(L, **bad) == 3, bad
    for call in (_attend, _tree):
        assert call(L, cu=None) == 1 and call(L, T=-1) == 1 and call(L, T=1 << 29) == 1 and call(L, T=0) == 0
    assert _attend(L, vis=260) == 1 and _decode(L, start=258) == 1 and _tree(L, start=258) == 1
    assert _tree(L, parents=None) == 1 and _tree(L, parents=258) == 1
    assert _decode(L, cache=_cache(B=0)) == 0
    plain = up.attend_paged_workspace(10, 2, 8, 2, 64)
    assert _tree(L, wsb=plain) == 3  # a tree's workspace holds its tokens' bits too


def test_workspace_sizes(L):  # noqa: F811
    assert up.attend_tree_workspace(1000, 4, 8, 2, 64) > up.attend_paged_workspace(1000, 4, 8, 2, 64)
    for bad in ((8, 3, 64), (8, 2, 96), (64, 2, 64), (0, 2, 64), (8, 0, 64)):
        assert up.attend_tree_workspace(1000, 4, *bad) == 0
    assert up.attend_tree_workspace(-1, 4, 8, 2, 64) == 0


# ------------------------------------------------------------------ the definitions

def oracle(m, q, seen, scale, softcap=0.0, slopes=None, q_pos=None):
    """test_paged's oracle for any set of slots: seen[s] is bool [n, kv]."""
    T, Hq, d = q.shape
    g, out = Hq // m.Hk, torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    big, t0 = 1.0, 0
    for s, (n, kv) in enumerate(m.lens):
        if n and kv:
            k, v = m.tokens(s, m.kp).double(), m.tokens(s, m.vp).double()
            place, rows, see = m.tokens(s, m.pp).double(), slice(t0, t0 + n), seen[s].cuda()
            k, v = k.nan_to_num(0.0), v.nan_to_num(0.0, 0.0, 0.0)  # poisoned where nobody sees
            some = see.any(1, keepdim=True)
            for h in range(Hq):
                z = q[rows, h].double() @ k[:, h // g].T * scale
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                if slopes is not None:
                    z = z - slopes[h].double() * (q_pos[rows].double()[:, None] - place).abs()
                z = z.masked_fill(~see, -math.inf)
                if bool(see.any()):
                    big = max(big, float(z[see].abs().max()))
                l = torch.logsumexp(z, 1)
                w = torch.where(some, torch.exp(z - l[:, None]), torch.zeros_like(z))
                out[rows, h], mag[rows, h], lse[rows, h] = w @ v[:, h // g], w @ v[:, h // g].abs(), l
        t0 += n
    return out, mag, lse, big


def sink_sets(lens, lo, hi, sinks):
    out, t0 = [], 0
    for n, kv in lens:
        i = torch.arange(kv)
        a, b = lo[t0:t0 + n, None].long().cpu(), hi[t0:t0 + n, None].long().cpu().clamp(max=kv)
        out.append((i < b) & ((i >= a) | (i < sinks)))
        t0 += n
    return out


def tree_sets(lens, parents, start=None, sinks=0):
    out, t0 = [], 0
    for n, kv in lens:
        past, i = kv - n, torch.arange(kv)
        see = torch.zeros(n, kv, dtype=torch.bool)
        for t in range(n):
            lo = 0 if start is None else int(start[t0 + t])
            see[t, :past] = ((i >= lo) | (i < sinks))[:past]
            j = t
            while j >= 0:
                see[t, past + j] = True
                j = int(parents[t0 + j])
        out.append(see)
        t0 += n
    return out


def grow(lens, seed, kind="bushy"):
    """Parents of every sequence's drafted tokens."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, _ in lens:
        for j in range(n):
            u = float(torch.rand(1, generator=g))
            out.append({"bushy": int(j * u ** 0.5) if j and u > 0.1 else -1, "chain": j - 1, "star": -1,
                        "near": max(-1, j - 1 - int(3 * u))}[kind])
    return torch.tensor(out, dtype=torch.int32).clamp(min=-1)


def poison(m, seen):
    """NaN and infinities in the slots that no query sees; pages without a seen slot leave the table."""
    for s, (n, kv) in enumerate(m.lens):
        if not kv:
            continue
        gone = ~seen[s].any(0).cuda() if n else torch.ones(kv, dtype=torch.bool, device="cuda")
        i = torch.arange(kv, device="cuda")[gone]
        at = m.table[s].long()[i // m.page]
        m.kp[at, :, i % m.page] = math.nan
        m.vp[at, :, i % m.page] = torch.where(i % 2 == 0, math.nan, math.inf)[:, None, None].to(m.dt)
        m.pp[at, i % m.page] = -2 ** 31
        pages = torch.nn.functional.pad(~gone, (0, -kv % m.page)).view(-1, m.page).any(1)
        m.table[s, :pages.numel()][~pages] = -1 - s


def held(m):
    """A cache like m before its poisoning (the oracle's)."""
    import copy
    c = copy.copy(m)
    c.kp, c.vp, c.pp, c.table = m.kp.clone(), m.vp.clone(), m.pp.clone(), m.table.clone()
    return c


def logits_of(kind, m, Hq, own_pos=None):
    kw = {}
    if kind in ("cap", "both"):
        kw["softcap"] = 12.0
    if kind in ("bias", "both"):
        kw["slopes"] = torch.linspace(0.03, 0.001, Hq, device="cuda")
        kw["q_pos"] = torch.randint(0, 2000, (m.T,), generator=m.g, device="cuda", dtype=torch.int32)
    return kw


# ------------------------------------------------------------------ sinks

@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d,dtype", [(8, 2, 64, "bf16"), (32, 8, 128, "bf16"), (12, 4, 128, "fp16"),
                                           (16, 1, 256, "fp16"), (3, 3, 256, "bf16"), (5, 1, 64, "fp16")])
@pytest.mark.parametrize("kind,sinks", [("window", 1), ("window", 4), ("window", 130), ("window", 4096), ("docs", 7),
                                        ("ragged", 33), ("prefix", 200)])
@pytest.mark.parametrize("logits", ["plain", "cap", "bias", "both"])
def test_chunks_with_sinks(logits, kind, sinks, Hq, Hk, d, dtype):
    lens = [(150, 700), (1, 1), (0, 77), (70, 70), (300, 1100)]
    m = Made(lens, Hk, d, 64 if d < 256 else 16, dtype, seed=sinks)
    q = m.normal(m.T, Hq, d) * 3
    vis = masks(kind, lens, 5)
    kw = logits_of(logits, m, Hq)
    seen = sink_sets(lens, vis[:, 0], vis[:, 1], sinks)
    was = held(m)
    poison(m, seen)
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=sinks, **kw)
    assert up.get_device_error() == 0
    check(m, out, lse, oracle(was, q, seen, d ** -0.5, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d,dtype", [(8, 2, 64, "bf16"), (32, 8, 128, "fp16"), (16, 1, 256, "bf16")])
@pytest.mark.parametrize("sinks", [1, 40, 300])
@pytest.mark.parametrize("logits", ["plain", "both"])
def test_windows_that_end_before_the_cache(logits, sinks, Hq, Hk, d, dtype):
    """Entries whose end is any negative number leave a row empty, first tokens included, beside rows of the
    same tile that see several key tiles."""
    lens = [(60, 900), (7, 300)]
    m = Made(lens, Hk, d, 64, dtype, seed=sinks)
    q = m.normal(m.T, Hq, d) * 3
    vis = masks("window", lens, 5)
    low = -2 ** 31
    for t, (lo, hi) in enumerate([(0, low), (5, low), (2 ** 31 - 1, low), (low, low), (0, -1), (3, low + 100), (700, low + 600)]):
        vis[2 + 3 * t] = torch.tensor([lo, hi], dtype=torch.int32)
    vis[62] = torch.tensor([0, low], dtype=torch.int32)
    kw = logits_of(logits, m, Hq)
    seen = sink_sets(lens, vis[:, 0], vis[:, 1], sinks)
    was = held(m)
    poison(m, seen)
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=sinks, **kw)
    assert up.get_device_error() == 0
    # (far keys are biased by hundreds, see test_tokens_with_sinks)
    (check if logits == "plain" else check_at)(m, out, lse, oracle(was, q, seen, d ** -0.5, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [1, 5, 16, 64, 65, 200])
@pytest.mark.parametrize("Hq,Hk,d,dtype,page", [(8, 2, 64, "bf16", 16), (32, 8, 128, "fp16", 48), (16, 1, 256, "bf16", 128),
                                                (12, 4, 64, "fp16", 64), (5, 1, 128, "bf16", 384), (3, 3, 256, "fp16", 32)])
def test_tokens_with_sinks(Hq, Hk, d, dtype, page, sinks):
    lens = [(1, kv) for kv in (1, 0, 64, 700, 701, 3000, 5000, 90, 200, 201)]
    # before the beginning, past the end, inside the first tokens, right behind them, far on, at the last slot
    start = torch.tensor([-5, 0, 70, 300, 3, 2999, 4000, 64, 199, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    m = Made(lens, Hk, d, page, dtype, seed=sinks)
    q = m.normal(m.T, Hq, d) * 2
    seen = sink_sets(lens, start, m.kv_lens, sinks)
    for kind in ("plain", "both"):
        kw = logits_of(kind, m, Hq)
        was = held(m)
        if kind == "both":
            poison(m, seen)
        out, lse = up.decode_attend(q, m.cache, kv_start=start, sinks=sinks, **kw)
        assert up.get_device_error() == 0
        # far keys are biased by hundreds: check's 2^-12 is for logits below 200, check_at's bound
        # counts 2^-18 of the logits that weigh (capped ones: 12 at most before their bias)
        (check if kind == "plain" else check_at)(m, out, lse, oracle(was, q, seen, d ** -0.5, **kw))


@pytest.mark.gpu
def test_sinks_without_a_window_change_nothing():
    m = Made([(9, 400), (64, 64)], 2, 128, 64, "bf16", seed=1)
    q = m.normal(m.T, 8, 128)
    for x, y in zip(up.attend_paged(q, m.cu, m.cache, sinks=5), up.attend_paged(q, m.cu, m.cache)):
        assert torch.equal(x, y)
    one = q[:2].contiguous()
    for x, y in zip(up.decode_attend(one, m.cache, sinks=5), up.decode_attend(one, m.cache)):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,Hk,n", [(128, 32, 8, 2000), (256, 16, 2, 700), (64, 8, 8, 1500)])
def test_long_chunks_with_sinks(d, Hq, Hk, n):
    """Enough units for every SM, whole ones and cut ones, with the first tokens' tiles at either end of a share."""
    lens = [(n, 9000), (n // 3, 5000), (77, 12000)]
    m = Made(lens, Hk, d, 128, "bf16", seed=2)
    q = m.normal(m.T, Hq, d)
    own = torch.cat([torch.arange(kv - k, kv) for k, kv in lens])
    vis = torch.stack([own - 1000, own + 1], 1).to(torch.int32).cuda()
    seen = sink_sets(lens, vis[:, 0], vis[:, 1], 70)
    was = held(m)
    poison(m, seen)
    out, lse = up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=70)
    assert up.get_device_error() == 0
    check(m, out, lse, oracle(was, q, seen, d ** -0.5))


# ------------------------------------------------------------------ trees

TREES = [[(1, 1)], [(1, 900)], [(8, 8)], [(5, 300), (0, 40), (7, 7), (1, 2)], [(31, 160), (32, 128 + 32), (33, 127 + 33)],
         [(64, 4000)], [(65, 700), (3, 131), (128, 129)], [(256, 256), (255, 1000), (2, 5)], [(40, 41)] * 9]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", TREES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tree_lengths(d, dtype, lens):
    i = TREES.index(lens)
    Hq, Hk = (HEADS + [(5, 1)])[(i + d // 64) % 6]
    m = Made(lens, Hk, d, [16, 128, 48, 64, 256, 384][(i + d) % 6], dtype, seed=i)
    q = m.normal(m.T, Hq, d) * 2
    parents = grow(lens, i, ["bushy", "chain", "star", "near"][(i + d // 64) % 4])
    out, lse = up.attend_tree(q, m.cu, parents.cuda(), m.cache)
    assert up.get_device_error() == 0
    check(m, out, lse, oracle(m, q, tree_sets(lens, parents), d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,d,dtype", [(8, 2, 64, "bf16"), (32, 8, 128, "bf16"), (12, 4, 128, "fp16"),
                                           (16, 1, 256, "fp16"), (3, 3, 256, "bf16"), (5, 1, 64, "fp16")])
@pytest.mark.parametrize("sinks", [0, 6, 150])
@pytest.mark.parametrize("logits", ["plain", "cap", "bias", "both"])
def test_trees_with_windows(logits, sinks, Hq, Hk, d, dtype):
    lens = [(60, 900), (1, 1), (20, 20), (130, 1300), (0, 5), (9, 640)]
    m = Made(lens, Hk, d, 32, dtype, seed=sinks)
    q = m.normal(m.T, Hq, d) * 3
    parents = grow(lens, 4)
    # windows that begin anywhere: before the beginning, inside, at the tree, past it
    start = torch.cat([torch.randint(max(0, kv - n - 300), kv - n + 20, (n,), generator=torch.Generator().manual_seed(n))
                       for n, kv in lens]).to(torch.int32)
    start[::9] = torch.where(start[::9] % 2 == 0, -3, 2 ** 31 - 1).to(torch.int32) if sinks == 6 else start[::9]
    kw = logits_of(logits, m, Hq)
    seen = tree_sets(lens, parents, start, sinks)
    was = held(m)
    poison(m, seen)
    out, lse = up.attend_tree(q, m.cu, parents.cuda(), m.cache, kv_start=start.cuda(), sinks=sinks, **kw)
    assert up.get_device_error() == 0
    check(m, out, lse, oracle(was, q, seen, d ** -0.5, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_chain_is_a_chunk(d):
    lens = [(100, 2300), (17, 17)]
    m = Made(lens, 2, d, 64, "bf16", seed=3)
    q = m.normal(m.T, 8, d)
    a, la = up.attend_tree(q, m.cu, grow(lens, 0, "chain").cuda(), m.cache)
    b, lb = up.attend_paged(q, m.cu, m.cache)
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -6 and torch.allclose(la, lb, atol=1e-4)


@pytest.mark.gpu
def test_malformed_trees():
    """A parent that does not come before its child, or too many tokens: the sequence's rows are
    empty, the others' are not touched by it, whatever its cache holds."""
    lens = [(5, 200), (6, 300), (257, 400), (4, 4), (7, 90)]
    m = Made(lens, 2, 64, 32, "bf16", seed=4)
    q = m.normal(m.T, 8, 64)
    parents = grow(lens, 1)
    want = oracle(m, q, tree_sets(lens, parents), 0.125)
    for t, wrong in ((2, 2), (2, 4), (0, 0), (4, -2), (3, 2 ** 31 - 1), (1, -2 ** 31)):
        bad = parents.clone()
        bad[t] = wrong
        out, lse = up.attend_tree(q, m.cu, bad.cuda(), m.cache)
        assert up.get_device_error() == 0x80
        w = [x.clone() if torch.is_tensor(x) else x for x in want]
        for rows in (slice(0, 5), slice(11, 268)):
            w[0][rows], w[1][rows], w[2][rows] = 0.0, 0.0, -math.inf
        check(m, out, lse, w)
    m.kv_lens[1] = 5  # fewer than its drafted tokens
    out, lse = up.attend_tree(q, m.cu, parents.cuda(), m.cache)
    assert up.get_device_error() == 0xc0
    assert bool((out[5:11] == 0).all()) and bool((lse[5:11] == -math.inf).all())
    for cu in ([0, 5, 11, 200, 272, 300], [3, 5, 11, 268, 272, 279], [0, 9, 8, 268, 272, 279]):
        out, lse = up.attend_tree(q, torch.tensor(cu, dtype=torch.int32, device="cuda"), parents.cuda(), m.cache)
        assert up.get_device_error() & 1
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,Hk", [(64, 8, 2), (128, 32, 8), (256, 16, 1)])
def test_a_malformed_tree_leaves_other_windows_alone(d, Hq, Hk):
    """The window of each sequence's tokens, beside a sequence whose parents are wrong."""
    lens = [(20, 700), (6, 300), (33, 1500), (9, 640)]
    m = Made(lens, Hk, d, 32, "bf16", seed=4)
    q = m.normal(m.T, Hq, d)
    parents = grow(lens, 1)
    start = torch.cat([torch.randint(kv - n - 400, kv - n, (n,), generator=torch.Generator().manual_seed(n)) for n, kv in lens])
    start = start.clamp(min=0).to(torch.int32)
    seen = tree_sets(lens, parents, start, 5)
    was = held(m)
    poison(m, seen)
    want = oracle(was, q, seen, d ** -0.5)
    bad = parents.clone()
    bad[22] = 2
    for x in want[:3]:
        x[20:26] = 0.0 if x is not want[2] else -math.inf
    for _ in range(50):
        out, lse = up.attend_tree(q, m.cu, bad.cuda(), m.cache, kv_start=start.cuda(), sinks=5)
        assert up.get_device_error() == 0x80
        check(m, out, lse, want)


# ------------------------------------------------------------------ how calls are made

@pytest.mark.gpu
def test_repeat_graph_and_side_stream():
    """The same bits again, from a captured graph replayed on other trees and from another stream."""
    t = Made([(30, 3000), (9, 77)], 8, 128, 64, "bf16", seed=9)
    c = Made([(130, 2000), (64, 64)], 8, 128, 64, "bf16", seed=10)
    q, qc = t.normal(t.T, 32, 128), c.normal(c.T, 32, 128)
    one = qc[:2].contiguous()
    parents, other = (grow(t.lens, k).cuda() for k in (1, 2))
    vis = masks("window", c.lens, 0)
    start = torch.tensor([1500, 20], dtype=torch.int32, device="cuda")
    line = parents.clone()

    def step(stream=None):
        return (up.attend_tree(q, t.cu, line, t.cache, stream=stream)
                + up.attend_paged(qc, c.cu, c.cache, visible=vis, sinks=9, stream=stream)
                + up.decode_attend(one, c.cache, kv_start=start, sinks=9, stream=stream))

    first = [x.clone() for x in step()]
    for x, y in zip(first, step()):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = step(side)
    side.synchronize()
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    line.copy_(other)
    want = [x.clone() for x in step()]
    assert not torch.equal(want[0], first[0])
    for src, ref in ((other, want), (parents, first)):
        line.copy_(src)
        for x in kept:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(ref, kept):
            assert torch.equal(x, y)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_offsets_past_32_bits():
    page, Hk, d = 256, 8, 128
    n = (1 << 32) // (page * Hk * d) + 5
    kp = torch.empty(n, Hk, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    m = Made([(30, 700)], Hk, d, page, "bf16", seed=8, poison=False)
    far = torch.tensor([[n - 1, n - 3, n - 4, -1]], dtype=torch.int32, device="cuda")
    at, to = m.table[0, :3].long(), far[0, :3].long()
    kp[to], vp[to] = m.kp[at], m.vp[at]
    cache = up.PagedKV(kp, vp, far, m.kv_lens)
    q = m.normal(30, 32, d)
    parents = grow(m.lens, 1).cuda()
    own = torch.arange(670, 700, device="cuda", dtype=torch.int32)
    vis = torch.stack([own - 100, own + 1], 1).contiguous()
    start = torch.tensor([600], dtype=torch.int32, device="cuda")
    for call in (lambda c: up.attend_tree(q, m.cu, parents, c),
                 lambda c: up.attend_paged(q, m.cu, c, visible=vis, sinks=3),
                 lambda c: up.decode_attend(q[:1].contiguous(), c, kv_start=start, sinks=3)):
        for x, y in zip(call(cache), call(m.cache)):
            assert torch.equal(x, y)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_python_refusals_on_the_gpu():
    m = Made([(3, 20)], 2, 64, 16, "bf16")
    q = m.normal(3, 8, 64)
    par = torch.tensor([-1, 0, 1], dtype=torch.int32, device="cuda")
    vis = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        up.attend_tree(q, m.cu, par.long(), m.cache)
    with pytest.raises(ValueError):
        up.attend_tree(q, m.cu, par[:2], m.cache)
    with pytest.raises(ValueError):
        up.attend_tree(q.transpose(0, 1), m.cu, par, m.cache)
    with pytest.raises(ValueError):
        up.attend_tree(q, m.cu, par, m.cache, kv_start=par[:1])
    with pytest.raises(ValueError):
        up.attend_tree(q, m.cu, par, m.cache, slopes=torch.zeros(8, device="cuda"))
    with pytest.raises(up.UpError):
        up.attend_tree(q, m.cu, par, m.cache, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    for sinks in (-1, 5000, 10 ** 12, -10 ** 12):
        for call in (lambda: up.attend_tree(q, m.cu, par, m.cache, kv_start=par, sinks=sinks),
                     lambda: up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=sinks),
                     lambda: up.decode_attend(q[:1].contiguous(), m.cache, kv_start=par[:1], sinks=sinks)):
            with pytest.raises(up.UpError):
                call()
    with pytest.raises(TypeError):
        up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=1.5)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_expired_wait_stops_the_kernel_cleanly():
    """(The waits of a few tokens' call end before the first look at the clock.)"""
    m = Made([(600, 2000)], 8, 128, 64, "bf16", seed=17)
    q = m.normal(600, 32, 128)
    own = torch.arange(1400, 2000, device="cuda")
    vis = torch.stack([own - 1000, own + 1], 1).to(torch.int32)
    want = [x.clone() for x in up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=9)]
    up.set_wait_limit(64)
    try:
        up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=9)
        assert up.get_device_error() & 0x4
    finally:
        up.set_wait_limit(0)
    for x, y in zip(want, up.attend_paged(q, m.cu, m.cache, visible=vis, sinks=9)):
        assert torch.equal(x, y)
    assert up.get_device_error() == 0
