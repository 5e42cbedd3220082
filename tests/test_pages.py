"""The pool of pages (reserve_pages, fork_pages, release_pages), copy_pages and compact_kv
against models on the host, and their refusals."""
import copy
import ctypes
import random

import pytest
import torch

import block_sparse_long_up_gb300 as up
from block_sparse_long_up_gb300.pages import _CPool
from test_paged import BAD_CACHES, L, Made, _cache  # noqa: F401 (L is a fixture)


# ------------------------------------------------------------------ refusals (no GPU)

def _pool(refs=256, free=256, num=256, pages=64):
    return ctypes.byref(_CPool(refs, free, num, pages))


def _reserve(L, pool=None, table=256, B=2, mp=8, ps=16, have=256, want=256):
    return L.up_reserve_pages(pool or _pool(), table, B, mp, ps, have, want, None)


def _release(L, pool=None, table=256, B=2, mp=8, ps=16, first=None, end=256):
    return L.up_release_pages(pool or _pool(), table, B, mp, ps, first, end, None)


def _fork(L, pool=None, table=1 << 20, lens=1 << 21, B=2, mp=8, ps=16, parents=1 << 22, n=3, out=1 << 23, lout=1 << 24,
          copies=1 << 25):
    return L.up_fork_pages(pool or _pool(), table, lens, B, mp, ps, parents, n, out, lout, copies, None)


def _copy(L, cache=None, copies=256, n=3):
    return L.up_copy_pages(cache or _cache(), copies, n, None)


def _compact(L, cache=None, cu=512, T=10, keep=256, nf=10, cb=None, G=1, out=1024, ws=256, wsb=1 << 40):
    return L.up_compact_kv(cache or _cache(), cu, T, keep, nf, cb, G, out, ws, wsb, None)


def test_pool_refusals(L):  # noqa: F811
    for call in (_reserve, _release, _fork):
        for bad in (dict(pool=_pool(refs=None)), dict(pool=_pool(free=None)), dict(pool=_pool(num=None)),
                    dict(pool=_pool(pages=0)), dict(pool=_pool(pages=1 << 31)), dict(pool=_pool(refs=258)),
                    dict(table=None), dict(table=258), dict(B=-1), dict(mp=0), dict(ps=0), dict(ps=24), dict(ps=-16),
                    dict(B=1 << 16, mp=1 << 16)):
            assert call(L, **bad) == 1, (call, bad)
    for bad in (dict(have=None), dict(want=None), dict(have=258), dict(want=257)):
        assert _reserve(L, **bad) == 1
    for bad in (dict(end=None), dict(end=257), dict(first=258)):
        assert _release(L, **bad) == 1
    for bad in (dict(lens=None), dict(parents=None), dict(out=None), dict(lout=None), dict(copies=None), dict(n=-1),
                dict(B=0), dict(n=1 << 28), dict(out=(1 << 20) + 4), dict(out=(1 << 20) - 4), dict(lout=(1 << 21) + 4),
                dict(lout=(1 << 22) + 8), dict(copies=258), dict(parents=258), dict(copies=1 << 20), dict(copies=1 << 21),
                dict(copies=(1 << 22) - 32), dict(copies=(1 << 23) + 4), dict(copies=(1 << 24) - 8), dict(out=1 << 21),
                dict(out=(1 << 22) - 4), dict(lout=(1 << 23) + 92), dict(lout=(1 << 20) + 60)):
        assert _fork(L, **bad) == 1, bad
    assert _reserve(L, B=0) == 0 and _release(L, B=0) == 0 and _fork(L, n=0) == 0
    assert L.up_reserve_pages(None, 256, 2, 8, 16, 256, 256, None) == 1


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, code):  # noqa: F811
    assert _copy(L, cache=_cache(**bad)) in ((code, 0) if bad in (dict(table=None), dict(lens=None)) else (code,))
    assert _compact(L, cache=_cache(**bad)) == code


def test_cache_refusals(L):  # noqa: F811
    for bad in (dict(copies=None), dict(copies=258), dict(n=-1), dict(n=1 << 30)):
        assert _copy(L, **bad) == 1, bad
    assert _copy(L, n=0) == 0
    for bad in (dict(cu=None), dict(keep=None), dict(out=None), dict(T=-1), dict(T=1 << 31), dict(nf=-1), dict(G=0),
                dict(G=-5), dict(G=2), dict(cu=258), dict(cb=258), dict(out=258),
                dict(T=2 ** 31 - 1, cache=_cache(Hk=64)), dict(out=260), dict(out=252), dict(out=520), dict(out=508),
                dict(out=1028, cb=1024)):
        assert _compact(L, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=272), dict(wsb=0)):
        assert _compact(L, **bad) == 3
    assert _compact(L, cache=_cache(B=0)) == 0
    assert up.compact_kv_workspace(1000, 4, 2, 64) > 0 and up.compact_kv_workspace(0, 4, 2, 64) > 0
    for bad in ((-1, 4, 2, 64), (10, -1, 2, 64), (10, 4, 0, 64), (10, 4, 2, 96), (2 ** 31 - 1, 4, 64, 64)):
        assert up.compact_kv_workspace(*bad) == 0


@pytest.mark.parametrize("n", [715827883, 1 << 30, (1 << 30) - 1])
def test_more_copies_than_indexes_reach_are_refused(L, n):  # noqa: F811
    """(One head of small pages: one launch would have the blocks.)"""
    assert _copy(L, cache=_cache(Hk=1, page=16), n=n) == 1


def test_python_refuses_host_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        up.PagePool(z, z, z[:1])
    with pytest.raises(TypeError):
        up.PagePool(None, z, z)
    with pytest.raises(ValueError):
        up.PagePool.full(0)
    with pytest.raises(TypeError):
        up.reserve_pages(None, z, 16, z, z)
    with pytest.raises(TypeError):
        up.copy_pages(None, z)
    with pytest.raises(TypeError):
        up.compact_kv(None, z, z)


# ------------------------------------------------------------------ the pool against a model

class Model:
    """The pool and block tables as plain lists."""

    def __init__(self, pages):
        self.refs, self.free = [0] * pages, list(range(pages - 1, -1, -1))

    def reserve(self, table, ps, have, want):
        err = 0
        for row, a, b in zip(table, have, want):
            if b > len(row) * ps:
                err |= 0x40
                continue
            for i in range(len(row)):
                if a <= i * ps < b and row[i] < 0:
                    if self.free:
                        row[i] = self.free.pop()
                        self.refs[row[i]] = 1
                    else:
                        err |= 0x100
        return err

    def release(self, table, ps, first, end):
        err, back = 0, []
        for row, a, b in zip(table, first, end):
            if b > len(row) * ps:
                err |= 0x40
                continue
            for i in range(len(row)):
                if a <= i * ps < b and row[i] >= 0:
                    p, row[i] = row[i], -1
                    if p >= len(self.refs):
                        err |= 8
                    elif self.refs[p] <= 0:
                        err |= 0x200
                    else:
                        self.refs[p] -= 1
                        if p not in back:
                            back.append(p)
        self.free += [p for p in reversed(back) if self.refs[p] == 0]
        return err

    def fork(self, table, lens, ps, parents):
        err, out, new, copies = 0, [], [], []
        width = len(table[0]) if table else 0
        for p in parents:
            row, n, c = [-1] * width, 0, (-1, -1, 0)
            if not 0 <= p < len(table):
                err |= 0x80
            elif not 0 <= lens[p] <= width * ps:
                err |= 0x40
            else:
                n, full = lens[p], lens[p] // ps
                own = table[p][full] if n % ps else -1
                if n % ps and own >= len(self.refs):
                    err, own = err | 8, -1
                c = (-1, -1, n % ps)
                if own >= 0 and not self.free:
                    err, n, full, c = err | 0x100, 0, 0, (-1, -1, 0)
                elif own >= 0:
                    q = self.free.pop()
                    self.refs[q], row[full], c = 1, q, (own, q, n % ps)
                for i in range(full):
                    if table[p][i] >= len(self.refs):
                        err |= 8
                    elif table[p][i] >= 0:
                        row[i] = table[p][i]
                        self.refs[row[i]] += 1
            out.append(row)
            new.append(n)
            copies.append(c)
        return out, new, copies, err


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(model, pool, table, rows):
    n = int(pool.num_free)
    assert n == len(model.free)
    assert pool.free_pages[:n].tolist() == model.free
    assert pool.refs.tolist() == model.refs
    assert table.tolist() == rows


@pytest.mark.gpu
@pytest.mark.parametrize("B,mp,ps,pages", [(1, 1, 16, 1), (3, 63, 16, 120), (2, 64, 48, 100), (5, 65, 128, 300),
                                           (40, 7, 64, 200), (300, 20, 16, 4000), (1, 3000, 32, 2900), (700, 2, 256, 1500)])
def test_pool_walks(B, mp, ps, pages):
    """Sequences that grow, end, are cut back, lose pages behind a window and are replaced by forks of
    others, in any order, until pages run out."""
    r = random.Random(B * mp)
    model, pool = Model(pages), up.PagePool.full(pages)
    rows, lens = [[-1] * mp for _ in range(B)], [0] * B
    table, kv = ints(rows), ints(lens)
    for step in range(30):
        what = r.choice(["grow", "grow", "end", "cut", "window", "fork"])
        if what == "grow":
            want = [min(mp * ps, n + r.randint(0, 3 * ps if B > 5 else mp * ps // 3 + 1)) for n in lens]
            if r.random() < 0.2:
                want[r.randrange(B)] = mp * ps + 1
            up.reserve_pages(pool, table, ps, ints(lens), ints(want))
            err = model.reserve(rows, ps, lens, want)
            # a sequence is as long as its pages go
            lens = [n if w > mp * ps else w if all(x >= 0 for x in row[-(-n // ps):-(-w // ps)]) else n
                    for n, w, row in zip(lens, want, rows)]
        elif what == "fork":
            parents = [r.randrange(B) if r.random() < 0.9 else r.choice([-1, B, 2 ** 31 - 1]) for _ in range(B)]
            new, nl, copies = up.fork_pages(pool, table, ints(lens), ps, ints(parents))
            mrows, mlens, mcopies, err = model.fork(rows, lens, ps, parents)
            assert new.tolist() == mrows and nl.tolist() == mlens and copies.T.tolist() == [list(c) for c in mcopies]
            assert up.get_device_error() == err
            end = [mp * ps] * B
            up.release_pages(pool, table, ps, None, ints(end))
            err = model.release(rows, ps, [0] * B, end)
            assert table.tolist() == rows
            table, rows, lens = new, mrows, mlens
        else:
            first = {"end": [0] * B, "cut": [r.randint(0, n) for n in lens], "window": [ps // 2] * B}[what]
            end = {"end": lens, "cut": lens, "window": [n // 2 - ps + 1 for n in lens]}[what]
            if r.random() < 0.2:
                end = list(end)
                end[r.randrange(B)] = mp * ps + 5
            picked = [r.random() < 0.4 for _ in range(B)]
            end = [e if k else -3 for e, k in zip(end, picked)]
            up.release_pages(pool, table, ps, ints(first), ints(end))
            err = model.release(rows, ps, first, end)
            if what != "window":
                lens = [f if k and e == n else n for f, k, n, e in zip(first, picked, lens, end)]
        assert up.get_device_error() == err, (step, what)
        same(model, pool, table, rows)


@pytest.mark.gpu
def test_fork_and_release_undo_one_another():
    pool = up.PagePool.full(100)
    table, lens = ints([[-1] * 12] * 3), ints([100, 64, 1])
    up.reserve_pages(pool, table, 16, ints([0] * 3), lens)
    was = [x.clone() for x in (pool.refs, pool.free_pages, pool.num_free, table)]
    for _ in range(2):
        t2, l2, copies = up.fork_pages(pool, table, lens, 16, ints([0, 0, 2, 1, 0]))
        assert l2.tolist() == [100, 100, 1, 64, 100] and copies[2].tolist() == [4, 4, 1, 0, 4]
        assert pool.refs[table[0, :6].long()].tolist() == [4] * 6 and pool.refs[table[1, :4].long()].tolist() == [2] * 4
        up.reserve_pages(pool, t2, 16, l2, l2 + 20)
        # what was taken last goes back first
        up.release_pages(pool, t2, 16, l2, l2 + 20)
        up.release_pages(pool, t2, 16, None, l2)
        assert bool((t2 == -1).all())
        for x, y in zip(was, (pool.refs, pool.free_pages, pool.num_free, table)):
            assert torch.equal(x, y)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_pool_errors():
    """What cannot be is reported and left out; counts stay what they should be."""
    def made():
        pool, table = up.PagePool.full(20), ints([[-1] * 8] * 3)
        up.reserve_pages(pool, table, 16, ints([0, 0, 0]), ints([50, 20, 128]))
        return pool, table

    pool, table = made()
    rows, model = table.tolist(), Model(20)
    model.reserve([[-1] * 8 for _ in range(3)], 16, [0, 0, 0], [50, 20, 128])
    same(model, pool, table, rows)
    # the same page twice, a page outside, a page that nobody holds
    for r in (rows, table):
        r[0][1] = rows[0][0] if r is rows else int(table[0, 0])
        r[1][0] = 20
        r[1][1] = 19
    held = list(model.refs)
    up.release_pages(pool, table, 16, None, ints([128, 128, 0]))
    err = model.release(rows, 16, [0] * 3, [128, 128, 0])
    assert err == 0x208 and up.get_device_error() == err and sum(held) - sum(model.refs) == 3
    same(model, pool, table, rows)
    # counts that cannot be
    for wrong in (-1, 21, 2 ** 31 - 1, -2 ** 31):
        pool, table = made()
        keep = table.clone()
        pool.num_free.fill_(wrong)
        up.reserve_pages(pool, table, 16, ints([50, 20, 128]), ints([60, 70, 128]))
        assert up.get_device_error() & 0x200
        assert torch.equal(table[:, :2], keep[:, :2])
        t2, l2, _ = up.fork_pages(pool, keep, ints([50, 20, 128]), 16, ints([0, 1, 2]))
        up.get_device_error()
        assert bool((t2 < 20).all()) and l2.tolist()[0] == 0
    # a stack that holds no pages
    pool, table = made()
    pool.free_pages.fill_(77)
    up.reserve_pages(pool, table, 16, ints([50, 20, 128]), ints([70, 70, 128]))
    assert up.get_device_error() == 0x200 and bool((table[:2, 5:] == -1).all())
    # lengths that cannot be
    pool, table = made()
    was = pool.refs.clone()
    t2, l2, c = up.fork_pages(pool, table, ints([-1, 129, 2 ** 31 - 1]), 16, ints([0, 1, 2]))
    assert up.get_device_error() == 0x40
    assert bool((t2 == -1).all()) and l2.tolist() == [0, 0, 0] and c[:2].tolist() == [[-1] * 3] * 2
    assert torch.equal(pool.refs, was)


@pytest.mark.gpu
@pytest.mark.parametrize("wrong", [-1, 21, 2 ** 31 - 1, -2 ** 31])
def test_a_count_that_cannot_be_changes_nothing(wrong):
    """A number of free pages that cannot be is reported by every call and stays, like the stack, the holders and the
    tables: once it is put right the pool is as it was."""
    pool, table = up.PagePool.full(20), ints([[-1] * 8] * 3)
    lens = ints([50, 20, 128])
    up.reserve_pages(pool, table, 16, ints([0, 0, 0]), lens)
    free = int(pool.num_free)
    was = [x.clone() for x in (pool.refs, pool.free_pages, table)]
    pool.num_free.fill_(wrong)

    def stays():
        assert up.get_device_error() == 0x200
        assert int(pool.num_free) == wrong
        for x, y in zip(was, (pool.refs, pool.free_pages, table)):
            assert torch.equal(x, y)

    up.reserve_pages(pool, table, 16, lens, ints([60, 70, 128]))
    stays()
    up.release_pages(pool, table, 16, None, lens)
    stays()
    t2, l2, copies = up.fork_pages(pool, table, lens, 16, ints([0, 1, 2]))
    stays()
    assert bool((t2 == -1).all()) and l2.tolist() == [0] * 3 and copies.tolist() == [[-1] * 3, [-1] * 3, [0] * 3]
    pool.num_free.fill_(free)
    up.release_pages(pool, table, 16, None, lens)
    assert up.get_device_error() == 0 and int(pool.num_free) == 20 and not pool.refs.any() and bool((table == -1).all())


@pytest.mark.gpu
def test_a_page_named_too_often_goes_back_with_its_first_entry():
    """The first entry of a page is looked at after the second one: at the end of a run of the table, and at the
    beginning of the next."""
    B, mp = 512, 64
    rows = [[-1] * mp for _ in range(B)]
    rows[1][10] = rows[2][0] = 3
    rows[1][40], rows[1][50] = 5, 4
    for _ in range(20):
        model, table = Model(9), ints(rows)
        model.refs, model.free = [0, 0, 0, 1, 1, 1, 0, 0, 0], [0, 1, 2]
        pool = up.PagePool(ints(model.refs), ints(model.free + [8] * 6), ints([3]))
        mine, end = [list(r) for r in rows], [mp * 16] * B
        up.release_pages(pool, table, 16, None, ints(end))
        assert model.release(mine, 16, [0] * B, end) == up.get_device_error() == 0x200
        same(model, pool, table, mine)


@pytest.mark.gpu
@pytest.mark.parametrize("B,mp,pages", [(512, 64, 3000), (3, 700, 300), (900, 130, 70000), (1, 40, 4)])
def test_pages_named_more_often_than_held(B, mp, pages):
    """Entries of pages with fewer holders than entries, with none, and with a count that cannot be: the same tables and
    stack as in order."""
    r = random.Random(B)
    for _ in range(3):
        model, rows = Model(pages), [[-1] * mp for _ in range(B)]
        for row in rows:
            for i in range(mp):
                row[i] = r.choice([-1, -5, r.randrange(pages), r.randrange(pages)])
        named = [0] * pages
        for row in rows:
            for p in row:
                if p >= 0:
                    named[p] += 1
        model.refs = [r.choice([n, n, max(n - 1, 0), n + 1, 0, -3]) if n else 0 for n in named]
        model.free = [p for p in range(pages) if not named[p]]
        pool = up.PagePool(ints(model.refs), ints(model.free + [0] * (pages - len(model.free))), ints([len(model.free)]))
        table = ints(rows)
        first, end = [r.randint(-5, mp * 4) for _ in range(B)], [r.randint(mp * 4, mp * 16) for _ in range(B)]
        up.release_pages(pool, table, 16, ints(first), ints(end))
        assert up.get_device_error() == model.release(rows, 16, first, end)
        same(model, pool, table, rows)


@pytest.mark.gpu
def test_pool_calls_on_a_side_stream():
    """All calls with stream=, ordered by it alone, and buffers that the caller brings."""
    m = Made([(0, 70), (0, 48)], 2, 64, 16, "bf16", seed=3, extra=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    held = int((m.table >= 0).sum())
    refs = torch.zeros(m.kp.shape[0], dtype=torch.int32, device="cuda")
    refs[m.table[m.table >= 0].long()] = 1
    order = torch.argsort(refs, stable=True).to(torch.int32)  # free pages first
    pool = up.PagePool(refs, order, ints([refs.numel() - held]))
    table, lens, copies = (ints([[-7] * m.table.shape[1]] * 3), ints([0] * 3), ints([[0] * 3] * 3))
    par, more = ints([1, 0, 0]), ints([60, 80, 80])
    torch.cuda.synchronize()
    out = up.fork_pages(pool, m.table, m.kv_lens, 16, par, table_out=table, lens_out=lens, copies=copies, stream=side)
    assert all(x is y for x, y in zip(out, (table, lens, copies)))
    up.copy_pages(m.cache, copies, stream=side)
    up.reserve_pages(pool, table, 16, lens, more, stream=side)
    side.synchronize()
    assert lens.tolist() == [48, 70, 70] and copies[2].tolist() == [0, 6, 6]
    assert [(row >= 0).sum().item() for row in table] == [4, 5, 5]
    for s, parent in enumerate(par.tolist()):
        i = torch.arange(int(lens[s]), device="cuda")
        for x in (m.kp, m.vp):
            assert equal(x[table[s].long()[i // 16], :, i % 16], x[m.table[parent].long()[i // 16], :, i % 16])
    up.release_pages(pool, table, 16, None, more, stream=side)
    side.synchronize()
    assert int(pool.num_free) == refs.numel() - held and int(refs.sum()) == held and up.get_device_error() == 0


@pytest.mark.gpu
def test_a_reserve_of_what_is_there_takes_nothing():
    """A decode step's reserve, captured once: a page only where a token begins one."""
    pool, table, lens = up.PagePool.full(64), ints([[-1] * 9] * 4), ints([1, 15, 16, 30])
    up.reserve_pages(pool, table, 16, ints([0] * 4), lens)
    graph, more = torch.cuda.CUDAGraph(), lens + 1
    with torch.cuda.graph(graph):
        up.reserve_pages(pool, table, 16, lens, more)
        lens.copy_(more)
        more.add_(1)
    for _ in range(100):
        graph.replay()
        graph_lens = lens.tolist()
        assert [(row >= 0).sum().item() for row in table] == [-(-n // 16) for n in graph_lens]
    assert up.get_device_error() == 0
    assert int(pool.num_free) == 64 - int((table >= 0).sum()) and sorted(table[table >= 0].tolist()) == list(
        range(int((table >= 0).sum())))


# ------------------------------------------------------------------ copies

@pytest.mark.gpu
@pytest.mark.parametrize("Hk,d,page,dtype", [(2, 64, 16, "bf16"), (8, 128, 256, "fp16"), (1, 256, 48, "bf16"), (3, 128, 128, "bf16")])
def test_copies(Hk, d, page, dtype):
    m = Made([(1, 20 * page)], Hk, d, page, dtype, seed=1)
    src = [0, 0, 3, -1, 7, 5, 9, 30, 2, 4]
    dst = [10, 11, 12, 13, -1, 15, 16, 17, 1 << 30, 18]
    rows = [page, 1, page - 3, page, 4, 0, page // 2, 3, 3, page + 1]
    want = [x.clone() for x in (m.kp, m.vp, m.pp)]
    for a, b, n in zip(src, dst, rows):
        if 0 <= a < m.kp.shape[0] and 0 <= b < m.kp.shape[0] and n <= page:
            for x, y in zip(want, (m.kp, m.vp, m.pp)):
                x[b][..., :n, :] if x.dim() == 4 else x[b]
                if x.dim() == 4:
                    x[b][:, :n] = y[a][:, :n]
                else:
                    x[b][:n] = y[a][:n]
    up.copy_pages(m.cache, ints([src, dst, rows]))
    assert up.get_device_error() == 8
    for x, y in zip(want, (m.kp, m.vp, m.pp)):
        assert torch.equal(x.nan_to_num(7.0) if x.is_floating_point() else x, y.nan_to_num(7.0) if y.is_floating_point() else y)
    bare = up.PagedKV(m.kp, m.vp, m.table, m.kv_lens)  # no positions
    before = m.pp.clone()
    up.copy_pages(bare, ints([[1], [19], [page]]))
    assert torch.equal(m.kp[19], m.kp[1]) and torch.equal(m.vp[19], m.vp[1]) and torch.equal(m.pp, before)
    up.copy_pages(m.cache, ints([[], [], []]).view(3, 0))
    assert up.get_device_error() == 0


# ------------------------------------------------------------------ compaction

def flags_of(lens, G, share, seed, first=None):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, _ in lens:
        f = torch.rand(-(-n // G), generator=g) < share
        if first is not None and f.numel():
            f[:first] = True
            f[first:first + 1] = False
        out.append(f)
    return out


def compacted(m, flags, G):
    """(k, v, positions, lengths) that a compaction leaves."""
    k, v, p, new = m.kp.clone(), m.vp.clone(), m.pp.clone(), []
    for s, ((n, kv), f) in enumerate(zip(m.lens, flags)):
        i = torch.arange(n)
        src = (kv - n + i[f[i // G]] if n else i).cuda()
        dst = torch.arange(kv - n, kv - n + src.numel(), device="cuda")
        row = m.table[s].long()
        a, b, c, e = row[src // m.page], src % m.page, row[dst // m.page], dst % m.page
        k[c, :, e], v[c, :, e], p[c, e] = m.kp[a, :, b], m.vp[a, :, b], m.pp[a, b]
        new.append(kv - n + src.numel())
    return k, v, p, new


def equal(x, y):
    return torch.equal(x.view(torch.int16), y.view(torch.int16)) if x.is_floating_point() else torch.equal(x, y)


COMPACT = [([(1, 1)], 1), ([(5, 300), (0, 40), (7, 7), (1, 2)], 1), ([(64, 4000)] * 9, 1), ([(300, 300), (255, 1000), (257, 700)], 1),
           ([(3000, 3100), (0, 0), (0, 9), (5000, 5000)], 1), ([(4000, 4000), (65, 65), (1, 500)], 64),
           ([(0, 5)] * 40 + [(9000, 9100)] + [(3, 3)] * 30, 1), ([(9000, 9001), (127, 127), (129, 400)], 128), ([(700, 700)], 32), ([(20000, 20000)], 1), ([(1000, 1000)], 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,G", COMPACT, ids=str)
@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("d,Hk,dtype", [(64, 2, "bf16"), (128, 8, "fp16"), (256, 1, "bf16")])
@pytest.mark.parametrize("into", ["new", "the cache's"])
def test_compaction(into, d, Hk, dtype, share, lens, G):
    """(Lengths written over the cache's own take the launches of many tokens, whatever their number.)"""
    i = COMPACT.index((lens, G))
    m = Made(lens, Hk, d, [16, 128, 48, 64, 256, 384][(i + d // 64) % 6], dtype, seed=i)
    flags = flags_of(lens, G, share, i)
    k, v, p, new = compacted(m, flags, G)
    keep = torch.cat(flags).to(torch.uint8).cuda() * 3  # any value but 0 counts
    cb = ints([0] + [f.numel() for f in flags]).cumsum(0, dtype=torch.int32)
    out = up.compact_kv(m.cache, m.cu, keep, cu_blocks=None if G == 1 else cb, G=G,
                        kv_lens_out=None if into == "new" else m.kv_lens)
    assert up.get_device_error() == 0
    assert out.tolist() == new and m.kv_lens.tolist() == ([kv for _, kv in lens] if into == "new" else new)
    assert equal(m.kp, k) and equal(m.vp, v) and equal(m.pp, p)


@pytest.mark.gpu
def test_nothing_flagged():
    m = Made([(0, 50), (0, 0)], 2, 64, 16, "bf16", seed=1)
    none = torch.zeros(0, dtype=torch.uint8, device="cuda")
    for most in (None, 0, 1, 50000):
        for into in (None, m.kv_lens):
            was = m.kp.clone()
            assert up.compact_kv(m.cache, m.cu, none, max_tokens=most, kv_lens_out=into).tolist() == [50, 0]
            assert equal(m.kp, was) and up.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,first,share", [(40000, 0, 1.0), (40000, 1, 1.0), (40000, 20000, 1.0), (60000, 100, 0.999),
                                           (131072, 0, 0.3)])
def test_every_tile_waits_for_its_neighbour(n, first, share):
    """One token dropped: every row moves by one slot, into the rows that the tile before read."""
    m = Made([(n, n), (77, 200)], 4, 128, 256, "bf16", seed=2)
    flags = flags_of(m.lens, 1, share, 3, first)
    k, v, p, new = compacted(m, flags, 1)
    keep = torch.cat(flags).to(torch.uint8).cuda()
    out = up.compact_kv(m.cache, m.cu, keep, kv_lens_out=m.kv_lens)
    assert up.get_device_error() == 0 and out is m.kv_lens and out.tolist() == new
    assert equal(m.kp, k) and equal(m.vp, v) and equal(m.pp, p)


@pytest.mark.gpu
def test_many_sequences_compact():
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 5, (2500,), generator=g).tolist()
    lens = [(a, a + b) for a, b in zip(n, torch.randint(0, 40, (2500,), generator=g).tolist())]
    m = Made(lens, 2, 64, 16, "bf16", seed=14)
    flags = flags_of(lens, 1, 0.5, 1)
    k, v, p, new = compacted(m, flags, 1)
    was = [x.clone() for x in (m.kp, m.vp, m.pp)]
    for into in (None, m.kv_lens):
        for x, y in zip((m.kp, m.vp, m.pp), was):
            x.copy_(y)
        out = up.compact_kv(m.cache, m.cu, torch.cat(flags).to(torch.uint8).cuda(), kv_lens_out=into)
        assert up.get_device_error() == 0 and out.tolist() == new
        assert equal(m.kp, k) and equal(m.vp, v) and equal(m.pp, p)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[(16, 20)] * 256, [(15, 20)] * 257, [(3841, 3900)] + [(1, 9)] * 255, [(3842, 3900)] + [(1, 9)] * 255,
                                  [(4096, 4096)] + [(0, 3)] * 15, [(1024, 1100)], [(1025, 1100)]], ids=lambda x: f"{len(x)}-{x[0]}")
def test_compaction_where_the_launches_change(lens):
    """About as many tokens and sequences as one launch serves, and one more."""
    m = Made(lens, 2, 64, 32, "bf16", seed=21)
    flags = flags_of(lens, 1, 0.6, 4)
    k, v, p, new = compacted(m, flags, 1)
    out = up.compact_kv(m.cache, m.cu, torch.cat(flags).to(torch.uint8).cuda())
    assert up.get_device_error() == 0 and out.tolist() == new
    assert equal(m.kp, k) and equal(m.vp, v) and equal(m.pp, p)


@pytest.mark.gpu
@pytest.mark.parametrize("more", [0, 20000])
def test_compaction_errors(more):
    """Of few tokens a sequence and of many (max_tokens counts)."""
    lens = [(100, 300), (50, 90), (64, 64)]
    most = dict(max_tokens=214 + more)

    def made():
        return Made(lens, 2, 64, 32, "bf16", seed=5)

    flags = flags_of(lens, 1, 0.5, 2)
    keep = torch.cat(flags).to(torch.uint8).cuda()
    full = compacted(made(), flags, 1)
    # a malformed cu_seqlens: nothing moves
    for cu in ([1, 100, 150, 214], [0, 100, 90, 214], [0, 100, 150, 215 + more], [0, -1, 150, 214], [0, 100, 150, 1 << 30]):
        m = made()
        was = m.kp.clone()
        out = up.compact_kv(m.cache, ints(cu), keep, **most)
        assert up.get_device_error() == 1 and torch.equal(out, m.kv_lens) and equal(m.kp, was)
    # sequences that cannot be stay, the others do not
    for cb, kv in (([0, 100, 149, 214], None), ([0, 100, 100, 164], None), (None, 49), (None, -1), (None, 10 ** 6)):
        m = made()
        if kv is not None:
            m.kv_lens[1] = kv
        out = up.compact_kv(m.cache, m.cu, keep, cu_blocks=None if cb is None else ints(cb), **most)
        assert up.get_device_error() == (0x10 if kv is None else 0x40)
        assert out.tolist()[1] == (90 if kv is None else kv) and out.tolist()[0] == full[3][0]
        at = m.table[1, :3].long()
        assert equal(m.kp[at], made().kp[at])
        at = m.table[0, :10].long()
        assert equal(m.kp[at], full[0][at]) and equal(m.pp[at], full[2][at])
    m = made()
    out = up.compact_kv(m.cache, m.cu, keep[:200])  # flags that end too early
    assert up.get_device_error() in (1, 0x10)
    # one flag for all of a sequence, however large its blocks; none for the last
    for G in (100, 300, 2 ** 31 - 1):
        m = made()
        out = up.compact_kv(m.cache, m.cu, keep[:2] * 0, cu_blocks=ints([0, 1, 2, 2]), G=G, **most)
        assert up.get_device_error() == 0x10 and out.tolist() == [200, 40, 64]
    m = made()
    out = up.compact_kv(m.cache, m.cu, keep[:200], **most)
    assert up.get_device_error() == 0x10 and out.tolist() == full[3][:2] + [64]
    # a page outside the pool: its tokens, and those that would move there, stay
    m = made()
    was = [x.clone() for x in (m.kp, m.vp, m.pp)]
    m.table[0, 8] = -1
    out = up.compact_kv(m.cache, m.cu, keep, **most)
    assert up.get_device_error() == 8 and out.tolist() == full[3]
    others = torch.ones(m.kp.shape[0], dtype=torch.bool, device="cuda")
    others[made().table[0, 8].long()] = False
    assert equal(m.kp[~others], was[0][~others])
    assert equal(m.kp[m.table[1, :3].long()], full[0][m.table[1, :3].long()])


@pytest.mark.gpu
def test_compaction_in_a_graph_and_on_a_side_stream():
    lens = [(3000, 5000), (64, 100)]
    m = Made(lens, 8, 128, 64, "bf16", seed=6, poison=False)
    flags = flags_of(lens, 1, 0.6, 2)
    keep = torch.cat(flags).to(torch.uint8).cuda()
    was = [x.clone() for x in (m.kp, m.vp, m.pp)]
    want = compacted(m, flags, 1)

    def check(out):
        assert out.tolist() == want[3]
        for x, y, z in zip((m.kp, m.vp, m.pp), want, was):
            assert equal(x, y)
            x.copy_(z)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = up.compact_kv(m.cache, m.cu, keep, stream=side)
    side.synchronize()
    check(out)
    graph = torch.cuda.CUDAGraph()
    up.compact_kv(m.cache, m.cu, keep)
    for x, z in zip((m.kp, m.vp, m.pp), was):
        x.copy_(z)
    with torch.cuda.graph(graph):
        out = up.compact_kv(m.cache, m.cu, keep)
    for _ in range(3):
        graph.replay()
        check(out)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_more_tokens_than_the_pool_has_slots():
    """Sequences that share pages, or have let pages go, count more tokens than there are slots; none of them is kept,
    so nothing moves."""
    pool, table = up.PagePool.full(60), ints([[-1] * 64])
    lens = ints([900])
    up.reserve_pages(pool, table, 16, ints([0]), lens)
    kp, vp = (torch.zeros(60, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    t3, l3, copies = up.fork_pages(pool, table, lens, 16, ints([0, 0, 0]))
    cache, cu = up.PagedKV(kp, vp, t3, l3), ints([0, 900, 1800, 2700])
    none = torch.zeros(2700, dtype=torch.uint8, device="cuda")
    assert l3.tolist() == [900] * 3
    assert up.compact_kv(cache, cu, none).tolist() == [0] * 3
    # a flag for all of a sequence
    assert up.compact_kv(cache, cu, none[:3], cu_blocks=ints([0, 1, 2, 3]), G=2 ** 31 - 1).tolist() == [0] * 3
    # pages behind a window that went back
    gone = up.PagedKV(kp[:4].contiguous(), vp[:4].contiguous(), ints([[-1] * 300]), ints([4700]))
    assert up.compact_kv(gone, ints([0, 4700]), torch.zeros(4700, dtype=torch.uint8, device="cuda")).tolist() == [0]
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_offsets_past_32_bits():
    page, Hk, d = 256, 8, 128
    n = (1 << 32) // (page * Hk * d) + 5
    kp = torch.empty(n, Hk, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    pp = torch.zeros(n, page, dtype=torch.int32, device="cuda")
    m = Made([(700, 700)], Hk, d, page, "bf16", seed=8, poison=False)
    far = ints([[n - 1, n - 3, n - 4, -1]])
    at, to = m.table[0, :3].long(), far[0, :3].long()
    kp[to], vp[to], pp[to] = m.kp[at], m.vp[at], m.pp[at]
    cache = up.PagedKV(kp, vp, far, m.kv_lens, pp)
    keep = torch.cat(flags_of(m.lens, 1, 0.5, 2)).to(torch.uint8).cuda()
    assert torch.equal(up.compact_kv(cache, m.cu, keep), up.compact_kv(m.cache, m.cu, keep))
    for x, y in ((kp, m.kp), (vp, m.vp), (pp, m.pp)):
        assert equal(x[to], y[at])
    up.copy_pages(cache, ints([[n - 1], [n - 2], [page]]))
    assert equal(kp[n - 2], kp[n - 1]) and equal(vp[n - 2], vp[n - 1]) and equal(pp[n - 2], pp[n - 1])
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_python_refusals_on_the_gpu():
    pool, table, lens = up.PagePool.full(10), ints([[-1] * 4] * 2), ints([3, 4])
    with pytest.raises(AttributeError):
        pool.refs = lens
    other = copy.copy(pool)
    assert other.refs is pool.refs and other.struct is not pool.struct
    with pytest.raises(TypeError):
        up.reserve_pages(pool, table.long(), 16, lens, lens)
    with pytest.raises(ValueError):
        up.reserve_pages(pool, table, 16, lens[:1], lens)
    with pytest.raises(ValueError):
        up.reserve_pages(pool, table[0], 16, lens, lens)
    with pytest.raises(ValueError):
        up.reserve_pages(pool, table[:, :2], 16, lens, lens)
    with pytest.raises(up.UpError):
        up.reserve_pages(pool, table, 24, lens, lens)
    with pytest.raises(up.UpError):
        up.fork_pages(pool, table, lens, 16, lens, table_out=table)
    with pytest.raises(ValueError):
        up.fork_pages(pool, table, lens, 16, lens, table_out=table[:1])
    with pytest.raises(up.UpError):
        up.fork_pages(pool, table, lens, 16, ints([0, 1]), lens_out=lens)
    m = Made([(2, 20)], 2, 64, 16, "bf16")
    keep = torch.ones(2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        up.copy_pages(m.cache, ints([1, 2, 3]))
    with pytest.raises(TypeError):
        up.compact_kv(m.cache, m.cu, keep.bool())
    with pytest.raises(ValueError):
        up.compact_kv(m.cache, m.cu[:1], keep)
    with pytest.raises(up.UpError):
        up.compact_kv(m.cache, m.cu, keep, G=2)
    with pytest.raises(up.UpError):
        up.compact_kv(m.cache, m.cu, keep, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(up.UpError):
        up.compact_kv(m.cache, m.cu, keep, max_tokens=-5)
    assert up.get_device_error() == 0


@pytest.mark.gpu
def test_expired_wait_stops_the_move():
    """A wait bound of one cycle, every tile waiting for the one before it: the timeout is reported and
    the context stays usable."""
    m = Made([(60000, 60000)], 8, 128, 256, "bf16", seed=2, poison=False)
    flags = flags_of(m.lens, 1, 1.0, 3, 0)
    keep = torch.cat(flags).to(torch.uint8).cuda()
    was = [x.clone() for x in (m.kp, m.vp, m.pp)]
    want = compacted(m, flags, 1)
    up.set_wait_limit(1)
    try:
        for _ in range(20):
            up.compact_kv(m.cache, m.cu, keep)
            if up.get_device_error() & 0x4:
                break
        else:
            raise AssertionError("no wait ran out")
    finally:
        up.set_wait_limit(0)
    for x, z in zip((m.kp, m.vp, m.pp), was):
        x.copy_(z)
    up.compact_kv(m.cache, m.cu, keep)
    assert up.get_device_error() == 0
    assert equal(m.kp, want[0]) and equal(m.vp, want[1]) and equal(m.pp, want[2])


# ------------------------------------------------------------------ together

@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,Hk,dtype", [(64, 8, 2, "bf16"), (128, 12, 4, "fp16"), (256, 16, 2, "bf16")])
def test_a_tree_is_verified_accepted_and_cut_back(d, Hq, Hk, dtype):
    """A forked sequence drafts a tree, keeps one path and lets the rest go: its cache then holds what
    appending the path's tokens one by one leaves, and a decode step over it gives the same."""
    ps, B, n = 16, 3, 9
    parents = [-1, 0, 0, 1, 1, 2, 3, 6, 4]
    path = [0, 1, 3, 6, 7]
    depth = [0, 1, 1, 2, 2, 2, 3, 4, 3]
    lens = [37, 16, 95]
    g = torch.Generator(device="cuda").manual_seed(d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    pool, width = up.PagePool.full(60), 8
    kp, vp = normal(60, Hk, ps, d), normal(60, Hk, ps, d)
    pp = torch.zeros(60, ps, dtype=torch.int32, device="cuda")
    freq = 10000.0 ** -(torch.arange(0, d, 2, device="cuda") / d)
    cu0 = ints([0, 37, 53, 148])
    x = [normal(148, h, d) for h in (Hq, Hk, Hk)]
    table, kv = ints([[-1] * width] * B), ints(lens)
    up.reserve_pages(pool, table, ps, ints([0] * B), kv)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens]).to(torch.int32)
    up.append_kv(None, x[1], x[2], pos, cu0, up.PagedKV(kp, vp, table, kv, pp), freq)
    # two continuations of the same prompts: one drafts, the other gets the path's tokens one at a time
    both, l2, copies = up.fork_pages(pool, table, kv, ps, ints([0, 1, 2, 0, 1, 2]))
    up.copy_pages(up.PagedKV(kp, vp, both, l2, pp), copies)
    up.release_pages(pool, table, ps, None, kv)
    tree, line = both[:B].contiguous(), both[B:].contiguous()
    tl, ll = l2[:B].clone(), l2[B:].clone()
    q, k, v = (normal(B * n, h, d) for h in (Hq, Hk, Hk))
    old = tl.clone()
    up.reserve_pages(pool, tree, ps, old, old + n)
    tl += n
    cache = up.PagedKV(kp, vp, tree, tl, pp)
    cu = ints([0, n, 2 * n, 3 * n])
    tpos = (old[:, None] + ints(depth)[None]).flatten().contiguous()
    qr = up.append_kv(q, k, v, tpos, cu, cache, freq)
    out, lse = up.attend_tree(qr, cu, ints(parents * B), cache)
    flags = torch.zeros(B, n, dtype=torch.uint8, device="cuda")
    flags[:, path] = 1
    new = up.compact_kv(cache, cu, flags.view(-1))
    up.release_pages(pool, tree, ps, new, tl)
    assert torch.equal(new, old + len(path))
    tl.copy_(new)
    one = ints([0, 1, 2, 3])
    for j in path:
        up.reserve_pages(pool, line, ps, ll, ll + 1)
        ll += 1
        at = torch.arange(B, device="cuda") * n + j
        c = up.PagedKV(kp, vp, line, ll, pp)
        qj = up.append_kv(q[at], k[at], v[at], (ll - 1), one, c, freq)
        o, l = up.decode_attend(qj, c)
        # (each rounds its weights its own way: a step of the type on values of a few units)
        assert float((o.float() - out[at].float()).abs().max()) <= 2.0 ** (-5 if dtype == "bf16" else -8)
        assert torch.allclose(l, lse[at], atol=1e-4)
    assert torch.equal(tl, ll)
    for s in range(B):
        i = torch.arange(int(ll[s]), device="cuda")
        for y in (kp, vp):
            assert equal(y[tree[s].long()[i // ps], :, i % ps], y[line[s].long()[i // ps], :, i % ps])
        assert torch.equal(pp[tree[s].long()[i // ps], i % ps], pp[line[s].long()[i // ps], i % ps])
    a = up.decode_attend(qr[:B].contiguous(), cache)
    b = up.decode_attend(qr[:B].contiguous(), up.PagedKV(kp, vp, line, ll, pp))
    assert all(torch.equal(u, w) for u, w in zip(a, b))
    for t, m in ((tree, tl), (line, ll)):
        up.release_pages(pool, t, ps, None, m)
    assert int(pool.num_free) == 60 and not pool.refs.any() and up.get_device_error() == 0


@pytest.mark.gpu
def test_pages_between_first_tokens_and_window_are_released():
    """A decode loop with a sliding window: the pages that fall behind it go back to the pool, and
    what is seen does not change."""
    ps, sinks, span, Hq, Hk, d = 16, 5, 70, 8, 2, 64
    pool, g = up.PagePool.full(16), torch.Generator(device="cuda").manual_seed(1)
    full = up.PagePool.full(64)

    def store(n):
        return (torch.zeros(n, Hk, ps, d, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(n, Hk, ps, d, dtype=torch.bfloat16, device="cuda"))

    lens = ints([0, 0])
    few, all_ = ints([[-1] * 32] * 2), ints([[-1] * 32] * 2)
    small = up.PagedKV(*store(16), few, lens)
    large = up.PagedKV(*store(64), all_, lens)
    one = ints([0, 1, 2])
    for t in range(300):
        old = lens.clone()
        for p, table in ((pool, few), (full, all_)):
            up.reserve_pages(p, table, ps, old, old + 1)
        lens += 1
        q, k, v = (torch.randn(2, h, d, generator=g, device="cuda").bfloat16() for h in (Hq, Hk, Hk))
        start = (lens - span).contiguous()
        up.release_pages(pool, few, ps, torch.full_like(start, sinks), start - (ps - 1))
        res = []
        for c in (small, large):
            up.append_kv(None, k, v, old, one, c, None)
            res.append(up.decode_attend(q, c, kv_start=start, sinks=sinks))
        assert all(torch.equal(x, y) for x, y in zip(*res)), t
        assert int((few >= 0).sum()) <= 2 * (2 + span // ps + 1)
    assert up.get_device_error() == 0 and int(pool.num_free) == 16 - int((few >= 0).sum())


@pytest.mark.gpu
def test_blocks_that_the_selection_keeps_stay_in_the_cache():
    """score -> select -> compact_kv: a prompt's cache keeps the selected blocks, in place."""
    lens = [(700, 700), (3000, 3000)]
    m = Made(lens, 2, 64, 128, "bf16", seed=3)
    q = m.normal(256, 8, 64)
    scores, cb = up.score_blocks_paged(q, m.kp.nan_to_num_(0.0), m.table, m.cu, 3700, 128, 64)
    keep, kept = up.select_topp(scores, cb, m.cu, 64, 0.5)
    nb = [-(-n // 64) for n, _ in lens]
    flags = [keep[int(cb[s]):int(cb[s]) + nb[s]].bool().cpu() for s in range(2)]
    k, v, p, new = compacted(m, flags, 64)
    out = up.compact_kv(m.cache, m.cu, keep, cu_blocks=cb, G=64)
    assert up.get_device_error() == 0
    assert out.tolist() == new == kept.tolist()
    assert equal(m.kp, k) and equal(m.vp, v) and equal(m.pp, p)


@pytest.mark.gpu
def test_example_decodes_trees():
    """Twice the same tokens, at least one a step, and no page lost (the example checks that)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    a, b = (ex.main(["--prompt", "200", "77", "--children", "3", "--steps", "5"]) for _ in range(2))
    assert a == b and len(a) == 6 and all(len(t) >= 6 for t in a)
