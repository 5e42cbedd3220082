"""What the serving operators around the paged cache are measured on: attention with a
sliding window and first tokens that stay visible (a chunk's, and one token's), attention
of a tree of drafted tokens, compaction of a cache in place, and forking and releasing
sequences that share pages.

`own` selects what run() computes with: False, the operators' plain form in elementary
torch operations; True, the library's calls.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------- the cases

MAX_LOGITS = 32 * 8192 * 12352
MAX_FLOPS = 4.0 * 128 * 32 * 8192 * 4160
MAX_CACHE = 131072 * 8 * 128  # elements of the keys that an attention case reads
MAX_MOVED = 131072 * 8 * 128  # and of those in a cache that is compacted or forked


def listed():
    """Head layouts 32/8 x 128, 16/2 x 256 and 8/2 x 64 and the lengths are those of the
    repository's own workloads."""
    return [
        # a short chunk behind a short cache, 4 tokens kept visible: latency
        dict(name="sink_chunk_128", op="chunk", dtype="bf16", B=1, Hq=8, Hk=2, d=64, page=128, n=128, kv=4096,
             ragged=False, lens=1, softcap=0.0, bias=False, span=1024, sinks=4),
        # a long chunk of a prompt, windows of 4K
        dict(name="sink_chunk_8k", op="chunk", dtype="bf16", B=1, Hq=32, Hk=8, d=128, page=256, n=8192, kv=65536,
             ragged=False, lens=2, softcap=0.0, bias=False, span=4096, sinks=64),
        # ragged prompts at head_dim 256, capped and biased, sinks past a key tile
        dict(name="sink_ragged_capped", op="chunk", dtype="fp16", B=4, Hq=16, Hk=2, d=256, page=64, n=1777, kv=8191,
             ragged=True, lens=3, softcap=50.0, bias=True, span=700, sinks=130),
        # one token of one conversation: latency
        dict(name="sink_decode_b1", op="token", dtype="bf16", B=1, Hq=8, Hk=2, d=64, page=128, n=1, kv=4096,
             ragged=False, lens=4, softcap=0.0, bias=False, span=512, sinks=4),
        # a serving batch of mixed lengths, windows of 8K
        dict(name="sink_decode_b64", op="token", dtype="bf16", B=64, Hq=32, Hk=8, d=128, page=256, n=1, kv=131072,
             ragged=True, lens=5, softcap=0.0, bias=False, span=8192, sinks=64),
        # a few drafted tokens of one conversation: latency
        dict(name="tree_b1_4k", op="tree", dtype="bf16", B=1, Hq=8, Hk=2, d=64, page=128, n=8, kv=4096,
             ragged=False, lens=6, softcap=0.0, bias=False, span=0, sinks=0),
        # a wide tree at 128K: the cache's bandwidth
        dict(name="tree_b1_128k", op="tree", dtype="bf16", B=1, Hq=32, Hk=8, d=128, page=256, n=64, kv=131072,
             ragged=False, lens=7, softcap=0.0, bias=False, span=0, sinks=0),
        # a batch of trees of other sizes at head_dim 256
        dict(name="tree_b32_ragged", op="tree", dtype="fp16", B=32, Hq=16, Hk=2, d=256, page=64, n=61, kv=20011,
             ragged=True, lens=8, softcap=0.0, bias=False, span=0, sinks=0),
        # the accepted paths of a batch of trees move together
        dict(name="compact_accept_b64", op="compact", dtype="bf16", B=64, Hk=8, d=128, page=256, n=64, kv=8192,
             ragged=True, lens=9, block=1, share=0.08),
        # a 128K prompt's cache keeps a quarter of its blocks
        dict(name="compact_blocks_128k", op="compact", dtype="bf16", B=1, Hk=8, d=128, page=256, n=131072, kv=131072,
             ragged=False, lens=10, block=64, share=0.25),
        # four continuations of one short conversation, one page more each, and gone again
        dict(name="fork_b4", op="fork", dtype="bf16", B=1, Hk=2, d=64, page=128, kv=4001, ragged=False, lens=11,
             children=4, grow=128),
        # a beam step: 256 children of 32 parents
        dict(name="fork_b256", op="fork", dtype="bf16", B=32, Hk=8, d=128, page=256, kv=8191, ragged=True, lens=12,
             children=256, grow=300),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: chunks, tokens and trees over caches of one token to
    128K, any window and number of first tokens, every head layout, page size and type."""
    op = rng.choice(["chunk", "token", "tree", "tree", "compact", "fork"])
    Hq, Hk = rng.choice([(32, 8), (16, 2), (8, 2), (8, 8), (12, 4), (16, 1)])
    d = rng.choice([64, 128, 256])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), B=_log_int(rng, 1, 64), Hk=Hk, d=d,
             page=rng.choice([16, 32, 48, 64, 128, 256, 384]), ragged=rng.random() < 0.7,
             lens=rng.randrange(1 << 30))
    if op == "compact":
        tree = rng.random() < 0.5
        c["n"] = _log_int(rng, 2, 128 if tree else 131072)
        c["kv"] = c["n"] + (_log_int(rng, 1, 30000) if tree else rng.choice([0, 0, _log_int(rng, 1, 3000)]))
        c["block"] = 1 if tree else rng.choice([1, 32, 64, 128])
        c["share"] = rng.choice([0.05, 0.2, 0.5, 0.9])
        while c["B"] * c["kv"] * Hk * d > MAX_MOVED:
            if c["B"] > 1:
                c["B"] //= 2
            else:
                c["kv"] = max(2, c["kv"] // 2)
                c["n"] = min(c["n"], c["kv"])
        return c
    if op == "fork":
        c["B"] = min(c["B"], 32)
        c["kv"] = _log_int(rng, 16, 32768)
        c["children"] = _log_int(rng, 1, 256)
        c["grow"] = _log_int(rng, 1, 1000)
        while c["B"] * c["kv"] * Hk * d > MAX_MOVED // 2 or c["children"] * c["page"] * Hk * d > MAX_MOVED // 2:
            c["B"] = max(1, c["B"] // 2)
            c["kv"] = max(16, c["kv"] // 2)
            c["children"] = max(1, c["children"] // 2)
        return c
    c["Hq"] = Hq
    c["softcap"] = rng.choice([0.0, 0.0, 0.0, 20.0, 50.0])
    c["bias"] = rng.random() < 0.2
    c["sinks"] = rng.choice([0, 1, 4, 4, 16, 64, 130])
    c["span"] = _log_int(rng, 16, 8192)
    if op == "token":
        c["n"], c["kv"] = 1, _log_int(rng, 1, 131072)
    elif op == "tree":
        c["n"] = _log_int(rng, 1, 128)
        c["kv"] = c["n"] + _log_int(rng, 1, 131072 - 128) - 1
        c["span"] = c["span"] if rng.random() < 0.25 else 0
    else:
        c["B"] = min(c["B"], 8)
        c["n"] = _log_int(rng, 2, 8192)
        c["kv"] = max(c["n"], _log_int(rng, 16, 65536))

    def cols():  # columns of the plain form
        return min(c["kv"], c["n"] + c["span"] if c["span"] else c["kv"]) + c["sinks"]

    while (c["B"] * Hq * c["n"] * cols() > MAX_LOGITS or 4.0 * d * Hq * c["B"] * c["n"] * cols() > MAX_FLOPS
           or c["B"] * cols() * Hk * d > MAX_CACHE or c["B"] * c["kv"] * Hk * d > 8 * MAX_CACHE):
        if c["B"] > 1:
            c["B"] //= 2
        else:
            c["kv"] = max(1, c["kv"] * 3 // 4)
            c["n"] = min(c["n"], c["kv"])
            c["n"] = max(1, c["n"] * 3 // 4)
    return c


def _lengths(case):
    """(tokens that the call is about, cached tokens with them) of every sequence."""
    n = case.get("n", 0)
    if not case["ragged"]:
        return [(n, case["kv"])] * case["B"]
    r = random.Random(case["lens"])
    out = []
    for s in range(case["B"]):
        m = n if s == 0 or n < 2 else r.randint(1, n)
        kv = case["kv"] if s == 0 else max(m, 1, int(case["kv"] * r.random() ** 1.5))
        out.append((m, kv))
    r.shuffle(out)
    return out


def _parents(case):
    """Of the drafted tokens of every sequence: an earlier one's number or -1."""
    r = random.Random(case["lens"] + 1)
    return [[min(int((j + 1) * r.random() ** 0.5), j) - 1 for j in range(n)] for n, _ in _lengths(case)]


def _depths(parents):
    out = []
    for p in parents:
        out.append(1 + out[p] if p >= 0 else 0)
    return out


def _first(case, n, kv, parents):
    """The first slot of the window of each of the n newest tokens of kv."""
    if not case["span"]:
        return [0] * n
    place = [kv - n + x for x in _depths(parents)] if case["op"] == "tree" else range(kv - n, kv)
    return [max(0, i - case["span"] + 1) for i in place]


def _sequences(case):
    lens = _lengths(case)
    trees = _parents(case) if case["op"] == "tree" else [None] * len(lens)
    return [(n, kv, _first(case, n, kv, p), p) for (n, kv), p in zip(lens, trees)]


def _kept(case):
    """The flags of every sequence's blocks."""
    r = random.Random(case["lens"] + 2)
    out = []
    for n, _ in _lengths(case):
        f = [r.random() < case["share"] for _ in range(-(-n // case["block"]))]
        f[-1] = case["block"] > 1 or f[-1]
        out.append(f)
    return out


def _fork_plan(case):
    r = random.Random(case["lens"] + 3)
    return [r.randrange(case["B"]) for _ in range(case["children"])]


def work(case):
    """Each input read once, each output written once; the products of the visible pairs."""
    Hk, d = case["Hk"], case["d"]
    lens = _lengths(case)
    if case["op"] == "compact":
        moved = flags = 0
        for (n, kv), f in zip(lens, _kept(case)):
            flags += len(f)
            b, gone = case["block"], False
            for i, keep in enumerate(f):
                gone = gone or not keep
                if keep and gone:
                    moved += min(n, (i + 1) * b) - i * b
        return {"bytes": 2.0 * moved * (2 * Hk * d * 2 + 4) + flags + 8.0 * len(lens), "flops": 0.0}
    if case["op"] == "fork":
        page, total = case["page"], 0
        for p in _fork_plan(case):
            kv = lens[p][1]
            pages = -(-kv // page)
            more = -(-(kv + case["grow"]) // page) - pages
            # the parent's entries and reference counts read, the child's written, the last page's rows copied;
            # all of it let go again
            total += 8 * pages + 8 * pages + 12 * more + 2 * (kv % page) * (2 * Hk * d * 2 + 4) + 12 * (pages + more)
        return {"bytes": float(total), "flops": 0.0}
    Hq, S = case["Hq"], case["sinks"]
    seen = pairs = T = 0
    for n, kv, first, parents in _sequences(case):
        T += n
        past = kv - n if parents is not None else None
        depth = _depths(parents) if parents is not None else None
        lo = min(first)
        seen += kv - lo + min(S, lo)
        for t in range(n):
            end = past if parents is not None else kv - n + t + 1
            f = min(first[t], end)
            pairs += end - f + min(S, f) + (depth[t] + 1 if parents is not None else 0)
    return {"bytes": 2.0 * seen * Hk * d * 2 + 2.0 * T * Hq * d * 2 + 4.0 * T * Hq, "flops": 4.0 * pairs * Hq * d}


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    """What an engine holds before the call: the cache with its shuffled pages, queries and
    their windows or trees; the flags of what is kept; the pool of pages and who forks whom."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]
    B, Hk, d, page = (case[k] for k in ("B", "Hk", "d", "page"))
    lens = _lengths(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def sums(v):
        return ints([0] + torch.tensor(v, dtype=torch.int64).cumsum(0).tolist())

    need = [-(-kv // page) for _, kv in lens]
    max_pages, num_pages = max(need) + 1, sum(need) + 1
    if case["op"] == "fork":
        max_pages = -(-(max(kv for _, kv in lens) + case["grow"]) // page)
        num_pages += case["children"] * (2 + -(-case["grow"] // page))
    order = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
    st = {"case": case, "k_pages": normal(num_pages, Hk, page, d), "v_pages": normal(num_pages, Hk, page, d),
          "pos_pages": torch.randint(0, 131072, (num_pages, page), generator=gen, device=dev, dtype=torch.int32),
          "table": table, "kv_lens": ints([kv for _, kv in lens]), "cu": sums([n for n, _ in lens])}
    if case["op"] == "compact":
        kept = _kept(case)
        st["keep"] = torch.tensor([x for f in kept for x in f], dtype=torch.uint8, device=dev)
        st["cu_blocks"] = sums([len(f) for f in kept])
        st["n_max"] = max(n for n, _ in lens)
        return st
    if case["op"] == "fork":
        st["refs"] = torch.zeros(num_pages, dtype=torch.int32, device=dev)
        st["refs"][order[:at].long()] = 1
        st["free"] = torch.cat([order[at:], order[:at]])
        st["num_free"] = ints([num_pages - at])
        st["parents"] = ints(_fork_plan(case))
        return st
    Hq, T, seqs = case["Hq"], sum(n for n, _ in lens), _sequences(case)
    # queries with some weight on few keys, as trained heads have
    st["q"] = normal(T, Hq, d) * 1.5
    st["scale"] = d ** -0.5
    # the cached tokens' positions: a compacted cache skips some; drafted tokens lie by their depth
    step = torch.randint(1, 3, (B, max_pages * page), generator=gen, device=dev, dtype=torch.int32)
    pos = step.cumsum(1, dtype=torch.int32)
    if case["op"] == "tree":
        for s, (n, kv, _, p) in enumerate(seqs):
            pos[s, kv - n:kv] = pos[s, kv - n] + ints(_depths(p))
        st["tree"] = ints([x for _, _, _, p in seqs for x in p])
    live = table.long() >= 0
    st["pos_pages"][table.long()[live]] = pos.view(B, max_pages, page)[live]
    last = torch.cat([torch.arange(kv - n, kv) + s * max_pages * page for s, (n, kv) in enumerate(lens)])
    st["q_pos"] = pos.reshape(-1)[last.to(dev)].contiguous()
    st["slopes"] = 2.0 ** -torch.linspace(3.0, 10.0, Hq, device=dev) if case["bias"] else None
    first = ints([x for _, _, f, _ in seqs for x in f])
    st["first"] = first if case["span"] else None
    if case["op"] == "chunk":
        end = torch.cat([torch.arange(kv - n, kv) + 1 for n, kv in lens]).to(dev, torch.int32)
        st["visible"] = torch.stack([first, end], 1).contiguous()
    st["n_max"] = max(n for n, _ in lens)
    st["columns"] = max(kv - min(f) for _, kv, f, _ in seqs)  # cached tokens behind the earliest window's start
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        import block_sparse_long_up_gb300 as up
        cache = up.PagedKV(st["k_pages"], st["v_pages"], st["table"], st["kv_lens"], st["pos_pages"])
        if op == "compact":
            lens = up.compact_kv(cache, st["cu"], st["keep"], cu_blocks=st["cu_blocks"], G=st["case"]["block"])
            return {"lens": lens, **_pages(st)}
        if op == "fork":
            pool, page = up.PagePool(st["refs"], st["free"], st["num_free"]), st["case"]["page"]
            table, lens, copies = up.fork_pages(pool, st["table"], st["kv_lens"], page, st["parents"])
            up.copy_pages(cache, copies)
            more = lens + st["case"]["grow"]
            up.reserve_pages(pool, table, page, lens, more)
            held = {"table": table.clone(), "lens": lens, "copies": copies, "shared": st["refs"].clone()}
            up.release_pages(pool, table, page, None, more)
            return {**held, "gone": table, "refs": st["refs"], "free": st["free"], "num_free": st["num_free"], **_pages(st)}
        more = dict(scale=st["scale"], softcap=st["case"]["softcap"], sinks=st["case"]["sinks"])
        if st["slopes"] is not None:
            more.update(slopes=st["slopes"], q_pos=st["q_pos"])
        if op == "token":
            out, lse = up.decode_attend(st["q"], cache, kv_start=st["first"], **more)
        elif op == "tree":
            out, lse = up.attend_tree(st["q"], st["cu"], st["tree"], cache, kv_start=st["first"], **more)
        else:
            out, lse = up.attend_paged(st["q"], st["cu"], cache, visible=st["visible"], **more)
        return {"out": out, "lse": lse}
    return _plain_compact(st) if op == "compact" else _plain_fork(st) if op == "fork" else _plain_attend(st)


def _pages(st):
    return {k: st[k] for k in ("k_pages", "v_pages", "pos_pages")}


def _plain_attend(st):
    case, cu, kv = st["case"], st["cu"].long(), st["kv_lens"].long()
    q = st["q"].float()
    T, Hq, d = q.shape
    B, Hk, page = st["table"].shape[0], st["k_pages"].shape[1], st["k_pages"].shape[2]
    N, g, S = st["n_max"], Hq // Hk, case["sinks"]
    t = torch.arange(T, device=q.device)
    s = (t[:, None] >= cu[None, 1:]).sum(1)
    n = cu[1:] - cu[:-1]
    j = t - cu[s]

    def padded(x, fill):
        y = torch.full((B, N) + x.shape[1:], fill, dtype=x.dtype, device=x.device)
        y[s, j] = x
        return y

    first = torch.zeros_like(t) if st["first"] is None else st["first"].long()
    # the columns: the first S slots, and what follows the earliest window's start
    start = torch.maximum(padded(first, 1 << 40).amin(1), torch.full_like(kv, S))
    slot = torch.cat([torch.arange(S, device=q.device).expand(B, S),
                      start[:, None] + torch.arange(st["columns"], device=q.device)], 1)
    there = slot < kv[:, None]
    at = torch.gather(st["table"].long(), 1, torch.where(there, slot, 0) // page).clamp(min=0)
    row = slot % page

    def cached(x):
        return x[at, :, row].transpose(1, 2).float()

    past = kv - n  # slots before the tokens of the call
    own_slot = past[s] + j
    lo = padded(first, 0)[..., None]
    i = slot[:, None, :]
    seen = ((i >= lo) | (i < S)) & there[:, None]
    if case["op"] == "tree":
        # who descends from whom: a path of any length
        up_to = torch.zeros(B, N, N + 1, dtype=torch.float64, device=q.device)
        up_to.scatter_(2, torch.where(padded(st["tree"], -1) < 0, N, padded(st["tree"], -1)).long()[..., None], 1.0)
        line = torch.matrix_power(torch.eye(N, dtype=torch.float64, device=q.device) + up_to[..., :N], N) > 0.5
        k = i - past[:, None, None]
        below = torch.gather(line, 2, k.clamp(0, N - 1).expand(B, N, -1))
        seen = torch.where(k < 0, seen, below & there[:, None])
    else:
        seen = seen & (i <= padded(own_slot, -1)[..., None])
    x = padded(q, 0.0).view(B, N, Hk, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * N, d)
    x = (x @ cached(st["k_pages"]).transpose(2, 3)).view(B, Hk, g, N, -1).mul_(st["scale"])
    if case["softcap"]:
        x = x.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    if st["slopes"] is not None:
        far = (padded(st["q_pos"], 0)[:, :, None] - st["pos_pages"][at, row][:, None, :]).abs().float()
        x -= st["slopes"].view(1, Hk, g, 1, 1) * far[:, None, None]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    v = cached(st["v_pages"]).masked_fill(~there[:, None, :, None], 0.0)
    y = (x.view(B, Hk, g * N, -1) @ v).view(B, Hk, g, N, d) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + z.log()).squeeze(-1)
    return {"out": y.permute(0, 3, 1, 2, 4)[s, j].reshape(T, Hq, d).to(st["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2)[s, j].reshape(T, Hq)}


def _plain_compact(st):
    cu, cb, kv, page = st["cu"].long(), st["cu_blocks"].long(), st["kv_lens"].long(), st["k_pages"].shape[2]
    N = st["n_max"]
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(N, device=cu.device)[None]
    flag = torch.minimum(cb[:-1, None] + i // st["case"]["block"], cb[1:, None] - 1)
    kept = (i < n) & (st["keep"].bool()[flag])
    rank = kept.cumsum(1) - kept.long()
    base = kv[:, None] - n
    s = torch.arange(cu.numel() - 1, device=cu.device)[:, None].expand_as(kept)
    s, src, to = s[kept], (base + i)[kept], (base + rank)[kept]
    ps, rs = st["table"].long()[s, src // page], src % page
    pd, rd = st["table"].long()[s, to // page], to % page
    st["k_pages"][pd, :, rd] = st["k_pages"][ps, :, rs]
    st["v_pages"][pd, :, rd] = st["v_pages"][ps, :, rs]
    st["pos_pages"][pd, rd] = st["pos_pages"][ps, rs]
    return {"lens": (base + kept.sum(1, keepdim=True)).squeeze(1).to(torch.int32), **_pages(st)}


def _plain_pop(st, need):
    """Fresh pages for the true entries of `need`, in order, and the pool without them."""
    flat = need.flatten().long()
    rank = flat.cumsum(0) - flat
    top = st["num_free"].long() - 1
    fresh = st["free"].long()[(top - rank).clamp(min=0)]
    st["num_free"] -= flat.sum().to(torch.int32)
    st["refs"].index_add_(0, fresh, flat.to(torch.int32))
    return fresh.view(need.shape).to(torch.int32)


def _plain_fork(st):
    case = st["case"]
    page, p = case["page"], st["parents"].long()
    lens = st["kv_lens"][p]
    full, rem = lens // page, lens % page
    j = torch.arange(st["table"].shape[1], device=p.device)[None]
    rows = st["table"][p]
    share = (j < full[:, None]) & (rows >= 0)
    st["refs"].index_add_(0, rows.long().clamp(min=0).flatten(), share.flatten().to(torch.int32))
    last = (j == full[:, None]) & (rem > 0)[:, None]
    fresh = _plain_pop(st, last)
    table = torch.where(share, rows, torch.where(last, fresh, torch.full_like(rows, -1)))
    none = torch.full_like(rem, -1)
    at = full.long().clamp(max=rows.shape[1] - 1)[:, None]
    copies = torch.stack([torch.where(rem > 0, rows.gather(1, at)[:, 0], none),
                          torch.where(rem > 0, table.gather(1, at)[:, 0], none), rem])
    # a child without a page of its own writes its first page, a shared one, onto itself
    src = torch.where(rem > 0, copies[0], table[:, 0]).long()
    dst = torch.where(rem > 0, copies[1], table[:, 0]).long()
    inside = torch.arange(page, device=p.device)[None] < rem[:, None]
    for x, mask in ((st["k_pages"], inside[:, None, :, None]), (st["v_pages"], inside[:, None, :, None]),
                    (st["pos_pages"], inside)):
        x[dst] = torch.where(mask, x[src], x[dst])
    # room for the next tokens
    more = lens + case["grow"]
    new = (j >= (-(-lens // page))[:, None]) & (j < (-(-more // page))[:, None])
    table = torch.where(new, _plain_pop(st, new), table)
    held = {"table": table, "lens": lens, "copies": copies, "shared": st["refs"].clone()}
    # the children go: pages that nobody holds any more return, the first entry's last
    out = (j < (-(-more // page))[:, None]) & (table >= 0)
    pages, flat = table.long().clamp(min=0).flatten(), out.flatten()
    num, big = st["refs"].numel(), 1 << 40
    st["refs"].index_add_(0, pages, -flat.to(torch.int32))
    order = torch.arange(flat.numel(), device=p.device)
    first = torch.full((num,), big, dtype=torch.long, device=p.device)
    first.scatter_reduce_(0, pages, torch.where(flat, order, torch.full_like(order, big)), "amin")
    gone = (first < big) & (st["refs"] == 0)
    rank = torch.where(gone, first, torch.full_like(first, -1)).argsort(descending=True).argsort()
    free = torch.cat([st["free"], st["free"][:1]])
    to = torch.where(gone, st["num_free"].long() + rank, torch.full_like(rank, num))
    free[to] = torch.arange(num, device=p.device, dtype=torch.int32)
    st["free"].copy_(free[:num])
    st["num_free"] += gone.sum().to(torch.int32)
    return {**held, "gone": torch.where(out, torch.full_like(table, -1), table), "refs": st["refs"], "free": st["free"],
            "num_free": st["num_free"], **_pages(st)}


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The same from the definitions, sequence by sequence, in 64 bits."""
    if work(case)["flops"] > 2e12:
        return None
    st = prepare(case, seed)
    page, lens = case["page"], _lengths(case)
    if case["op"] == "compact":
        out, new = {k: x.clone() for k, x in _pages(st).items()}, []
        table = st["table"].tolist()
        for s, ((n, kv), f) in enumerate(zip(lens, _kept(case))):
            src = [kv - n + i for i in range(n) if f[i // case["block"]]]
            to = list(range(kv - n, kv - n + len(src)))
            new.append(kv - n + len(src))
            a = torch.tensor([[table[s][i // page], i % page] for i in src] or [[0, 0]], device="cuda")
            b = torch.tensor([[table[s][i // page], i % page] for i in to] or [[0, 0]], device="cuda")
            for k in ("k_pages", "v_pages"):
                if src:
                    out[k][b[:, 0], :, b[:, 1]] = st[k][a[:, 0], :, a[:, 1]]
            if src:
                out["pos_pages"][b[:, 0], b[:, 1]] = st["pos_pages"][a[:, 0], a[:, 1]]
        out["k_pages"], out["v_pages"] = out["k_pages"].double(), out["v_pages"].double()
        return {"lens": torch.tensor(new, dtype=torch.int32), **out}
    if case["op"] == "fork":
        table, refs, free = st["table"].tolist(), st["refs"].tolist(), st["free"].tolist()
        top, width = int(st["num_free"]), st["table"].shape[1]
        out, new, size, copies = {k: x.clone() for k, x in _pages(st).items()}, [], [], []
        for p in _fork_plan(case):
            kv = lens[p][1]
            row = table[p][:kv // page]
            for x in row:
                refs[x] += 1
            if kv % page:
                top -= 1
                copies.append((table[p][kv // page], free[top], kv % page))
                refs[free[top]] = 1
                row.append(free[top])
                for k in ("k_pages", "v_pages"):
                    out[k][row[-1]][:, :kv % page] = st[k][copies[-1][0]][:, :kv % page]
                out["pos_pages"][row[-1]][:kv % page] = st["pos_pages"][copies[-1][0]][:kv % page]
            else:
                copies.append((-1, -1, 0))
            new.append(row)
            size.append(kv)
        for row, kv in zip(new, size):
            while len(row) * page < kv + case["grow"]:
                top -= 1
                refs[free[top]] = 1
                row.append(free[top])
        held, back = list(refs), []
        for row in new:
            for x in row:
                refs[x] -= 1
        seen = set()
        for x in (x for row in new for x in row):
            if refs[x] == 0 and x not in seen:
                seen.add(x)
                back.append(x)
        for x in reversed(back):
            free[top] = x
            top += 1
        full = torch.tensor([r + [-1] * (width - len(r)) for r in new], dtype=torch.int32)
        out["k_pages"], out["v_pages"] = out["k_pages"].double(), out["v_pages"].double()
        return {"table": full, "lens": torch.tensor(size, dtype=torch.int32),
                "copies": torch.tensor(copies, dtype=torch.int32).T.contiguous(), "shared": torch.tensor(held, dtype=torch.int32),
                "gone": torch.full_like(full, -1), "refs": torch.tensor(refs, dtype=torch.int32),
                "free": torch.tensor(free, dtype=torch.int32), "num_free": torch.tensor([top], dtype=torch.int32), **out}
    Hq, Hk, S = case["Hq"], case["Hk"], case["sinks"]
    g, t0 = Hq // Hk, 0
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (n, kv, first, parents) in enumerate(_sequences(case)):
        at = st["table"][b, :-(-kv // page)].long()
        place = st["pos_pages"][at].flatten()[:kv].double()
        i = torch.arange(kv, device="cuda")
        if parents is not None:
            line = torch.zeros(n, kv, dtype=torch.bool)
            line[:, :kv - n] = True
            for t, p in enumerate(parents):
                if p >= 0:
                    line[t] = line[p]
                line[t, kv - n + t] = True
            line = line.cuda()
        for h in range(Hq):
            keys = st["k_pages"][at, h // g].flatten(0, 1)[:kv].double()
            vals = st["v_pages"][at, h // g].flatten(0, 1)[:kv].double()
            for a in range(0, n, 1024):
                rows, m = slice(t0 + a, t0 + min(n, a + 1024)), min(n, a + 1024) - a
                lo = torch.tensor(first[a:a + m], device="cuda")[:, None]
                j = slice(max(0, int(lo.min())), kv)
                cols = torch.cat([i[:min(S, j.start)], i[j]])
                z = (st["q"][rows, h].double() @ keys[cols].T) * st["scale"]
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                if case["bias"]:
                    z = z - st["slopes"][h].double() * (st["q_pos"][rows].double()[:, None] - place[cols]).abs()
                seen = (cols >= lo) | (cols < S)
                if parents is None:
                    seen = seen & (cols <= torch.arange(kv - n + a, kv - n + a + m, device="cuda")[:, None])
                else:
                    seen = (seen | (cols >= kv - n)) & line[a:a + m][:, cols]
                z = z.masked_fill(~seen, -math.inf)
                lse[rows, h] = torch.logsumexp(z, 1)
                some = seen.any(1, keepdim=True)
                out[rows, h] = torch.where(some, torch.softmax(z, 1), torch.zeros_like(z)) @ vals[cols]
        t0 += n
    return {"out": out, "lse": lse}
