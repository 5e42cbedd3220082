"""What the paged-cache operators are measured on: appending rotated keys and values to a
paged KV-head-major cache, attention of a chunk of new tokens over such a cache, and
attention of one new token per sequence.

`own` selects what run() computes with: False, the operators' plain form in elementary
torch operations; True, the library's calls.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------- the cases

# Elements of the plain form's padded logits and key-value copies: what a drawn case may cost.
MAX_LOGITS = 32 * 2048 * 65536
MAX_FLOPS = 4.4e12


def listed():
    """Head layouts 32/8 x 128, 16/2 x 256 and 8/2 x 64 and the length sets are those of the
    repository's own workloads (128K, 32K and 4K tokens, eight mixed lengths up to 128K)."""
    return [
        # one decode step of one conversation near its 128K limit: pure latency
        dict(name="append_step_b1", op="append", dtype="bf16", B=1, Hq=32, Hk=8, d=128, page=256,
             n=1, kv=131072, ragged=False, lens=1, rot=128, interleaved=False, axes=1),
        # one decode step of 64 conversations, pair-interleaved rotation of a part of the head
        dict(name="append_step_b64", op="append", dtype="fp16", B=64, Hq=16, Hk=2, d=256, page=64,
             n=1, kv=20011, ragged=True, lens=2, rot=64, interleaved=True, axes=1),
        # a 32K prompt's layer
        dict(name="append_prompt_32k", op="append", dtype="bf16", B=1, Hq=32, Hk=8, d=128, page=256,
             n=32768, kv=32768, ragged=False, lens=3, rot=128, interleaved=False, axes=1),
        # eight ragged prompts with image patches: time, height and width positions
        dict(name="append_mixed_axes", op="append", dtype="bf16", B=8, Hq=8, Hk=2, d=64, page=16,
             n=4099, kv=9001, ragged=True, lens=4, rot=64, interleaved=False, axes=3),
        # one conversation of 4K tokens: latency
        dict(name="decode_b1_4k", op="decode", dtype="bf16", B=1, Hq=8, Hk=2, d=64, page=128,
             n=1, kv=4096, ragged=False, lens=5, softcap=0.0, bias=False, mask="causal", span=0),
        # one conversation at 128K: the cache's length has to be split
        dict(name="decode_b1_128k", op="decode", dtype="bf16", B=1, Hq=32, Hk=8, d=128, page=256,
             n=1, kv=131072, ragged=False, lens=6, softcap=0.0, bias=False, mask="causal", span=0),
        # a serving batch of mixed lengths up to 128K
        dict(name="decode_b24_mixed", op="decode", dtype="bf16", B=24, Hq=32, Hk=8, d=128, page=256,
             n=1, kv=131072, ragged=True, lens=7, softcap=0.0, bias=False, mask="causal", span=0),
        # capped scores, a sliding window and a distance bias at head_dim 256, small pages
        dict(name="decode_b48_window", op="decode", dtype="fp16", B=48, Hq=16, Hk=2, d=256, page=16,
             n=1, kv=30011, ragged=True, lens=8, softcap=30.0, bias=True, mask="window", span=4096),
        # a short chunk on a short cache: latency
        dict(name="attend_chunk_128", op="attend", dtype="bf16", B=1, Hq=8, Hk=2, d=64, page=128,
             n=128, kv=4096, ragged=False, lens=9, softcap=0.0, bias=False, mask="causal", span=0),
        # a chunk of a long prompt over the chunks before it
        dict(name="attend_chunk_64k", op="attend", dtype="bf16", B=1, Hq=32, Hk=8, d=128, page=256,
             n=2048, kv=65536, ragged=False, lens=10, softcap=0.0, bias=False, mask="causal", span=0),
        # a batch of ragged prompts whole, documents packed inside them
        dict(name="attend_prompts_docs", op="attend", dtype="bf16", B=6, Hq=32, Hk=8, d=128, page=128,
             n=5003, kv=5003, ragged=True, lens=11, softcap=0.0, bias=False, mask="docs", span=1500),
        # head_dim 256 with capped scores, a distance bias and a bidirectional prefix
        dict(name="attend_prefix_capped", op="attend", dtype="fp16", B=3, Hq=16, Hk=2, d=256, page=64,
             n=1777, kv=8191, ragged=True, lens=12, softcap=50.0, bias=True, mask="prefix", span=700),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: steps and prompts, caches of one token to 128K, every
    head layout, page size, type, rotation and mask."""
    op = rng.choice(["append", "decode", "attend"])
    Hq, Hk = rng.choice([(32, 8), (16, 2), (8, 2), (8, 8), (12, 4), (16, 1)])
    d = rng.choice([64, 128, 256])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), B=_log_int(rng, 1, 48), Hq=Hq, Hk=Hk,
             d=d, page=rng.choice([16, 32, 48, 64, 128, 256, 384]), ragged=rng.random() < 0.7,
             lens=rng.randrange(1 << 30))
    if op == "append":
        step = rng.random() < 0.4
        c["n"] = 1 if step else _log_int(rng, 2, min(32768, max(2, 32768 // c["B"] * 128 // d)))
        c["kv"] = c["n"] + _log_int(rng, 1, 30000) - 1
        c["rot"] = rng.choice([d, d, d // 2, d // 4])
        c["interleaved"] = rng.random() < 0.4
        c["axes"] = rng.choice([1, 1, 3])
        # the cache that the tokens are written to stays of a size with the others
        while c["B"] * c["kv"] * Hk * d > 1 << 30:
            c["kv"] = max(c["n"], c["kv"] // 2)
            c["B"] = max(1, c["B"] - 1)
        return c
    c["softcap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    c["bias"] = rng.random() < 0.25
    c["mask"] = rng.choice(["causal", "causal", "window"] + (["docs", "prefix"] if op == "attend" else []))
    c["span"] = _log_int(rng, 16, 8192)
    if op == "decode":
        c["n"], c["kv"] = 1, _log_int(rng, 1, 131072)
        while c["B"] * c["kv"] * Hk * d > 24 * 131072 * 8 * 128:
            c["B"] = max(1, c["B"] // 2)
        return c
    c["B"] = min(c["B"], 8)
    c["n"] = _log_int(rng, 2, 6000)
    c["kv"] = max(c["n"], _log_int(rng, 16, 65536))
    while c["B"] * Hq * c["n"] * c["kv"] > MAX_LOGITS or 4.0 * d * c["B"] * Hq * c["n"] * c["kv"] > MAX_FLOPS:
        c["B"] = max(1, c["B"] // 2)
        c["n"] = max(1, c["n"] * 3 // 4)
        c["kv"] = max(c["n"], c["kv"] * 3 // 4)
    return c


def _lengths(case):
    """(new tokens, cached tokens with them) of every sequence."""
    if not case["ragged"]:
        return [(case["n"], case["kv"])] * case["B"]
    r = random.Random(case["lens"])
    out = []
    for s in range(case["B"]):
        n = case["n"] if s == 0 or case["n"] == 1 else r.randint(1, case["n"])
        kv = case["kv"] if s == 0 else max(n, int(case["kv"] * r.random() ** 1.5))
        out.append((n, kv))
    r.shuffle(out)
    return out


def _visible(case, n, kv):
    """First visible slot and the end of the visible slots of the n newest of kv tokens."""
    i = torch.arange(kv - n, kv, dtype=torch.int64)
    lo, hi, w = torch.zeros_like(i), i + 1, case["span"]
    if case["mask"] == "window":
        lo = (i - w + 1).clamp(min=0)
    elif case["mask"] == "docs":
        lo = i // w * w
    elif case["mask"] == "prefix":
        hi = torch.maximum(hi, torch.full_like(hi, min(w, kv)))
    return lo, hi


def work(case):
    """Each input read once, each output written once; the products of the visible pairs."""
    lens, size = _lengths(case), 2
    T = sum(n for n, _ in lens)
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "append":
        rows = T * (Hq + 2 * Hk)
        return {"bytes": 2.0 * rows * d * size + 4.0 * T * (case["axes"] + 1),
                "flops": 6.0 * T * (Hq + Hk) * case["rot"] / 2}
    seen = pairs = 0
    for n, kv in lens:
        lo, hi = _visible(case, n, kv)
        seen += int(hi.max() - lo.min())
        pairs += int((hi - lo).sum())
    return {"bytes": 2.0 * seen * Hk * d * size + 2.0 * T * Hq * d * size + 4.0 * T * Hq,
            "flops": 4.0 * pairs * Hq * d}


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    """What an engine holds before the call: the projections of the new tokens (views of one
    fused row for the append), their positions, and the cache with its shuffled pages."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]
    lens = _lengths(case)
    B, Hq, Hk, d, page = (case[k] for k in ("B", "Hq", "Hk", "d", "page"))
    T = sum(n for n, _ in lens)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    max_pages = -(-max(kv for _, kv in lens) // page) + 1
    num_pages = sum(-(-kv // page) for _, kv in lens) + 1
    order = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, (_, kv) in enumerate(lens):
        k = -(-kv // page)
        table[s, :k] = order[at:at + k]
        at += k
    st = {"case": case, "k_pages": normal(num_pages, Hk, page, d), "v_pages": normal(num_pages, Hk, page, d),
          "pos_pages": torch.zeros(num_pages, page, dtype=torch.int32, device=dev), "table": table,
          "kv_lens": ints([kv for _, kv in lens]),
          "cu": ints([0] + torch.tensor([n for n, _ in lens]).cumsum(0).tolist()),
          "n_max": max(n for n, _ in lens), "kv_max": max(kv for _, kv in lens)}
    if case["op"] == "append":
        x = normal(T, (Hq + 2 * Hk) * d)
        st["q"] = x[:, :Hq * d].view(T, Hq, d)
        st["k"] = x[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
        st["v"] = x[:, (Hq + Hk) * d:].view(T, Hk, d)
        index = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).to(dev, torch.int32)
        if case["axes"] == 1:
            st["pos"] = index
            st["axes"] = None
        else:  # image patches: rows and columns of a 48-wide grid beside the time
            st["pos"] = torch.stack([index // 1024, index % 1024 // 48, index % 48]).contiguous()
            st["axes"] = torch.arange(case["rot"] // 2, device=dev, dtype=torch.int32) % 3
        half = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"]
        st["inv_freq"] = (500000.0 ** -half).float()
        return st
    # queries with some weight on few keys, as trained heads have
    st["q"] = normal(T, Hq, d) * 1.5
    st["scale"] = d ** -0.5
    # the cached tokens' positions: a compacted cache skips some
    step = torch.randint(1, 3, (B, max_pages * page), generator=gen, device=dev, dtype=torch.int32)
    pos = step.cumsum(1, dtype=torch.int32)
    live = table.long() >= 0
    st["pos_pages"][table.long()[live]] = pos.view(B, max_pages, page)[live]
    last = torch.cat([torch.arange(kv - n, kv) + s * max_pages * page for s, (n, kv) in enumerate(lens)])
    st["q_pos"] = pos.reshape(-1)[last.to(dev)]
    st["slopes"] = 2.0 ** -torch.linspace(3.0, 10.0, Hq, device=dev) if case["bias"] else None
    if case["op"] == "decode":
        st["kv_start"] = None if case["mask"] == "causal" else ints(
            [int(_visible(case, 1, kv)[0]) for _, kv in lens])
    else:
        st["visible"] = None if case["mask"] == "causal" else torch.cat(
            [torch.stack(_visible(case, n, kv), 1) for n, kv in lens]).to(dev, torch.int32)
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        import block_sparse_long_up_gb300 as up
        cache = up.PagedKV(st["k_pages"], st["v_pages"], st["table"], st["kv_lens"], st["pos_pages"])
        if op == "append":
            q = up.append_kv(st["q"], st["k"], st["v"], st["pos"], st["cu"], cache, st["inv_freq"],
                             axes=st["axes"], interleaved=st["case"]["interleaved"])
            return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"], "pos_pages": st["pos_pages"]}
        more = dict(scale=st["scale"], softcap=st["case"]["softcap"])
        if st["slopes"] is not None:
            more.update(slopes=st["slopes"], q_pos=st["q_pos"])
        if op == "decode":
            out, lse = up.decode_attend(st["q"], cache, kv_start=st["kv_start"], **more)
        else:
            out, lse = up.attend_paged(st["q"], st["cu"], cache, visible=st["visible"], **more)
        return {"out": out, "lse": lse}
    return _plain_append(st) if op == "append" else _plain_attend(st)


def _tokens(st):
    """Sequence and slot of every new token."""
    cu = st["cu"].long()
    t = torch.arange(st["q"].shape[0], device=cu.device)
    s = (t[:, None] >= cu[None, 1:]).sum(1)
    return s, st["kv_lens"].long()[s] - cu[s + 1] + t, t - cu[s]


def _rotate(x, cos, sin, interleaved):
    """Pairs (2i, 2i+1) or (i, i + rot/2) of the first rot dims turned by their angles."""
    half = cos.shape[-1]
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., :2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_append(st):
    s, slot, _ = _tokens(st)
    page = st["k_pages"].shape[2]
    to, row = st["table"].long()[s, slot // page], slot % page
    pos = st["pos"]
    first = pos if pos.dim() == 1 else pos[0]
    at = first[:, None] if st["axes"] is None else pos[st["axes"].long()].T
    angle = at.double() * st["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    turn = st["case"]["interleaved"]
    q = _rotate(st["q"], cos, sin, turn).to(st["q"].dtype)
    st["k_pages"][to, :, row] = _rotate(st["k"], cos, sin, turn).to(st["q"].dtype)
    st["v_pages"][to, :, row] = st["v"]
    st["pos_pages"][to, row] = first
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"], "pos_pages": st["pos_pages"]}


def _plain_attend(st):
    s, slot, t = _tokens(st) if st["case"]["op"] == "attend" else (
        torch.arange(st["q"].shape[0], device="cuda"), st["kv_lens"].long() - 1, 0)
    q = st["q"].float()
    T, Hq, d = q.shape
    B, Hk, page, L = st["table"].shape[0], st["k_pages"].shape[1], st["k_pages"].shape[2], st["kv_max"]
    N, g = st["n_max"], Hq // Hk
    pages = st["table"].long()[:, :-(-L // page)].clamp(min=0)

    def cached(x):
        return x[pages].transpose(1, 2).flatten(2, 3)[:, :, :L].float()

    def padded(x, fill):
        y = torch.full((B, N) + x.shape[1:], fill, dtype=x.dtype, device=x.device)
        y[s, t] = x
        return y

    lo, hi = torch.zeros_like(slot), slot + 1
    if st.get("kv_start") is not None:
        lo = st["kv_start"].long()
    if st.get("visible") is not None:
        lo, hi = st["visible"].long().unbind(1)
    hi = torch.minimum(hi, st["kv_lens"].long()[s])
    x = padded(q, 0.0).view(B, N, Hk, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * N, d)
    x = (x @ cached(st["k_pages"]).transpose(2, 3)).view(B, Hk, g, N, L).mul_(st["scale"])
    if st["case"]["softcap"]:
        x = x.div_(st["case"]["softcap"]).tanh_().mul_(st["case"]["softcap"])
    if st["slopes"] is not None:
        kp = st["pos_pages"][pages].flatten(1)[:, :L]
        far = (padded(st["q_pos"], 0)[:, :, None] - kp[:, None, :]).abs().float()
        x -= st["slopes"].view(1, Hk, g, 1, 1) * far[:, None, None]
    i = torch.arange(L, device=x.device)
    out = (i < padded(lo, 0)[..., None]) | (i >= padded(hi, 0)[..., None])
    x = x.masked_fill_(out[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    y = (x.view(B, Hk, g * N, L) @ cached(st["v_pages"])).view(B, Hk, g, N, d) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + z.log()).squeeze(-1)
    return {"out": y.permute(0, 3, 1, 2, 4)[s, t].reshape(T, Hq, d).to(st["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2)[s, t].reshape(T, Hq)}


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The same from the definitions, token by token's sequence, in 64 bits."""
    if work(case)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    Hq, Hk, d, page = (case[k] for k in ("Hq", "Hk", "d", "page"))
    lens, g = _lengths(case), case["Hq"] // case["Hk"]
    if case["op"] == "append":
        kp, vp, q = st["k_pages"].double(), st["v_pages"].double(), st["q"].double().clone()
        pp = st["pos_pages"].clone()
        pos = st["pos"].view(case["axes"], -1).double()
        half = case["rot"] // 2
        phase = torch.stack([pos[i % case["axes"]] * st["inv_freq"][i].double() for i in range(half)], 1)
        turn = torch.polar(torch.ones_like(phase), phase)[:, None]
        one = torch.arange(half, device=q.device) * (2 if case["interleaved"] else 1)
        two = one + (1 if case["interleaved"] else half)
        k = st["k"].double().clone()
        for x in (q, k):
            z = torch.complex(x[..., one], x[..., two]) * turn
            x[..., one], x[..., two] = z.real, z.imag
        t0 = 0
        for b, (n, kv) in enumerate(lens):
            for a in range((kv - n) // page, -(-kv // page)):
                r0, r1 = max(kv - n, a * page), min(kv, (a + 1) * page)
                at, rows, new = int(st["table"][b, a]), slice(r0 - a * page, r1 - a * page), slice(t0 + r0 - kv + n, t0 + r1 - kv + n)
                kp[at][:, rows] = k[new].transpose(0, 1)
                vp[at][:, rows] = st["v"][new].transpose(0, 1).double()
                pp[at][rows] = pos[0, new].int()
            t0 += n
        return {"q": q, "k_pages": kp, "v_pages": vp, "pos_pages": pp}
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, kv) in enumerate(lens):
        at = st["table"][b, :-(-kv // page)].long()
        i = torch.arange(kv, device="cuda")
        lo, hi = (x.to("cuda") for x in _visible(case, n, kv))
        place = st["pos_pages"][at].flatten()[:kv].double()
        for h in range(Hq):
            keys = st["k_pages"][at, h // g].flatten(0, 1)[:kv].double()
            vals = st["v_pages"][at, h // g].flatten(0, 1)[:kv].double()
            for a in range(0, n, 2048):
                rows = slice(t0 + a, t0 + min(n, a + 2048))
                z = torch.einsum("td,kd->tk", st["q"][rows, h].double(), keys) * st["scale"]
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                if case["bias"]:
                    z = z - st["slopes"][h].double() * (st["q_pos"][rows].double()[:, None] - place[None]).abs()
                seen = (i[None] >= lo[a:a + 2048, None]) & (i[None] < hi[a:a + 2048, None])
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                lse[rows, h] = torch.logsumexp(z, 1)
                out[rows, h] = torch.softmax(z, 1) @ vals
        t0 += n
    return {"out": out, "lse": lse}
