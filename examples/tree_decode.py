"""Speculative decoding with trees of drafted tokens, over one pool of pages.

A small random-weight decoder reads a batch of prompts, every layer with its own paged cache
and all of them with one block table.  Each prompt is then forked: its
continuations share the prompt's full pages and differ in their first token.  A step drafts
a tree of tokens for every continuation (guesses without the layers), runs all layers on
the tree at once (append_kv, attend_tree), walks down the tree as far as the model agrees,
moves the accepted path together in every cache (compact_kv) and lets go of the pages
behind it.  Lengths, tables and the pool stay on the device; a step is one CUDA graph.

    python examples/tree_decode.py [--prompt 900 333] [--children 2] [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_sparse_long_up_gb300 as up  # noqa: E402

HIDDEN, HQ, HK, D, LAYERS, VOCAB, PAGE = 256, 8, 2, 64, 3, 500, 16
# the drafted tree: the last token, two guesses behind it, two behind each, one behind the first of these
PARENTS = [-1, 0, 0, 1, 1, 2, 2, 3]
CHILD = [0, 0, 1, 0, 1, 0, 1, 0]  # which of its parent's guesses a token is
DEPTH = 4


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Model:
    def __init__(self, gen, pages, table, lens):
        def w(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[0] ** -0.5).bfloat16()
        self.embed = torch.randn(VOCAB, HIDDEN, generator=gen, device="cuda").bfloat16()
        self.head = self.embed[torch.randperm(VOCAB, generator=gen, device="cuda")].T.contiguous()
        self.layers = [(w(HIDDEN, (HQ + 2 * HK) * D), w(HQ * D, HIDDEN), w(HIDDEN, 2 * HIDDEN), w(2 * HIDDEN, HIDDEN))
                       for _ in range(LAYERS)]
        self.stores = [(torch.empty(pages, HK, PAGE, D, dtype=torch.bfloat16, device="cuda"),
                        torch.empty(pages, HK, PAGE, D, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(pages, PAGE, dtype=torch.int32, device="cuda")) for _ in range(LAYERS)]
        self.inv_freq = 10000.0 ** -(torch.arange(0, D, 2, device="cuda") / D)
        self.use(table, lens)

    def use(self, table, lens):
        """The sequences that the next calls are about."""
        self.table, self.lens = table, lens
        self.caches = [up.PagedKV(k, v, table, lens, p) for k, v, p in self.stores]

    def run(self, tokens, pos, cu, parents=None):
        """Logits of new tokens, whose slots kv_lens counts; in a tree if they have parents."""
        x, t = self.embed[tokens], tokens.numel()
        for (qkv, o, wide, narrow), cache in zip(self.layers, self.caches):
            q, k, v = (y.view(t, -1, D) for y in (norm(x) @ qkv).split([HQ * D, HK * D, HK * D], 1))
            q = up.append_kv(q, k, v, pos, cu, cache, self.inv_freq)
            a, _ = up.attend_paged(q, cu, cache) if parents is None else up.attend_tree(q, cu, parents, cache)
            x = x + a.reshape(t, HQ * D) @ o
            x = x + torch.nn.functional.silu(norm(x) @ wide) @ narrow
        return norm(x) @ self.head


def ancestors(j):
    return [] if PARENTS[j] < 0 else [PARENTS[j]] + ancestors(PARENTS[j])


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, nargs="+", default=[900, 333])
    ap.add_argument("--children", type=int, default=2)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    P, N, n = len(a.prompt), len(a.prompt) * a.children, len(PARENTS)
    most = max(a.prompt) + a.steps * DEPTH + n
    width = -(-most // PAGE)
    pages = sum(-(-x // PAGE) for x in a.prompt) + N * (2 + -(-(a.steps * DEPTH + n) // PAGE))
    pool = up.PagePool.full(pages)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    # the prompts
    table, lens = torch.full((P, width), -1, dtype=torch.int32, device="cuda"), ints(a.prompt)
    up.reserve_pages(pool, table, PAGE, torch.zeros_like(lens), lens)
    model = Model(gen, pages, table, lens)
    cu = torch.cat([ints([0]), lens.cumsum(0, dtype=torch.int32)])
    ids = torch.randint(0, VOCAB, (sum(a.prompt),), generator=gen, device="cuda")
    logits = model.run(ids, torch.cat([torch.arange(x, dtype=torch.int32, device="cuda") for x in a.prompt]), cu)
    first = logits[cu[1:].long() - 1].topk(a.children).indices  # a first token for each child

    # their continuations
    t2, l2, copies = up.fork_pages(pool, table, lens, PAGE, torch.arange(P, dtype=torch.int32, device="cuda").repeat_interleave(a.children))
    for cache in model.caches:
        up.copy_pages(cache, copies)
    up.release_pages(pool, table, PAGE, None, lens)  # the children hold what they share
    model.use(t2, l2)
    root = first.flatten().clone()

    cu = torch.arange(0, (N + 1) * n, n, dtype=torch.int32, device="cuda")
    parents = ints(PARENTS * N)
    up_to = torch.tensor(PARENTS, device="cuda")
    depth = ints([len(ancestors(j)) for j in range(n)]).repeat(N)
    out = torch.full((N, DEPTH), -1, device="cuda")

    def step():
        # the draft: guesses from the embedding alone
        tree = [root]
        for j in range(1, n):
            tree.append((norm(model.embed[tree[PARENTS[j]]]) @ model.head).topk(2).indices[:, CHILD[j]])
        tokens = torch.stack(tree, 1)
        old = l2.clone()
        up.reserve_pages(pool, t2, PAGE, old, old + n)
        l2.add_(n)
        best = model.run(tokens.flatten(), old.repeat_interleave(n) + depth, cu, parents).argmax(-1).view(N, n)
        # down the tree while the model's choice is among the guesses
        at = torch.zeros(N, dtype=torch.long, device="cuda")
        on = torch.ones(N, dtype=torch.bool, device="cuda")
        keep = torch.zeros(N, n, dtype=torch.uint8, device="cuda")
        out.fill_(-1)
        for d in range(DEPTH):
            keep.scatter_(1, at[:, None], 1)
            choice = best.gather(1, at[:, None])
            out[:, d] = torch.where(on, choice[:, 0], out[:, d])
            hit = (up_to[None] == at[:, None]) & (tokens == choice) & on[:, None]
            on = hit.any(1)
            at = torch.where(on, hit.int().argmax(1), at)
        root.copy_(best.gather(1, at[:, None])[:, 0])
        whole = l2.clone()
        for cache in model.caches:
            new = up.compact_kv(cache, cu, keep.view(-1))
        l2.copy_(new)
        up.release_pages(pool, t2, PAGE, l2, whole)

    step()  # warm-up, a real step
    said = [out.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(a.steps - 1):
        graph.replay()
        said.append(out.clone())
    torch.cuda.synchronize()
    tokens = [[int(f)] + [t for t in row if t >= 0]
              for f, row in zip(first.flatten(), torch.cat(said, 1).tolist())]
    up.release_pages(pool, t2, PAGE, None, l2)
    if up.get_device_error() or int(pool.num_free) != pages:
        raise RuntimeError("the device reported an error, or pages were lost")
    for s, t in enumerate(tokens):
        print(f"prompt {s // a.children}, continuation {s % a.children}: {len(t)} tokens in {a.steps} steps: {t}")
    return tokens


if __name__ == "__main__":
    main()
