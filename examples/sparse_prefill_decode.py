"""Prefill with dropped tokens, then decode, over one paged cache per layer.

A small random-weight decoder runs a batch of prompts: the first layer sees every
token, its last queries score the key blocks, and the layers behind it keep only the
selected tokens (score -> select -> compact).  Every layer appends its rotated keys,
values and positions to its own paged cache and attends over it; the kept tokens
keep their positions.  Then tokens are decoded one step at a time, each a call per
layer of append_kv and decode_attend, captured once in a CUDA graph.

    python examples/sparse_prefill_decode.py [--prompt 6000 2500] [--steps 32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_sparse_long_up_gb300 as up  # noqa: E402

HIDDEN, HQ, HK, D, LAYERS, VOCAB = 512, 8, 2, 64, 4, 1000
PAGE, WINDOW, BLOCK, MASS = 128, 128, 64, 0.99


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Layer:
    def __init__(self, gen, max_pages, num_seqs):
        def w(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[0] ** -0.5).bfloat16()
        self.qkv, self.o = w(HIDDEN, (HQ + 2 * HK) * D), w(HQ * D, HIDDEN)
        self.up, self.down = w(HIDDEN, 2 * HIDDEN), w(2 * HIDDEN, HIDDEN)
        kp = torch.empty(num_seqs * max_pages, HK, PAGE, D, dtype=torch.bfloat16, device="cuda")
        table = torch.arange(num_seqs * max_pages, dtype=torch.int32, device="cuda").view(num_seqs, max_pages)
        self.kv_lens = torch.zeros(num_seqs, dtype=torch.int32, device="cuda")
        pos = torch.zeros(num_seqs * max_pages, PAGE, dtype=torch.int32, device="cuda")
        self.cache = up.PagedKV(kp, torch.empty_like(kp), table, self.kv_lens, pos)

    def attend(self, x, pos, cu, inv_freq):
        """Attention of the new tokens x (packed by cu), appended to the cache first;
        returns the layer's output and the rotated queries."""
        t = x.shape[0]
        p = norm(x) @ self.qkv
        q, k, v = (y.view(t, -1, D) for y in p.split([HQ * D, HK * D, HK * D], 1))
        if t == self.cache.num_seqs:  # one token per sequence
            self.kv_lens += 1
            q = up.append_kv(q, k, v, pos, cu, self.cache, inv_freq)
            a, _ = up.decode_attend(q, self.cache)
        else:
            self.kv_lens += cu[1:] - cu[:-1]
            q = up.append_kv(q, k, v, pos, cu, self.cache, inv_freq)
            a, _ = up.attend_paged(q, cu, self.cache)
        x = x + a.reshape(t, HQ * D) @ self.o
        return x + torch.nn.functional.silu(norm(x) @ self.up) @ self.down, q


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, nargs="+", default=[6000, 2500])
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    lens, B = a.prompt, len(a.prompt)
    max_pages = -(-(max(lens) + a.steps + 2) // PAGE)
    layers = [Layer(gen, max_pages, B) for _ in range(LAYERS)]
    embed = torch.randn(VOCAB, HIDDEN, generator=gen, device="cuda").bfloat16()
    inv_freq = 10000.0 ** -(torch.arange(0, D, 2, device="cuda") / D)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    ids = torch.randint(0, VOCAB, (sum(lens),), generator=gen, device="cuda")
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens]).to(torch.int32)

    # prefill: the first layer on every token, the others on the kept ones
    x, q = layers[0].attend(embed[ids], pos, cu, inv_freq)
    ends = cu[1:].tolist()
    q_last = torch.cat([q[e - min(WINDOW, n):e] for e, n in zip(ends, lens)])
    c = layers[0].cache
    scores, cu_blocks = up.score_blocks_paged(q_last, c.k_pages, c.block_table, cu, sum(lens), WINDOW, BLOCK)
    # the last block stays: decoding goes on from the prompt's last token
    keep, kept = up.select_blocks(scores, cu_blocks, cu, BLOCK, p=MASS, keep_last=True)
    x, pos, cu, total, _ = up.compact(x, pos, cu, BLOCK, keep, cu_blocks)
    n = int(total)
    x, pos = x[:n], pos[:n]
    for layer in layers[1:]:
        x, _ = layer.attend(x, pos, cu, inv_freq)
    print(f"prefill: {sum(lens)} tokens, {n} kept behind the first layer")

    # decode: one captured step, replayed
    token = (norm(x[cu[1:].long() - 1]) @ embed.T).argmax(-1)
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def step():
        y = embed[token]
        for layer in layers:
            y, _ = layer.attend(y, at, one, inv_freq)
        token.copy_((norm(y) @ embed.T).argmax(-1))
        at.add_(1)

    step()  # warm-up, a real step
    out = [token.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(a.steps - 1):
        graph.replay()
        out.append(token.clone())
    torch.cuda.synchronize()
    if up.get_device_error():
        raise RuntimeError("the device reported an error")
    tokens = torch.stack(out, 1).tolist()
    for s, t in enumerate(tokens):
        print(f"sequence {s}: {t}")
    return tokens


if __name__ == "__main__":
    main()
