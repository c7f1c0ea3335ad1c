"""A decoder layer's attention over a 4-bit key/value cache, prompt and tokens, on cuda:0.

    python examples/kv_cache_decode.py [--fmt e2m1|e4m3] [--tokens N]

Sequences of unequal length come in as prompts: their keys and values are written
into pages as they are projected, the prompts attend over the cache, and then every
sequence takes one token at a time -- write its key and value, attend over what is
there -- as one HIP graph that is replayed.  An encoder's states are written once and
attended to by every step (cross attention).  At the end one sequence's cache is read
back, and the last step's result compared with attention over the unquantised keys
and values.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_fp8_casting_amd as nc  # noqa: E402

HEADS, GROUP, DIM, PAGE = 8, 4, 128, 64


class Pages:
    """Hands out pages of a cache to sequences; the table and lengths live on the GPU."""

    def __init__(self, cache: nc.KvCache, batch: int, most: int):
        self.cache, self.free = cache, list(range(cache.pages))
        self.host = torch.zeros((batch, -(-most // cache.page)), dtype=torch.int32)
        self.table = self.host.cuda()
        self.len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.have = [0] * batch

    def grow(self, tokens):
        """Room for so many tokens of every sequence."""
        for b, n in enumerate(tokens):
            while self.have[b] * self.cache.page < n:
                self.host[b, self.have[b]] = self.free.pop()
                self.have[b] += 1
        self.table.copy_(self.host)

    def slots(self, seq, pos):
        """Slots of tokens pos of sequences seq (int64 tensors on the GPU)."""
        return self.table[seq, pos // self.cache.page].long() * self.cache.page + pos % self.cache.page


def reference(q, k, v):
    """Attention of one query [heads * group, dim] over [tokens, heads, dim], fp32."""
    k, v = (x.float().repeat_interleave(GROUP, 1).transpose(0, 1) for x in (k, v))
    w = torch.softmax((k * q.float()[:, None]).sum(-1) / math.sqrt(DIM), -1)
    return (w[..., None] * v).sum(1)


def run(fmt="e2m1", prompts=(700, 64, 1, 333), encoder=(150, 31, 77, 410), tokens=20, seed=0):
    """Returns the last step's results and what they are over the unquantised keys and values, its queries, and the
    keys and values of the first encoder's states."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch, width = len(prompts), HEADS * (GROUP + 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    project = lambda n: torch.randn(n, width, DIM, generator=g, device="cuda").bfloat16()  # noqa: E731
    split = lambda x: (x[:, :HEADS * GROUP], x[:, HEADS * GROUP:-HEADS], x[:, -HEADS:])  # noqa: E731

    # the decoder's own cache and the encoder's
    most = max(prompts) + tokens
    pages = Pages(nc.new_kv_cache(sum(-(-(n + tokens) // PAGE) for n in prompts), PAGE, HEADS, DIM, fmt), batch, most)
    other = Pages(nc.new_kv_cache(sum(-(-n // PAGE) for n in encoder), PAGE, HEADS, DIM, fmt), batch, max(encoder))
    other.grow(encoder)
    other.len.copy_(i32(encoder))
    seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(encoder)).cuda()
    pos = torch.cat([torch.arange(n) for n in encoder]).cuda()
    _, ek, ev = split(project(sum(encoder)))
    nc.nc_kv_write(other.cache, ek, ev, other.slots(seq, pos))

    # prompts: written, then attended over
    pages.grow(prompts)
    pages.len.copy_(i32(prompts))
    seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(prompts)).cuda()
    pos = torch.cat([torch.arange(n) for n in prompts]).cuda()
    q, k, v = split(project(sum(prompts)))
    nc.nc_kv_write(pages.cache, k, v, pages.slots(seq, pos))
    start = torch.cat([i32([0]), pages.len.cumsum(0, dtype=torch.int32)])
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    nc.nc_kv_attention(pages.cache, q, out, start, pages.len, pages.table, max(prompts), max(prompts))

    # tokens: one graph, replayed
    pages.grow([n + tokens for n in prompts])
    fused = project(batch)
    one, every = torch.arange(batch + 1, dtype=torch.int32, device="cuda"), torch.arange(batch, device="cuda")
    tq, tk, tv = split(fused)
    own, cross = (torch.empty(tq.shape, dtype=tq.dtype, device="cuda") for _ in range(2))
    ws = nc.new_kv_workspace(pages.cache, tq, batch, 1, most)
    ws2 = nc.new_kv_workspace(other.cache, tq, batch, 1, max(encoder))

    def step():
        nc.nc_kv_write(pages.cache, tk, tv, pages.slots(every, pages.len.long()))
        pages.len.add_(1)
        nc.nc_kv_attention(pages.cache, tq, own, one, pages.len, pages.table, 1, most, ws=ws)
        nc.nc_kv_attention(other.cache, tq, cross, one, other.len, other.table, 1, max(encoder), causal=False, ws=ws2)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = [[k[seq == b], v[seq == b]] for b in range(batch)]
    for _ in range(tokens):
        fused.copy_(project(batch))
        for b in range(batch):
            seen[b] = [torch.cat([seen[b][0], tk[b:b + 1]]), torch.cat([seen[b][1], tv[b:b + 1]])]
        graph.replay()
    ends = torch.tensor(encoder).cumsum(0).tolist()
    want_own = torch.stack([reference(tq[b], *seen[b]) for b in range(batch)])
    want_cross = torch.stack([reference(tq[b], ek[e - n:e], ev[e - n:e]) for b, (e, n) in enumerate(zip(ends, encoder))])

    # one sequence's keys and values back
    n = int(pages.len[0])
    back = torch.empty(2, n, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(n, device="cuda")
    nc.nc_kv_read(pages.cache, pages.slots(torch.zeros_like(at), at), back[0], back[1])
    torch.cuda.synchronize()
    return {"own": (own, want_own), "cross": (cross, want_cross), "keys": (back[0], seen[0][0]),
            "values": (back[1], seen[0][1]), "query": tq, "encoder": (ek[:encoder[0]], ev[:encoder[0]]),
            "bytes": pages.cache.data.numel()}


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--fmt", choices=sorted(nc.KV_FMT), default="e2m1")
    ap.add_argument("--tokens", type=int, default=20)
    a = ap.parse_args()
    r = run(a.fmt, tokens=a.tokens)
    for name in ("keys", "values", "own", "cross"):
        got, want = (x.float() for x in r[name])
        print(f"{name:8s} against unquantised: {float((got - want).norm() / want.norm()):.4f} of their size apart")
    print(f"cache: {r['bytes'] / 2 ** 20:.1f} MiB")


if __name__ == "__main__":
    main()
