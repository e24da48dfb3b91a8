"""Decoding with entropy-coded weights and the 4-bit key/value cache.

A small transformer (random weights, stored Huffman-coded; no embedding or sampler: the
"tokens" are random hidden states) decodes with several beams:

  prompt   ec_gemm_group   q, k, v of the whole prompt
           ec_kv_fork      room for it in the cache
           ec_kv_append    its keys and values, quantised into pages
           ec_kv_attend    causal attention over them
  steps    ec_kv_fork      beams take new parents and one more place each
           ec_gemv_group   q, k, v of the new tokens
           ec_kv_append, ec_kv_attend, ec_gemv (o projection)
  now and then ec_kv_compact moves the pages in use together.

    python examples/decode_with_cache.py

prints the largest difference from the same model in plain FP32 torch (which reads the
cache's values back, so that both see the same quantised keys and values).
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import lossless_entropy_coded_gb300 as ec

LAYERS, HIDDEN, Q_HEADS, KV_HEADS, DIM, PAGE = 2, 1024, 8, 2, 128, 16
WINDOW, SINKS = 96, 4


def bf16(x):
    return x.to(torch.bfloat16)


class Model:
    """q, k, v and o projections of each layer, dense (for the reference) and encoded."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dense, self.coded = [], []
        for _ in range(LAYERS):
            shapes = {"q": (Q_HEADS * DIM, HIDDEN), "k": (KV_HEADS * DIM, HIDDEN), "v": (KV_HEADS * DIM, HIDDEN), "o": (HIDDEN, Q_HEADS * DIM)}
            w = {n: bf16(torch.randn(s, generator=g) * s[1] ** -0.5) for n, s in shapes.items()}
            self.dense.append({n: x.float().cuda() for n, x in w.items()})
            self.coded.append({n: ec.encode_bf16(x.view(torch.int16).numpy().view(np.uint16)) for n, x in w.items()})

    def qkv(self, layer, x):
        """FP32 q, k, v [rows, heads, DIM] of BF16 rows x."""
        rows = x.shape[0]
        ys = [torch.empty((rows, n * DIM), device="cuda") for n in (Q_HEADS, KV_HEADS, KV_HEADS)]
        ws = [self.coded[layer][n] for n in "qkv"]
        if rows <= ec.EC_MAX_BATCH:
            ec.gemv_group(ws, x, ys, batch=rows)
        else:
            ec.gemm_group(ws, [x] * 3, ys, rows)
        return [y.view(rows, -1, DIM) for y in ys]

    def o(self, layer, a):
        y = torch.empty((a.shape[0], HIDDEN), device="cuda")
        if a.shape[0] <= ec.EC_MAX_BATCH:
            ec.gemv(self.coded[layer]["o"], a, y, batch=a.shape[0])
        else:
            ec.gemm(self.coded[layer]["o"], a, y, a.shape[0])
        return y


class Beams:
    """Sequences of a cache with their page tables, double-buffered as ec_kv_fork wants them."""

    def __init__(self, beams, pages, width):
        self.cache = ec.kv_cache(LAYERS, pages, KV_HEADS, DIM, PAGE)
        make = lambda: ec.kv_seqs(torch.full((beams, width), -1, dtype=torch.int32, device="cuda"),
                                  torch.zeros(beams, dtype=torch.int32, device="cuda"))
        self.now, self.spare = make(), make()
        self.refs, self.refs_spare = (torch.zeros(pages, dtype=torch.int32, device="cuda") for _ in range(2))

    def _swap(self):
        self.now, self.spare, self.refs, self.refs_spare = self.spare, self.now, self.refs_spare, self.refs

    def fork(self, parents, grow):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        ec.kv_fork(self.cache, self.now, self.refs, self.spare, self.refs_spare, parents=i32(parents), grow=i32(grow))
        self._swap()

    def compact(self):
        ec.kv_compact(self.cache, self.now, self.refs, self.spare, self.refs_spare)
        self._swap()


def forward(model, beams, x, starts, max_new):
    """New rows x (FP32 hidden states) through all layers; appends to the cache as it goes."""
    i32 = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for layer in range(LAYERS):
        q, k, v = model.qkv(layer, bf16(x))
        ec.kv_append(beams.cache, layer, beams.now, k, v, starts=i32, max_new=max_new)
        a = torch.empty((x.shape[0], Q_HEADS, DIM), dtype=torch.bfloat16, device="cuda")
        ec.kv_attend(beams.cache, layer, beams.now, q, a, starts=i32, max_new=max_new, window=WINDOW, sinks=SINKS)
        x = x + model.o(layer, a.view(x.shape[0], -1))
    return x


def reference(model, beams, x, starts):
    """The same in plain torch; the cache's values are read back from where forward left them."""
    lens = beams.now.lens.tolist()
    whole = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    for layer in range(LAYERS):
        k, v = (torch.empty((sum(lens), KV_HEADS, DIM), device="cuda") for _ in range(2))
        ec.kv_read(beams.cache, layer, beams.now, k, v, starts=whole, max_new=max(lens))
        q = (bf16(x).float() @ model.dense[layer]["q"].T).view(-1, KV_HEADS, Q_HEADS // KV_HEADS, DIM)
        outs, at = [], 0
        for i, n in enumerate(lens):
            m = starts[i + 1] - starts[i]
            pos = torch.arange(n - m, n, device="cuda")[:, None]
            t = torch.arange(n, device="cuda")[None]
            see = (t <= pos) & ((t > pos - WINDOW) | (t < SINKS))
            s = torch.einsum("mhgd,thd->hgmt", q[starts[i]:starts[i + 1]], k[at:at + n]) * DIM ** -0.5
            p = s.masked_fill(~see, float("-inf")).softmax(-1)
            outs.append(torch.einsum("hgmt,thd->mhgd", p, v[at:at + n]).reshape(m, Q_HEADS * DIM))
            at += n
        x = x + bf16(torch.cat(outs)).float() @ model.dense[layer]["o"].T
    return x


def main(prompt=150, beams=4, steps=24, seed=1):
    """Returns the largest relative difference from the reference over prompt and steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    model = Model()
    b = Beams(beams, pages=96, width=24)
    worst = 0.0

    def check(x, y, starts):
        nonlocal worst
        want = reference(model, b, x, starts)
        worst = max(worst, float((y - want).norm() / want.norm()))

    b.fork([-1] * beams, [0] * beams)                     # empty sequences
    b.fork(list(range(beams)), [prompt] + [0] * (beams - 1))  # room for the prompt in beam 0
    x = torch.randn((prompt, HIDDEN), generator=g, device="cuda")
    starts = [0] + [prompt] * beams
    check(x, forward(model, b, x, starts, prompt), starts)
    parents = [0] * beams                                 # every beam continues the prompt
    for step in range(steps):
        b.fork(parents, [1] * beams)
        x = torch.randn((beams, HIDDEN), generator=g, device="cuda")
        starts = list(range(beams + 1))
        check(x, forward(model, b, x, starts, 1), starts)
        parents = torch.randint(0, beams, (beams,), generator=g, device="cuda").tolist()
        if step % 8 == 7:
            b.compact()
    assert ec.status() == 0
    return worst


if __name__ == "__main__":
    print(f"largest relative difference from the plain model: {main():.2e}")
