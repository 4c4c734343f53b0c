"""Two attention layers with 4-bit projections over the 8-bit key-value cache.

    python examples/cached_attention.py

Two prompts go in as one ragged batch, the first one branches into two
continuations that share its pages, and all of them decode token by token
under a sliding window with a few first tokens that stay visible, one captured
graph per step.  Queries and keys are turned by their positions as they are
appended, and attention knows which tokens the continuations share.  Then the prompt's own row is released and the pool compacted.
A longer prompt is then continued eighty times without a window: there attention reads the
shared tokens once for all of them (two continuations under a short window would save too
little, and run as without sharing).
The last hidden states are compared with the same computation in fp32 without
a cache: the difference is the cache's (keys and values in 8 bits).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_only_amd import nf4  # noqa: E402

HIDDEN, HEADS, KV, DIM, LAYERS = 512, 8, 2, 64, 2
PAGE, PAGES, WINDOW, SINKS = 32, 40, 48, 4
SCALE = DIM ** -0.5
ROTARY = nf4.Rotary(DIM)


def rotate(x, at):
    """What ROTARY does to rows x [rows][heads * DIM] at positions at, in fp32."""
    x = x.reshape(len(x), -1, 2, DIM // 2)
    angle = at[:, None] * 10000.0 ** (-torch.arange(DIM // 2, device=x.device) / (DIM // 2))
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[:, :, 0], x[:, :, 1]
    return torch.stack([a * c - b * s, a * s + b * c], 2).reshape(len(x), -1)


class Layers:
    """The weights, packed to 4 bits, and what they stand for."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(0)
        self.codebook = nf4.nf4_codebook()
        self.packed, self.dense = [], []
        for _ in range(LAYERS):
            shapes = ((HEADS + 2 * KV) * DIM, HIDDEN), (HIDDEN, HEADS * DIM)
            ws = [torch.randn(*s, generator=g, device="cuda") * 0.05 for s in shapes]
            self.packed.append([nf4.pack_weight(w, self.codebook) for w in ws])
            for p, w in zip(self.packed[-1], ws):
                nf4.nf4_dequant(p.qweight, p.absmax, self.codebook, p.N, p.K, w)
            self.dense.append(ws)

    def linear(self, x, w):
        """x . dequant(W)^T: the GEMV for up to 8 rows, the GEMM for more."""
        y = torch.empty(len(x), w.N, dtype=torch.float32, device="cuda")
        f = nf4.nf4_gemv if len(x) <= 8 else nf4.nf4_gemm
        n = nf4.nf4_workspace_bytes(len(x), w.N, w.K)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        f(x, len(x), w.qweight, w.absmax, self.codebook, w.N, w.K, y, ws, n)
        return y


def forward(net, cache, batch, x, window, groups=None):
    """One step of rows x (fp32 hidden states) through the layers."""
    shared = () if groups is None else (groups,)
    size, attention = ((nf4.nf4_kv_attention_workspace_bytes, nf4.nf4_kv_attention) if groups is None
                       else (nf4.nf4_kv_attention_shared_workspace_bytes, nf4.nf4_kv_attention_shared))
    n = size(cache, batch, *shared, HEADS, window, SINKS)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    for layer, (qkv, wo) in enumerate(net.packed):
        y = net.linear(x.bfloat16(), qkv)
        # slices of the rows as the projection left them, fp32 and strided
        k, v = y[:, HEADS * DIM:], y[:, (HEADS + KV) * DIM:]
        q = torch.empty(len(y), HEADS * DIM, dtype=torch.bfloat16, device="cuda")
        nf4.nf4_kv_append_rotated(cache, layer, batch, ROTARY, y, y.stride(0), HEADS, None, k,
                                  k.stride(0), None, v, v.stride(0), nf4.NF4_KV_F32, 0.0, q)
        out = torch.empty_like(q)
        attention(cache, layer, batch, *shared, q, q.stride(0), HEADS, SCALE, window, SINKS, out,
                  None, ws, n)
        x = x + net.linear(out, wo)
    return x


def reference(net, xs, window_from):
    """The same in fp32 for one sequence's hidden states xs [tokens][HIDDEN]:
    rows from window_from on see the window only."""
    at = torch.arange(len(xs), device="cuda")
    seen = at <= at[:, None]
    near = (at > at[:, None] - WINDOW) | (at < SINKS)
    seen &= near | (at[:, None] < window_from)
    for qkv, wo in net.dense:
        y = xs.bfloat16().float() @ qkv.T
        q = rotate(y[:, :HEADS * DIM], at).reshape(-1, KV, HEADS // KV, DIM)
        k = rotate(y[:, HEADS * DIM:(HEADS + KV) * DIM], at).reshape(-1, KV, DIM)
        v = y[:, (HEADS + KV) * DIM:].reshape(-1, KV, DIM)
        out = torch.empty_like(q)
        for h in range(KV):
            for i in range(HEADS // KV):
                s = (q[:, h, i] @ k[:, h].T * SCALE).masked_fill(~seen, -torch.inf)
                out[:, h, i] = s.softmax(-1) @ v[:, h]
        xs = xs + out.reshape(len(xs), -1) @ wo.T
    return xs


def continuations(net, prompt=3600, branches=80, tokens=4):
    """One prompt, forked into so many continuations that reading what they share once
    pays: the worst relative error, and whether the shared tokens were taken apart."""
    torch.manual_seed(2)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    width = -(-(prompt + tokens) // PAGE)
    pages = width + 2 * branches
    cache = nf4.KVCache(LAYERS, pages, KV, PAGE, DIM)
    pool = nf4.KVPool(torch.zeros(pages, dtype=torch.int32, device="cuda"),
                      torch.full((1 + branches, width), -1, dtype=torch.int32, device="cuda"),
                      torch.zeros(1 + branches, dtype=torch.int32, device="cuda"), i32(0))
    first = torch.randn(prompt, HIDDEN, device="cuda")
    nf4.nf4_kv_reserve(cache, pool, i32(prompt, *[0] * branches))
    batch = nf4.KVBatch(pool.length[:1], pool.table[:1], row_start=i32(0, prompt), rows=prompt,
                        max_rows=prompt, max_len=prompt)
    forward(net, cache, batch, first, 0)
    nf4.nf4_kv_fork(cache, pool, i32(*[0] * branches), i32(*range(1, branches + 1)), branches)
    nf4.nf4_kv_release(cache, pool, i32(0), 1)
    assert int(pool.missing) == 0, "the pool ran out of pages"

    batch = nf4.KVBatch(pool.length[1:], pool.table[1:], max_len=width * PAGE)
    groups = nf4.KVGroups(i32(prompt), max_prefix=prompt)  # one group of all
    apart = (nf4.nf4_kv_attention_shared_workspace_bytes(cache, batch, groups, HEADS, 0, SINKS)
             != nf4.nf4_kv_attention_workspace_bytes(cache, batch, HEADS, 0, SINKS))
    new = torch.randn(tokens, branches, HIDDEN, device="cuda")
    for x in new:
        nf4.nf4_kv_reserve(cache, pool, i32(0, *[1] * branches))
        last = forward(net, cache, batch, x, 0, groups)
    worst = 0.0
    for i in (0, branches - 1):
        want = reference(net, torch.cat([first, new[:, i]]), prompt + tokens)[-1]
        worst = max(worst, float((last[i] - want).norm() / want.norm()))
    print(f"{branches} continuations of {prompt} tokens, shared ones read once: {apart}; rel-L2 {worst:.4f}")
    return worst, apart


def main(tokens=20):
    torch.manual_seed(1)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    net = Layers()
    cache = nf4.KVCache(LAYERS, PAGES, KV, PAGE, DIM)
    # rows 0 and 1: the prompts; 2 and 3: continuations of row 0
    lengths, rows, width = (150, 70), 4, 8
    pool = nf4.KVPool(torch.zeros(PAGES, dtype=torch.int32, device="cuda"),
                      torch.full((rows, width), -1, dtype=torch.int32, device="cuda"),
                      torch.zeros(rows, dtype=torch.int32, device="cuda"), i32(0))

    # the prompts, one ragged batch
    prompts = [torch.randn(n, HIDDEN, device="cuda") for n in lengths]
    nf4.nf4_kv_reserve(cache, pool, i32(*lengths, 0, 0))
    batch = nf4.KVBatch(pool.length[:2], pool.table[:2], row_start=i32(0, 150, 220), rows=220,
                        max_rows=150, max_len=150)
    forward(net, cache, batch, torch.cat(prompts), 0)

    # row 0 continues as rows 2 and 3; rows 1 to 3 go on, a token at a time
    nf4.nf4_kv_fork(cache, pool, i32(0, 0), i32(2, 3), 2)
    nf4.nf4_kv_release(cache, pool, i32(0), 1)
    new = torch.randn(tokens, 3, HIDDEN, device="cuda")
    batch = nf4.KVBatch(pool.length[1:], pool.table[1:], max_len=width * PAGE)
    # the last two of the batch share the prompt
    groups = nf4.KVGroups(i32(lengths[0]), i32(1, 3), max_rows=2, max_prefix=lengths[0])
    one, x, missing = i32(0, 1, 1, 1), torch.empty(3, HIDDEN, device="cuda"), i32(0)

    def step():
        nf4.nf4_kv_reserve(cache, pool, one)
        missing.add_(pool.missing)
        return forward(net, cache, batch, x, WINDOW, groups)

    x.copy_(new[0])
    last = step()  # eager once, then captured: lengths and pages live on the device
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        last = step()
    for t in range(1, tokens):
        x.copy_(new[t])
        graph.replay()
    assert int(missing) == 0, "the pool ran out of pages"

    used = int((pool.refs > 0).sum())
    ws = torch.empty(nf4.nf4_kv_compact_workspace_bytes(cache), dtype=torch.uint8, device="cuda")
    nf4.nf4_kv_compact(cache, pool, pool.refs, pool.table, ws, ws.numel())
    assert bool((pool.refs[:used] > 0).all()) and not bool((pool.refs[used:] > 0).any())
    x.copy_(new[-1])
    graph.replay()  # one more token, from the compacted pages
    torch.cuda.synchronize()

    worst = 0.0
    for i, p in enumerate((1, 0, 0)):
        xs = torch.cat([prompts[p], new[:, i], new[-1:, i]])
        want = reference(net, xs, lengths[p])[-1]
        worst = max(worst, float((last[i] - want).norm() / want.norm()))
    print(f"{used} of {PAGES} pages in use, lengths {pool.length.tolist()}; "
          f"last hidden states against fp32 without a cache: rel-L2 {worst:.4f}")
    return max(worst, continuations(net)[0])


if __name__ == "__main__":
    main()
