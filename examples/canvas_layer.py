"""One decoder layer over a paged cache: attention half and routed-MoE half.

A prompt is taken in chunks, then its sequence is forked into several
candidates and each denoises its own 256-token canvas behind the shared prompt
pages; finished canvases are committed (they stay in the cache) and a thinned
copy of the longest cache is made.  The projections around the attention are
plain library products; everything else is the package's kernels.

    python examples/canvas_layer.py          (needs a GPU and the built library)
"""

from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_expert_ffn_dg_gb300 as pkg  # noqa: E402
import moe_inputs as mi  # noqa: E402


class Layer:
    """Weights of one layer and the handles that run it over a cache."""

    def __init__(self, cache, wl, *, q_heads, max_tokens, seed=0):
        self.cache, self.hidden, self.q_heads = cache, wl.hidden, q_heads
        dev, d, kv = cache.device, cache.head_dim, cache.n_kv_heads
        gen = torch.Generator(device=dev).manual_seed(seed)

        def w(rows, cols):
            t = torch.randn(rows, cols, generator=gen, device=dev) * cols ** -0.5
            return t.to(torch.bfloat16)
        self.w_qkv = w((q_heads + 2 * kv) * d, wl.hidden)
        self.w_o = w(wl.hidden, q_heads * d)
        self.w_post = torch.ones(wl.hidden, dtype=torch.bfloat16, device=dev)
        self.rope = pkg.Rope(d, theta=10000.0)
        # prompts are causal; every token of a canvas sees its prompt and canvas
        self.causal = pkg.PagedAttention(cache, q_heads, right=0)
        self.canvas = pkg.PagedAttention(cache, q_heads, right=-1)
        self.moe = pkg.MoEBlock.from_params(
            mi.make_layer_inputs(wl, randvec=True), hidden=wl.hidden, n_experts=wl.n_experts,
            top_k=wl.top_k, expert_inter=wl.expert_inter, dense_inter=wl.dense_inter,
            max_tokens=max_tokens, device=dev)

    def attention(self, x, batch, causal):
        """Attention half up to its output projection; x is normed already."""
        d, kv, hq = self.cache.head_dim, self.cache.n_kv_heads, self.q_heads
        qkv = (x @ self.w_qkv.T).view(x.shape[0], hq + 2 * kv, d)
        q, k, v = qkv.split([hq, kv, kv], 1)
        q = self.cache.append(k, v, batch, q=q, rope=self.rope)
        o = (self.causal if causal else self.canvas).forward(q, batch)
        return o.view(x.shape[0], hq * d) @ self.w_o.T

    def forward(self, x, batch, causal):
        """Layer output and the next layer's normed input."""
        attn = self.attention(x, batch, causal)
        return self.moe.forward_neighbours(x, attn, self.w_post, self.w_post)


class Server:
    """Cache, page table and counts, taken from step to step by the pager."""

    def __init__(self, *, pages=64, page_size=64, kv_heads=2, head_dim=128, row=16, slots=1):
        shape = (1, pages, page_size, kv_heads, head_dim)
        self.cache = pkg.KvCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
                                   for _ in range(2)))
        self.pager = pkg.KvPager(pages, page_size)
        self.table = torch.full((slots, row), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(pages, dtype=torch.int32, device="cuda")

    def step(self, parent, grow):
        """Continue the sequences of `parent`, with room for `grow` tokens each."""
        def ints(a):
            return torch.tensor(a, dtype=torch.int32, device="cuda")
        f = self.pager.fork(self.table, self.lens, self.ref, ints(parent), ints(grow))
        self.table, self.lens, self.ref = f.table, f.lens, f.ref
        self.cache.copy(f.copies)
        cu = ints([sum(grow[:i]) for i in range(len(grow) + 1)])
        return pkg.KvBatch(self.table, self.lens, cu), f.short


def run(prompt_chunks=(100, 57), canvases=3, canvas=256, steps=2, seed=0):
    """Returns the outputs of every forward (for checking) and the server."""
    wl = mi.get_workload("tiny", tokens=canvases * canvas)
    server = Server()
    layer = Layer(server.cache, wl, q_heads=4, max_tokens=canvases * canvas)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def tokens(n):
        return torch.randn(n, wl.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    log = []
    for n in prompt_chunks:
        batch, _ = server.step([0], [n])
        x = tokens(n)
        log.append((x, batch, True, layer.forward(x, batch, True)))
    # the fork: all candidates share the prompt; its last page is split
    batch, short = server.step([0] * canvases, [canvas] * canvases)
    for _ in range(steps):  # the canvas's rows of the cache are rewritten in place
        x = tokens(canvases * canvas)
        log.append((x, batch, False, layer.forward(x, batch, False)))
    # a thinned copy of the first candidate: every other token, in fresh pages
    have = sum(prompt_chunks) + canvas
    keep = torch.arange(0, have, 2, dtype=torch.int32, device="cuda")
    src = server.table[:1].clone()
    server.step(list(range(canvases)) + [-1], [0] * canvases + [len(keep)])
    server.cache.gather(src, server.table[canvases:], torch.tensor(
        [0, len(keep)], dtype=torch.int32, device="cuda"), keep)
    return layer, server, log, short


if __name__ == "__main__":
    pkg.load_library()
    layer, server, log, short = run()
    torch.cuda.synchronize()
    assert int(short) == 0
    for name, status in (("cache", server.cache.device_status()),
                         ("pager", server.pager.device_status()),
                         ("attention", layer.canvas.device_status()),
                         ("moe", layer.moe.device_status())):
        assert status[0] == 0, (name, status)
    for x, _, causal, (out, _) in log:
        print(f"{'prompt' if causal else 'canvas'} of {x.shape[0]} tokens: "
              f"rms {out.float().pow(2).mean().sqrt():.3f}")
    print("tokens cached:", server.lens.tolist(), "pages held:", int((server.ref > 0).sum()))
