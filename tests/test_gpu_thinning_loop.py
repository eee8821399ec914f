"""Forks that share a prompt, step by step, and the thinning of their caches: the
pager, the append, the shared prefix, the attention over it, the weights of the
tokens, the choice of those that stay and the compaction, as a server runs them.

Each is held to its definition on what the one before it left, with the
tolerances of its own tests."""

import numpy as np
import pytest
import torch

import attn_ref
from test_gpu_attn import BF, _built, tolerance  # noqa: F401
from test_gpu_thin import chosen
from test_gpu_weights import reference

pytestmark = pytest.mark.gpu
PAGE, HKV, HQ, D = 16, 2, 8, 64
ROW = 6000  # columns: room for more than 256 MB, so that prefixes are taken together


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


class Server:
    def __init__(self, pages=400):
        import moe_expert_ffn_dg_gb300 as pkg
        g = torch.Generator(device="cuda").manual_seed(3)
        self.rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
        nan = torch.full((1, pages, PAGE, HKV, D), float("nan"), dtype=BF, device="cuda")
        self.pkg, self.cache = pkg, pkg.KvCache(nan, nan.clone())
        self.pager = pkg.KvPager(pages, PAGE)
        self.table = torch.full((1, ROW), -1, dtype=torch.int32, device="cuda")
        self.lens, self.ref = i32([0]), torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.attn = pkg.PagedAttention(self.cache, HQ, right=0, shared_tokens=64)

    def grow(self, parent, grow):
        f = self.pager.fork(self.table, self.lens, self.ref, i32(parent), i32(grow))
        assert int(f.short) == 0
        self.table, self.lens, self.ref = f.table, f.lens, f.ref
        self.cache.copy(f.copies)
        return self.pkg.KvBatch(self.table, self.lens, i32(np.concatenate([[0], np.cumsum(grow)])))

    def state(self):
        return (self.cache.k_pages[0].cpu(), self.cache.v_pages[0].cpu(), self.table.cpu(),
                self.lens.tolist())


def test_a_server_of_forks():
    s = Server()
    n = 300
    batch = s.grow([0], [n])
    s.cache.append(s.rand(n, HKV, D), s.rand(n, HKV, D), batch)
    forks = 6
    weights = torch.zeros(1, 400, device="cuda")
    parent = [0] * forks
    for step in range(4):
        batch = s.grow(parent, [1 + step % 2] * forks)
        weights = weights[parent].contiguous()
        tokens = int(batch.cu[-1])
        q = s.rand(tokens, HQ, D)
        s.cache.append(s.rand(tokens, HKV, D), s.rand(tokens, HKV, D), batch)
        shared = s.cache.shared(batch, i32([0, forks]))
        # whole pages of the prompt (the last one was split when the forks grew)
        assert shared.prefix.tolist() == [n // PAGE * PAGE] * forks
        lse = torch.empty(tokens, HQ, device="cuda")
        out, _ = s.attn.forward(q, batch, lse=lse, shared=shared)
        before = weights.cpu()
        s.attn.weights(q, lse, batch, weights, decay=0.9)
        k, v, table, lens = s.state()
        cu = batch.cu.tolist()
        ref = attn_ref.attention(q.cpu(), k, v, table, lens, cu, -1, 0, D ** -0.5)
        tol, ltol = tolerance(ref, BF, D, max(lens))
        assert ((out.double().cpu() - ref[0]).abs() <= tol).all()
        assert ((lse.double().cpu() - ref[1]).abs() <= ltol).all()
        want, wtol = reference(q.cpu(), k, lse.cpu(), before, table, lens, cu, -1, 0, D ** -0.5,
                               0.9, True)
        assert ((weights.double().cpu() - want).abs() <= wtol).all()
        # one candidate is dropped, another taken twice
        parent = [0, 1, 2, 3, 5, 5]
    # thin all of them, into fresh pages beside the old ones
    budget, first, last = 100, 4, 16
    sel = s.cache.select(weights, s.lens, budget, first=first, last=last)
    keep, cu = chosen(weights.cpu().numpy(), s.lens.tolist(), budget, first, last)
    assert sel.keep.tolist() == keep and sel.cu.tolist() == cu and cu[-1] == forks * budget
    old = s.table.clone()
    k, v, table, lens = s.state()
    batch = s.grow(list(range(forks)) + [-1] * forks, [0] * forks + sel.lens.tolist())
    s.cache.gather(old, s.table[forks:].contiguous(), sel.cu, sel.keep)
    # the old ones go; the thinned ones go on
    batch = s.grow(list(range(forks, 2 * forks)), [1] * forks)
    k2, v2, table2, lens2 = s.state()
    assert lens2 == [budget + 1] * forks
    for b in range(forks):
        some = torch.tensor(keep[cu[b]:cu[b + 1]])
        for new, was in ((k2, k), (v2, v)):
            assert torch.equal(attn_ref.cached(new, table2[b], budget),
                               attn_ref.cached(was, table[b], lens[b])[some])
    q, kn, vn = s.rand(forks, HQ, D), s.rand(forks, HKV, D), s.rand(forks, HKV, D)
    s.cache.append(kn, vn, batch)
    # nothing is shared any more
    shared = s.cache.shared(batch, i32([0, forks]))
    assert shared.prefix.tolist() == [0] * forks
    weights = torch.nn.functional.pad(sel.weights, (0, 4))
    lse = torch.empty(forks, HQ, device="cuda")
    out, _ = s.attn.forward(q, batch, lse=lse, shared=shared)
    s.attn.weights(q, lse, batch, weights)
    k, v, table, lens = s.state()
    ref = attn_ref.attention(q.cpu(), k, v, table, lens, list(range(forks + 1)), -1, 0, D ** -0.5)
    tol, _ = tolerance(ref, BF, D, max(lens))
    assert ((out.double().cpu() - ref[0]).abs() <= tol).all()
    # each of a sequence's rows spread a weight of one over its tokens
    gained = weights[:, :budget + 1].double().sum(1) - sel.weights.double().sum(1)
    assert torch.allclose(gained, torch.full_like(gained, HQ), rtol=1e-3)
    for h in (s.cache, s.pager, s.attn):
        assert h.device_status()[0] == 0


def test_a_step_captured_whole():
    """Plan, attention, weights and choice in one graph, replayed as the sequences
    grow."""
    s = Server()
    batch = s.grow([0], [200])
    s.cache.append(s.rand(200, HKV, D), s.rand(200, HKV, D), batch)
    batch = s.grow([0] * 4, [8] * 4)  # room; the steps use one more token each
    s.cache.append(s.rand(32, HKV, D), s.rand(32, HKV, D), batch)
    lens, cu = i32([201] * 4), i32(range(5))
    step = s.pkg.KvBatch(s.table, lens, cu)
    groups, q = i32([0, 4]), s.rand(4, HQ, D)
    lse, out = torch.empty(4, HQ, device="cuda"), torch.empty_like(q)
    weights = torch.zeros(4, 300, device="cuda")
    shared = s.cache.shared(step, groups)
    sel = s.cache.select(weights, lens, 64, first=2, last=8)

    def run():
        s.cache.shared(step, groups, out=shared)
        s.attn.forward(q, step, out=out, lse=lse, shared=shared)
        s.attn.weights(q, lse, step, weights, decay=0.5)
        s.cache.select(weights, lens, 64, first=2, last=8, out=sel)
    run()
    weights.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    want = torch.zeros_like(weights)
    for x in range(4):
        lens.fill_(201 + x)
        q.copy_(s.rand(4, HQ, D))
        graph.replay()
        ref = torch.empty_like(lse)
        got = s.attn.forward(q, step, lse=ref)[0]
        assert (got.float() - out.float()).abs().max() <= 2 ** -6
        assert (ref - lse).abs().max() <= 2 ** -12
        s.attn.weights(q, lse, step, want, decay=0.5)
        assert torch.equal(want, weights)
        keep, cu_ = chosen(weights.cpu().numpy(), lens.tolist(), 64, 2, 8)
        assert sel.keep.tolist() == keep and sel.cu.tolist() == cu_
    assert s.attn.device_status()[0] == 0 and s.cache.device_status()[0] == 0
