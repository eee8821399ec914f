"""Results that a call on a named stream allocates: memory that is free on that
stream, and stays theirs as long as the current stream uses them."""

import pytest
import torch

from test_gpu_attn import BF, _built  # noqa: F401
from test_gpu_shared import handles, i32, make

pytestmark = pytest.mark.gpu
BUSY = 200_000_000  # cycles: about 0.1 s


def caller(what):
    """A call of the entry point, which returns what it allocated."""
    import moe_expert_ffn_dg_gb300 as pkg
    attn, q, batch, groups = handles(make([(300, [(9, 2)] * 40)], 8, 2, 64, 16, BF, 30))
    cache = attn.cache
    if what == "rope":
        rope, at = pkg.Rope(64), torch.arange(q.shape[0], dtype=torch.int32, device="cuda")
        return lambda **kw: [rope.apply(q, at, **kw)]
    if what == "append":
        k = torch.zeros(q.shape[0], 2, 64, dtype=BF, device="cuda")
        return lambda **kw: [cache.append(k, k, batch, q=q, **kw)]
    if what == "forward":
        return lambda **kw: [attn.forward(q, batch, **kw)]
    if what == "forward shared":
        plan = cache.shared(batch, groups)
        return lambda **kw: [attn.forward(q, batch, shared=plan, **kw)]
    if what == "plan":
        return lambda **kw: [cache.shared(batch, groups, **kw).prefix]
    if what == "select":
        w, lens = torch.rand(40, 900, device="cuda"), i32([900 - 20 * i for i in range(40)])

        def select(**kw):
            r = cache.select(w, lens, 200, first=3, last=9, **kw)
            return [r.keep, r.cu, r.lens, r.weights]
        return select
    pager = pkg.KvPager(500, 16)
    state = (i32([[x, x + 1, -1, -1] for x in range(0, 80, 2)]), i32([20] * 40),
             i32([1] * 80 + [0] * 420), i32(list(range(40))), i32([30] * 40))

    def fork(**kw):
        r = pager.fork(*state, **kw)
        return [r.table, r.lens, r.ref, r.copies, r.short]
    return fork


CALLS = pytest.mark.parametrize("what", ["rope", "append", "forward", "forward shared", "plan",
                                         "select", "fork"])


@CALLS
def test_results_are_not_what_the_current_stream_gave_back(what):
    call, side = caller(what), torch.cuda.Stream()
    call()  # kernels are loaded
    torch.cuda.synchronize()
    gone = [t for _ in range(3) for t in call()]
    torch.cuda.synchronize()
    where = {t.data_ptr() for t in gone}
    del gone
    got = call(stream=side)
    torch.cuda.synchronize()
    assert not where & {t.data_ptr() for t in got}


@CALLS
def test_results_beside_work_of_the_current_stream(what):
    """The current stream still writes to memory that it has given back."""
    call, side = caller(what), torch.cuda.Stream()
    want = [t.clone() for t in call()]
    call(stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    junk = [torch.full_like(t, 3) for _ in range(3) for t in want]
    del junk
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@CALLS
def test_results_that_the_current_stream_still_reads(what):
    call, side = caller(what), torch.cuda.Stream()
    call(stream=side)
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in got]
    sizes = [(t.shape, t.dtype, t.data_ptr()) for t in got]
    want = call()
    del got
    with torch.cuda.stream(side):
        new = [torch.empty(s, dtype=d, device="cuda") for s, d, _ in sizes]
    assert not {t.data_ptr() for t in new} & {at for _, _, at in sizes}
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


@CALLS
def test_captured_on_a_stream_beside_the_captured_one(what):
    call, side = caller(what), torch.cuda.Stream()
    want = [t.clone() for t in call()]
    call(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for t in got:
        t.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
