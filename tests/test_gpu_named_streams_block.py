"""The MoE block and the self-conditioning MLP on a named stream: what they
allocate is memory that is free there.

Few tokens' experts are added up by atomics, so that sums may differ in their last
bits from call to call.  What is asked here is whether memory was written over, with
NaN (or -1): whole numbers are compared, and of the others that they are none."""

import pytest
import torch

import moe_inputs as mi
from gpu_util import make_block, to_dev_bf16
from test_gpu_handle_memory import BUSY, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def caller(what):
    """A call of the entry point, which returns what it allocated."""
    import moe_expert_ffn_dg_gb300 as pkg
    if what == "sc":
        wl = mi.get_workload("sc_tiny")
        p = mi.make_sc_inputs(wl)
        sc = pkg.ScMlp.from_params(p, hidden=wl.hidden, inter=wl.dense_inter, max_tokens=wl.tokens)
        e, s = to_dev_bf16(p["embeds"]), to_dev_bf16(p["signal"])
        return lambda **kw: [sc.forward(e, s, **kw)]
    wl = mi.get_workload("tiny")
    block, h = make_block(wl, mi.make_layer_inputs(wl, randvec=True)), to_dev_bf16(mi.make_tokens(wl))
    if what == "forward":
        return lambda **kw: [block.forward(h, **kw)]
    if what == "debug":
        def debug(**kw):
            out, parts = block.forward(h, debug=True, **kw)
            return [out, *parts.values()]
        return debug
    w = torch.ones(wl.hidden, dtype=torch.bfloat16, device="cuda")
    return lambda **kw: list(block.forward_neighbours(h, h.flip(0), w, w, **kw))


def spoiled(t):
    return torch.full_like(t, float("nan") if t.is_floating_point() else -1)


def check(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert not torch.isnan(a).any() if a.is_floating_point() else torch.equal(a, b)


CALLS = pytest.mark.parametrize("what", ["forward", "debug", "neighbours", "sc"])


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
    junk = [spoiled(t) for _ in range(3) for t in want]
    del junk
    got = call(stream=side)
    torch.cuda.synchronize()
    check(got, want)


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
        for t in new:
            t.copy_(spoiled(t))
    torch.cuda.synchronize()
    check(copies, want)
