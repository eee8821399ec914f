"""The memory of new MoE blocks and self-conditioning MLPs: cleared after its
last use by earlier work and before the handle's first call, on any stream."""

import pytest
import torch

import moe_inputs as mi
from gpu_util import make_block, to_dev_bf16

pytestmark = pytest.mark.gpu
BUSY = 200_000_000  # cycles: about 0.1 s


@pytest.fixture(scope="module", autouse=True)
def _built():
    import moe_expert_ffn_dg_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkg.build()
    pkg.load_library()


def maker(kind):
    """A function that builds the handle on given weights, and one that runs it."""
    import moe_expert_ffn_dg_gb300 as pkg
    if kind == "moe":
        wl = mi.get_workload("tiny")
        first = make_block(wl, mi.make_layer_inputs(wl, randvec=True))
        h = to_dev_bf16(mi.make_tokens(wl))
        return (lambda: pkg.MoEBlock(first.weights, hidden=wl.hidden, n_experts=wl.n_experts,
                                     top_k=wl.top_k, expert_inter=wl.expert_inter,
                                     dense_inter=wl.dense_inter, max_tokens=wl.tokens),
                lambda b: b.forward(h))
    wl = mi.get_workload("sc_tiny")
    p = mi.make_sc_inputs(wl)
    first = pkg.ScMlp.from_params(p, hidden=wl.hidden, inter=wl.dense_inter, max_tokens=wl.tokens)
    e, s = to_dev_bf16(p["embeds"]), to_dev_bf16(p["signal"])
    return (lambda: pkg.ScMlp(first.weights, hidden=wl.hidden, inter=wl.dense_inter,
                              max_tokens=wl.tokens), lambda b: b.forward(e, s))


@pytest.mark.parametrize("kind", ["moe", "sc"])
def test_a_new_handle_waits_for_the_memory_it_gets(kind):
    make, _ = maker(kind)
    size = make().workspace.numel()
    side = torch.cuda.Stream()
    torch.ones(size, dtype=torch.uint8, device="cuda").sum(dtype=torch.int64)  # loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x = torch.ones(size, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(BUSY)
        total = x.sum(dtype=torch.int64)
        where = x.data_ptr()
        del x
        new = make()
    torch.cuda.synchronize()
    assert new.workspace.data_ptr() == where, "the allocator gave other memory: nothing was tried"
    assert int(total) == size


@pytest.mark.parametrize("kind", ["moe", "sc"])
def test_a_new_handle_is_clear_before_its_first_call(kind):
    """Made and used on a side stream while the default one has work to do."""
    make, run = maker(kind)
    want = run(make()).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    end = torch.cuda.Event()
    end.record()
    with torch.cuda.stream(side):
        got = run(make())
    # the clearing goes through the default stream: that work is done by now
    assert end.query()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["moe", "sc"])
def test_memory_of_a_dropped_handle_outlives_its_calls(kind):
    """A handle that is dropped while a call runs on another stream: its
    workspace is not given out again before that call is done."""
    make, run = maker(kind)
    new = make()
    want = run(new).clone()
    size, where = new.workspace.numel(), new.workspace.data_ptr()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        got = run(new)
    del new
    other = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert other.data_ptr() != where
    other.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
