"""The attention half's handles beside other streams' work: status words,
workspaces and results."""

import pytest
import torch

from test_gpu_attn import BF, _built, handles, make  # noqa: F401

pytestmark = pytest.mark.gpu
BUSY = 200_000_000  # cycles: about 0.1 s


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def small_cache():
    import moe_expert_ffn_dg_gb300 as pkg
    return pkg.KvCache(*(torch.zeros(1, 4, 16, 1, 64, dtype=BF, device="cuda") for _ in range(2)))


def bad_append(cache, **kw):
    """One token whose page id is out of range: the kernel skips and reports it."""
    import moe_expert_ffn_dg_gb300 as pkg
    k = torch.zeros(1, 1, 64, dtype=BF, device="cuda")
    batch = pkg.KvBatch(i32([[9]]), i32([1]), i32([0, 1]))
    torch.cuda.synchronize()
    cache.append(k, k, batch, **kw)
    return k, batch


def test_reading_a_status_waits_for_its_stream_alone():
    from moe_expert_ffn_dg_gb300 import binding as B
    cache = small_cache()
    side = torch.cuda.Stream()
    keep = bad_append(cache, stream=side)
    torch.cuda._sleep(BUSY)
    end = torch.cuda.Event()
    end.record()
    assert cache.device_status(side)[0] == B.DG_ERR_DEVICE_CHECK
    assert not end.query()  # the other stream's work is still under way
    assert cache.device_status(side)[0] == 0
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    del keep


def test_a_new_handle_loses_no_report():
    """The word is clear when the handle is there: not later, behind whatever
    the default stream has to do."""
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    pools = [torch.zeros(1, 4, 16, 1, 64, dtype=BF, device="cuda") for _ in range(2)]
    k = torch.zeros(1, 1, 64, dtype=BF, device="cuda")
    batch = pkg.KvBatch(i32([[9]]), i32([1]), i32([0, 1]))
    side = torch.cuda.Stream()
    for _ in range(2):  # every kernel is loaded (which may wait for the GPU)
        old = pkg.KvCache(*pools)
        old.append(k, k, batch, stream=side)
        pkg.PagedAttention(old, 1).forward(k, batch, stream=side)
        torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    with torch.cuda.stream(side):
        cache = pkg.KvCache(*pools)
        attn = pkg.PagedAttention(cache, 1)
        cache.append(k, k, batch)
        attn.forward(k, batch)
    torch.cuda.synchronize()
    assert cache.device_status(side)[0] == B.DG_ERR_DEVICE_CHECK
    assert attn.device_status(side)[0] == B.DG_ERR_DEVICE_CHECK


@pytest.mark.parametrize("what", ["cache", "attention"])
def test_a_new_handle_waits_for_the_memory_it_gets(what):
    """Made on a side stream, its memory may be what an earlier kernel of that
    stream still reads."""
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    pools = [torch.zeros(1, 4, 16, 1, 64, dtype=BF, device="cuda") for _ in range(2)]
    cache = pkg.KvCache(*pools)
    size = 256 if what == "cache" else 1024 + B.dg_attn_workspace_size(
        B.dg_attn_config_t(1, -1, 0, 0.1, 0), cache.handle)
    side = torch.cuda.Stream()
    torch.ones(size, dtype=torch.uint8, device="cuda").sum(dtype=torch.int64)  # loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x = torch.ones(size, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(BUSY)
        total = x.sum(dtype=torch.int64)
        where = x.data_ptr()
        del x
        new = pkg.KvCache(*pools) if what == "cache" else pkg.PagedAttention(cache, 1)
        got = (new._status if what == "cache" else new.workspace).data_ptr()
    torch.cuda.synchronize()
    assert got == where, "the allocator gave other memory: nothing was tried"
    assert int(total) == size


def overwritten(size, old):
    """New memory of the size just given back, filled: must not be the old one
    while another stream may use it."""
    new = torch.empty(size, dtype=torch.uint8, device="cuda")
    new.fill_(255)
    return new.data_ptr() == old


@pytest.mark.parametrize("named", [True, False])
def test_memory_of_a_dropped_handle_outlives_its_calls(named):
    """A handle that is dropped while a call runs on another stream: its memory
    is not given out again before that call is done."""
    import moe_expert_ffn_dg_gb300 as pkg
    attn, q, batch = handles(make([2], [9000], 2, 1, 64, 64, BF, 60))
    cache, pager = attn.cache, pkg.KvPager(1 << 16, 16)
    table, lens, ref = i32([[0, 1, -1, -1]]), i32([20]), i32([1, 1] + [0] * ((1 << 16) - 2))
    parent, grow = i32([0, 0]), i32([30, 1])
    want = attn.forward(q, batch)
    step = pager.fork(table, lens, ref, parent, grow)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [(attn.workspace.nbytes, attn.workspace.data_ptr()),
             (pager.workspace.nbytes, pager.workspace.data_ptr())]
    out = torch.zeros_like(q)
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        if not named:
            attn.forward(q, batch, out=out)
            again = pager.fork(table, lens, ref, parent, grow)
    if named:
        attn.forward(q, batch, out=out, stream=side)
        again = pager.fork(table, lens, ref, parent, grow, stream=side)
    del attn, pager
    assert not any([overwritten(*s) for s in sizes])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and cache.device_status()[0] == 0
    for name in again.__slots__:
        assert torch.equal(getattr(again, name), getattr(step, name))


def test_two_attentions_on_two_streams():
    """Each has a workspace of its own: calls on two streams may overlap."""
    import moe_expert_ffn_dg_gb300 as pkg
    data = [make([2, 90], [9000, 700], 4, 2, 128, 64, BF, 61),
            make([1, 1, 1], [5000, 3000, 40], 4, 2, 128, 64, BF, 62)]
    both = [handles(d) for d in data]
    want = [a.forward(q, b).clone() for a, q, b in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [a.forward(q, b, stream=s) for (a, q, b), s in zip(both, streams)]
    torch.cuda.synchronize()
    for got, w, (a, _, _) in zip(outs, want, both):
        assert torch.equal(got, w) and a.device_status()[0] == 0
