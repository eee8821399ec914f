"""Plans of shared prefixes (KvCache.shared) beside other streams' work, and what a
call with one reports."""

import pytest
import torch

from test_gpu_attn import BF, _built  # noqa: F401
from test_gpu_shared import handles, i32, make, widened

pytestmark = pytest.mark.gpu


def test_a_bad_page_of_a_prefix_is_reported_under_a_sequence():
    """Not under its group: the first sequence of the group, whose row of the page
    table is read for all."""
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    data = make([(300, [(3, 1)] * 3), (200, [(5, 1)]), (400, [(3, 1), (9, 2)])], 4, 2, 64, 16, BF, 20)
    attn, q, batch, groups = handles(data)
    table = data[3].clone()
    table[4:, 2] = 1 << 20  # page 2 of the last group's sequences, 4 and 5
    bad = pkg.KvBatch(widened(table, data[1]).cuda(), batch.lens, batch.cu)
    attn.forward(q, bad, shared=attn.cache.shared(bad, groups))
    status, _, sequence = attn.device_status()
    assert status == B.DG_ERR_DEVICE_CHECK and sequence == 4


BUSY = 200_000_000  # cycles: about 0.1 s


@pytest.mark.parametrize("named", [True, False])
@pytest.mark.parametrize("call", ["forward", "plan"])
def test_memory_of_a_dropped_plan_outlives_its_calls(call, named):
    """A plan that is dropped while a call that reads or writes it runs on another
    stream: its memory is not given out again before that call is done."""
    data = make([(700, [(40, 1)] * 5)], 4, 2, 64, 16, BF, 21)
    attn, q, batch, groups = handles(data)
    plan = attn.cache.shared(batch, groups.clone())
    out, want = torch.zeros_like(q), attn.forward(q, batch, shared=plan)
    attn.forward(q, batch, out=out, shared=plan)  # (no list of streams begins in a call below)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [(t.numel(), t.data_ptr()) for t in (plan.prefix, plan.groups)]

    def run(**kw):
        if call == "forward":
            attn.forward(q, batch, out=out, shared=plan, **kw)
        else:
            attn.cache.shared(batch, plan.groups, out=plan, **kw)
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        if not named:
            run()
    if named:
        run(stream=side)
    del plan
    new = [torch.empty(n, dtype=torch.int32, device="cuda") for n, _ in sizes]
    assert not {t.data_ptr() for t in new} & {at for _, at in sizes}
    for t in new:
        t.fill_(1)
    torch.cuda.synchronize()
    assert torch.equal(out, want) if call == "forward" else all((t == 1).all() for t in new)
