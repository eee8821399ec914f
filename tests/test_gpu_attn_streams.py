"""The attention half's handles beside other streams' work: status words,
workspaces and results."""

import pytest
import torch

from test_gpu_attn import BF, _built  # noqa: F401

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
