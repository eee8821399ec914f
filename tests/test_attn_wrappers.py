"""The Python holders of the attention half without a GPU: what they refuse
before anything reaches the library."""

import pytest
import torch

import moe_expert_ffn_dg_gb300 as pkg

BF = torch.bfloat16


class Stream:
    """Stands for a stream that the caller names."""
    cuda_stream = 0


@pytest.fixture(scope="module", autouse=True)
def _built():
    pkg.build()


def test_host_memory_is_refused():
    """A kernel must not be given a pointer to host memory, with a stream named
    or without."""
    rope = pkg.Rope(64)
    x, pos = torch.zeros(2, 3, 64, dtype=BF), torch.zeros(2, dtype=torch.int32)
    for kw in ({}, dict(stream=Stream()), dict(stream=Stream(), out=x)):
        with pytest.raises(ValueError):
            rope.apply(x, pos, **kw)
    pool = torch.zeros(1, 4, 16, 1, 64, dtype=BF)
    with pytest.raises(ValueError):
        pkg.KvCache(pool, pool.clone())
    with pytest.raises(ValueError):
        pkg.KvPager(8, 16, device="cpu")
