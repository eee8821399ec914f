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
