"""Refusals of the thinning and sharing entry points that need no GPU."""

import ctypes

import pytest

import moe_expert_ffn_dg_gb300 as pkg
from moe_expert_ffn_dg_gb300 import binding as B

INV = B.DG_ERR_INVALID_ARG
P = 0x10000  # stands for a device pointer; never followed


@pytest.fixture(scope="module")
def lib():
    pkg.build()
    return B.load_library()


def test_null_handles(lib):
    batch, x = B.dg_kv_batch_t(P, 4, P, P, 1, 4), B.dg_heads_t(P, 256, 128)
    s = B.dg_kv_select_t(P, 9, P, 1, 9, 5, 0, 0, P, P, 2 * P, 2 * P, 9)
    w = B.dg_attn_weights_t(P, P, 9, 9, 9, 1.0, 1)
    assert lib.dg_kv_select(None, ctypes.byref(s), None) == INV
    assert lib.dg_kv_shared(None, batch, P, 1, P, None) == INV
    assert lib.dg_attn_weights(None, 0, x, P, ctypes.byref(w), batch, 1, None) == INV


def test_structures_match_the_header():
    """Sizes as the C compiler lays them out: pointers, 64-bit strides, ints."""
    assert ctypes.sizeof(B.dg_kv_select_t) == 3 * 8 + 5 * 4 + 4 + 5 * 8
    assert ctypes.sizeof(B.dg_attn_weights_t) == 4 * 8 + 3 * 4 + 4
