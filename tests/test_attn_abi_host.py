"""Host-side checks of include/dg_attn.h that need no GPU: every declared
function is exported, and bad arguments are refused before any CUDA call."""

import ctypes
import os
import re

import pytest

import moe_expert_ffn_dg_gb300 as pkg
from moe_expert_ffn_dg_gb300 import binding as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "dg_attn.h")
INV, ALIGN, UNSUP, WS = (B.DG_ERR_INVALID_ARG, B.DG_ERR_ALIGNMENT, B.DG_ERR_UNSUPPORTED,
                         B.DG_ERR_WORKSPACE)
P = 0x10000  # stands for a device pointer; never followed


@pytest.fixture(scope="module")
def lib():
    pkg.build()
    return B.load_library()


def test_library_exports_every_declared_function(lib):
    decl = set(re.findall(r"\b(dg_(?:rope|kv|attn)_\w+)\s*\(", open(HEADER).read()))
    assert decl == set(B.EXPORTED_ATTN)
    for name in decl:
        assert hasattr(lib, name)


def rope_cfg(**kw):
    c = dict(head_dim=128, rot_dim=128, layout=0, scaling=0, theta=1e4, factor=1.0, orig_len=0.0,
             beta_slow=1.0, beta_fast=32.0, amplitude=1.0, flags=0)
    c.update(kw)
    return B.dg_rope_config_t(**c)


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=0), INV), (dict(rot_dim=0), INV), (dict(rot_dim=7), INV),
    (dict(rot_dim=130), INV), (dict(head_dim=514, rot_dim=64), UNSUP), (dict(layout=2), INV),
    (dict(scaling=4), INV), (dict(scaling=-1), INV), (dict(theta=1.0), INV),
    (dict(theta=float("nan")), INV), (dict(theta=float("inf")), INV), (dict(amplitude=0.0), INV),
    (dict(amplitude=float("nan")), INV), (dict(scaling=1, factor=0.5), INV),
    (dict(scaling=2, rot_dim=2), INV), (dict(scaling=3, factor=2.0), INV),
    (dict(scaling=3, factor=2.0, orig_len=10.0, beta_fast=0.5), INV), (dict(flags=1), INV)])
def test_rope_config_refusals(lib, bad, code):
    h = ctypes.c_void_p(1)
    assert lib.dg_rope_create(ctypes.byref(rope_cfg(**bad)), ctypes.byref(h)) == code
    assert h.value is None


@pytest.fixture(scope="module")
def rope(lib):
    h = B.dg_rope_create(rope_cfg())
    yield h
    B.dg_rope_destroy(h)


def test_rope_apply_refusals(lib, rope):
    def go(dtype=0, x=P, xs=(128, 128), out=P, pos=P, n=3, heads=1, handle=rope):
        return lib.dg_rope_apply(handle, dtype, B.dg_heads_t(x, *xs), B.dg_heads_t(out, 128, 128),
                                 pos, n, heads, 0, None)
    assert go(handle=None) == INV
    assert go(dtype=3) == INV and go(n=-1) == INV and go(heads=-1) == INV
    assert go(x=None) == INV and go(out=None) == INV and go(pos=None) == INV
    assert go(xs=(-128, 128)) == INV
    assert go(x=P + 1) == ALIGN and go(dtype=2, x=P + 2) == ALIGN and go(pos=P + 2) == ALIGN
    assert go(n=0) == B.DG_OK and go(heads=0) == B.DG_OK
    assert go(heads=1 << 20) == UNSUP
    assert lib.dg_rope_apply(rope, 0, None, None, P, 3, 1, 0, None) == INV
    assert lib.dg_rope_destroy(None) == B.DG_OK


def kv_cfg(pool=None, **kw):
    p = dict(p=P, layer_stride=8192, page_stride=4096, token_stride=256, head_stride=128)
    p.update(pool or {})
    c = dict(n_layers=1, n_pages=4, page_size=16, n_kv_heads=2, head_dim=128, dtype=0,
             k=B.dg_kv_pool_t(**p), v=B.dg_kv_pool_t(P, 8192, 4096, 256, 128), flags=0)
    c.update(kw)
    return B.dg_kv_config_t(**c)


@pytest.mark.parametrize("bad,code", [
    (dict(n_layers=0), INV), (dict(n_pages=0), INV), (dict(n_kv_heads=0), INV),
    (dict(page_size=24), UNSUP), (dict(page_size=8), UNSUP), (dict(page_size=512), UNSUP),
    (dict(head_dim=96), UNSUP), (dict(dtype=2), UNSUP), (dict(n_kv_heads=257), UNSUP),
    (dict(flags=1), INV), (dict(pool=dict(p=None)), INV), (dict(pool=dict(p=P + 8)), ALIGN),
    (dict(pool=dict(token_stride=-8)), INV), (dict(pool=dict(token_stride=260)), ALIGN),
    (dict(pool=dict(token_stride=64)), INV), (dict(pool=dict(head_stride=64)), INV),
    (dict(pool=dict(page_stride=0)), INV), (dict(pool=dict(page_stride=1 << 37)), INV)])
def test_cache_config_refusals(lib, bad, code):
    h = ctypes.c_void_p(1)
    assert lib.dg_kv_create(ctypes.byref(kv_cfg(**bad)), P, ctypes.byref(h)) == code
    assert h.value is None


def test_cache_status_word_and_null_handles(lib):
    h = ctypes.c_void_p(1)
    assert lib.dg_kv_create(ctypes.byref(kv_cfg()), None, ctypes.byref(h)) == WS
    assert lib.dg_kv_create(ctypes.byref(kv_cfg()), P + 4, ctypes.byref(h)) == WS
    assert lib.dg_kv_create(None, P, ctypes.byref(h)) == INV
    assert lib.dg_kv_create(ctypes.byref(kv_cfg()), P, None) == INV
    assert lib.dg_kv_destroy(None) == B.DG_OK and lib.dg_attn_destroy(None) == B.DG_OK
    batch, x = B.dg_kv_batch_t(P, 4, P, P, 1, 4), B.dg_heads_t(P, 256, 128)
    assert lib.dg_kv_append(None, 0, None, x, x, None, None, 0, batch, None, 1, None) == INV
    assert lib.dg_kv_copy(None, P, 1, None) == INV
    assert lib.dg_kv_gather(None, P, 1, 1, P, 1, 1, P, 1, P, 1, None) == INV
    assert lib.dg_attn_forward(None, 0, x, x, None, batch, 1, None) == INV
    for f in (lib.dg_kv_last_device_status, lib.dg_attn_last_device_status):
        assert f(None, None, None, None) == INV
    assert lib.dg_kv_fork_last_device_status(None, None, None, None) == WS
    n = ctypes.c_size_t(0)
    cfg = B.dg_attn_config_t(8, -1, 0, 0.1, 0)
    assert lib.dg_attn_workspace_size(ctypes.byref(cfg), None, ctypes.byref(n)) == INV
    assert lib.dg_attn_create(ctypes.byref(cfg), None, P, 1 << 30, ctypes.byref(h)) == INV


def fork_args(**kw):
    a = dict(n_pages=100, page_size=16, row=8, n_old=2, n_new=2, table_in=P, lens_in=P, ref_in=P,
             parent=P, grow=P, table_out=2 * P, lens_out=2 * P, ref_out=P, copies=P, short_by=P)
    a.update(kw)
    return B.dg_kv_fork_t(**a)


@pytest.mark.parametrize("bad,code", [
    (dict(n_pages=0), INV), (dict(row=0), INV), (dict(n_old=-1), INV), (dict(n_new=-1), INV),
    (dict(page_size=48), UNSUP), (dict(n_old=4097), UNSUP), (dict(n_new=4097), UNSUP),
    (dict(row=1 << 19), UNSUP), (dict(ref_in=None), INV), (dict(ref_out=None), INV),
    (dict(short_by=None), INV), (dict(table_in=None), INV), (dict(parent=None), INV),
    (dict(copies=None), INV), (dict(grow=P + 2), ALIGN), (dict(table_out=P), INV),
    (dict(lens_out=P), INV)])
def test_fork_refusals(lib, bad, code):
    assert lib.dg_kv_fork(ctypes.byref(fork_args(**bad)), P, 1 << 30, None) == code


def test_fork_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.dg_kv_fork_workspace_size(0, ctypes.byref(n)) == INV
    assert lib.dg_kv_fork_workspace_size(100, None) == INV
    assert lib.dg_kv_fork_workspace_size(1 << 29, ctypes.byref(n)) == UNSUP
    need = B.dg_kv_fork_workspace_size(100)
    f = fork_args()
    assert lib.dg_kv_fork(ctypes.byref(f), None, need, None) == WS
    assert lib.dg_kv_fork(ctypes.byref(f), P, need - 1, None) == WS
    assert lib.dg_kv_fork(ctypes.byref(f), P + 8, need, None) == WS
    assert lib.dg_kv_fork(None, P, need, None) == INV
