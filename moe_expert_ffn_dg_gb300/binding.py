"""ctypes binding of the C ABI in ``include/dg_moe.h`` and ``include/dg_attn.h``.

The functions below carry the C names and only marshal arguments; every step
of the block runs in the CUDA library ``lib/libdgmoe.so``.  There is no other
code path: if the library is missing, :func:`load_library` raises.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import (POINTER, c_char_p, c_double, c_float, c_int, c_int64, c_size_t, c_uint,
                    c_void_p)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libdgmoe.so")

DG_OK = 0
DG_ERR_INVALID_ARG = 1
DG_ERR_ALIGNMENT = 2
DG_ERR_UNSUPPORTED = 3
DG_ERR_CUDA = 4
DG_ERR_TIMEOUT = 5
DG_ERR_DEVICE_CHECK = 6
DG_ERR_WORKSPACE = 7

DG_FMT_BF16 = 0
DG_FMT_AFFINE_U4_G64 = 1
DG_FMT_AFFINE_U8_G64 = 2
DG_FMT_NVFP4_G16 = 3

EXPORTED = (
    "dg_moe_workspace_size", "dg_moe_create", "dg_moe_forward", "dg_moe_forward_host",
    "dg_moe_destroy", "dg_moe_last_device_status", "dg_moe_kernel_names",
    "dg_moe_set_profile_events", "dg_moe_status_string", "dg_moe_last_error",
    "dg_moe_route_noalloc", "dg_moe_forward_neighbours", "dg_moe_arm_wait_timeout_test",
    "dg_sc_mlp_workspace_size", "dg_sc_mlp_create", "dg_sc_mlp_forward",
    "dg_sc_mlp_last_device_status", "dg_sc_mlp_destroy", "dg_sc_mlp_kernel_names",
    "dg_sc_mlp_set_profile_events",
)

# include/dg_attn.h
DG_T_BF16 = 0
DG_T_FP16 = 1
DG_T_FP32 = 2

DG_ROPE_HALF = 0
DG_ROPE_INTERLEAVED = 1

DG_ROPE_PLAIN = 0
DG_ROPE_LINEAR = 1
DG_ROPE_BASE = 2
DG_ROPE_RAMP = 3

EXPORTED_ATTN = (
    "dg_rope_create", "dg_rope_destroy", "dg_rope_apply",
    "dg_kv_create", "dg_kv_destroy", "dg_kv_last_device_status", "dg_kv_append", "dg_kv_copy",
    "dg_kv_gather", "dg_kv_select", "dg_kv_shared", "dg_kv_fork_workspace_size", "dg_kv_fork", "dg_kv_fork_last_device_status",
    "dg_attn_workspace_size", "dg_attn_create", "dg_attn_destroy", "dg_attn_forward",
    "dg_attn_shared_workspace_size", "dg_attn_forward_shared", "dg_attn_weights",
    "dg_attn_last_device_status",
)


class dg_moe_config_t(ctypes.Structure):
    _fields_ = [("hidden", c_int), ("n_experts", c_int), ("top_k", c_int),
                ("expert_inter", c_int), ("dense_inter", c_int), ("max_tokens", c_int),
                ("expert_fmt", c_int), ("dense_fmt", c_int), ("router_fmt", c_int),
                ("rms_eps", c_float), ("flags", c_uint)]


class dg_qtensor_t(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("scales", c_void_p), ("biases", c_void_p)]


class dg_moe_weights_t(ctypes.Structure):
    _fields_ = [("router", dg_qtensor_t), ("gate_up", dg_qtensor_t), ("down", dg_qtensor_t),
                ("dense_gate", dg_qtensor_t), ("dense_up", dg_qtensor_t),
                ("dense_down", dg_qtensor_t),
                ("router_scale", c_void_p), ("per_expert_scale", c_void_p),
                ("w_pre_ff", c_void_p), ("w_pre_ff2", c_void_p), ("w_post_ff1", c_void_p),
                ("w_post_ff2", c_void_p), ("w_post_ff", c_void_p), ("router_bias", c_void_p)]


class dg_moe_neighbours_t(ctypes.Structure):
    _fields_ = [("attn_out", c_void_p), ("w_post_attn", c_void_p), ("w_next_in", c_void_p),
                ("next_in", c_void_p), ("h_mid", c_void_p)]


class dg_moe_debug_t(ctypes.Structure):
    _fields_ = [("idx", c_void_p), ("w", c_void_p), ("logits", c_void_p),
                ("offsets", c_void_p), ("perm", c_void_p), ("xd", c_void_p),
                ("xe_perm", c_void_p), ("y_moe", c_void_p), ("y_dense", c_void_p),
                ("n_refined", c_void_p)]


class dg_sc_mlp_config_t(ctypes.Structure):
    _fields_ = [("hidden", c_int), ("inter", c_int), ("max_tokens", c_int), ("fmt", c_int),
                ("rms_eps", c_float), ("flags", c_uint)]


class dg_sc_mlp_weights_t(ctypes.Structure):
    _fields_ = [("gate", dg_qtensor_t), ("up", dg_qtensor_t), ("down", dg_qtensor_t),
                ("pre_norm", c_void_p)]


class dg_heads_t(ctypes.Structure):
    _fields_ = [("p", c_void_p), ("token_stride", c_int64), ("head_stride", c_int64)]


class dg_rope_config_t(ctypes.Structure):
    _fields_ = [("head_dim", c_int), ("rot_dim", c_int), ("layout", c_int), ("scaling", c_int),
                ("theta", c_double), ("factor", c_double), ("orig_len", c_double),
                ("beta_slow", c_double), ("beta_fast", c_double), ("amplitude", c_double),
                ("flags", c_uint)]


class dg_kv_pool_t(ctypes.Structure):
    _fields_ = [("p", c_void_p), ("layer_stride", c_int64), ("page_stride", c_int64),
                ("token_stride", c_int64), ("head_stride", c_int64)]


class dg_kv_config_t(ctypes.Structure):
    _fields_ = [("n_layers", c_int), ("n_pages", c_int), ("page_size", c_int),
                ("n_kv_heads", c_int), ("head_dim", c_int), ("dtype", c_int),
                ("k", dg_kv_pool_t), ("v", dg_kv_pool_t), ("flags", c_uint)]


class dg_kv_batch_t(ctypes.Structure):
    _fields_ = [("page_table", c_void_p), ("table_stride", c_int64), ("lens", c_void_p),
                ("cu", c_void_p), ("n_seqs", c_int), ("max_pages", c_int)]


class dg_kv_fork_t(ctypes.Structure):
    _fields_ = [("n_pages", c_int), ("page_size", c_int), ("row", c_int), ("n_old", c_int),
                ("n_new", c_int), ("table_in", c_void_p), ("lens_in", c_void_p),
                ("ref_in", c_void_p), ("parent", c_void_p), ("grow", c_void_p),
                ("table_out", c_void_p), ("lens_out", c_void_p), ("ref_out", c_void_p),
                ("copies", c_void_p), ("short_by", c_void_p)]


class dg_attn_config_t(ctypes.Structure):
    _fields_ = [("n_q_heads", c_int), ("left", c_int), ("right", c_int), ("scale", c_float),
                ("flags", c_uint)]


class dg_kv_select_t(ctypes.Structure):
    _fields_ = [("weights", c_void_p), ("weights_stride", c_int64), ("lens", c_void_p),
                ("n_seqs", c_int), ("width", c_int), ("budget", c_int), ("first", c_int),
                ("last", c_int), ("keep", c_void_p), ("cu", c_void_p), ("lens_out", c_void_p),
                ("weights_out", c_void_p), ("out_stride", c_int64)]


class dg_attn_shared_t(ctypes.Structure):
    _fields_ = [("groups", c_void_p), ("prefix", c_void_p), ("n_groups", c_int),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t)]


class dg_attn_weights_t(ctypes.Structure):
    _fields_ = [("in", c_void_p), ("out", c_void_p), ("in_stride", c_int64),
                ("out_stride", c_int64), ("width", c_int), ("decay", c_float), ("fresh", c_int)]


class DgError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {dg_moe_status_string(status)} (status {status})")


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} not found: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    lib.dg_moe_workspace_size.argtypes = [POINTER(dg_moe_config_t), POINTER(c_size_t)]
    lib.dg_moe_create.argtypes = [POINTER(dg_moe_config_t), POINTER(dg_moe_weights_t), c_void_p,
                                  c_size_t, POINTER(c_void_p)]
    lib.dg_moe_forward.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p,
                                   POINTER(dg_moe_debug_t)]
    lib.dg_moe_forward_host.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p]
    lib.dg_moe_forward_neighbours.argtypes = [c_void_p, c_void_p, POINTER(dg_moe_neighbours_t),
                                              c_void_p, c_int, c_float, c_void_p,
                                              POINTER(dg_moe_debug_t)]
    lib.dg_moe_destroy.argtypes = [c_void_p]
    lib.dg_moe_last_device_status.argtypes = [c_void_p, c_void_p, POINTER(c_uint), POINTER(c_uint)]
    lib.dg_moe_kernel_names.argtypes = [c_void_p, POINTER(c_char_p), POINTER(c_int)]
    lib.dg_moe_set_profile_events.argtypes = [c_void_p, POINTER(c_void_p), c_int]
    lib.dg_moe_arm_wait_timeout_test.argtypes = [c_void_p]
    lib.dg_moe_route_noalloc.argtypes = [POINTER(dg_moe_config_t), POINTER(dg_moe_weights_t),
                                         c_void_p, c_int, c_void_p, c_void_p, c_void_p]
    lib.dg_sc_mlp_workspace_size.argtypes = [POINTER(dg_sc_mlp_config_t), POINTER(c_size_t)]
    lib.dg_sc_mlp_create.argtypes = [POINTER(dg_sc_mlp_config_t), POINTER(dg_sc_mlp_weights_t),
                                     c_void_p, c_size_t, POINTER(c_void_p)]
    lib.dg_sc_mlp_forward.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p]
    lib.dg_sc_mlp_last_device_status.argtypes = [c_void_p, c_void_p]
    lib.dg_sc_mlp_destroy.argtypes = [c_void_p]
    lib.dg_sc_mlp_kernel_names.argtypes = [c_void_p, POINTER(c_char_p), POINTER(c_int)]
    lib.dg_sc_mlp_set_profile_events.argtypes = [c_void_p, POINTER(c_void_p), c_int]
    lib.dg_moe_status_string.argtypes = [c_int]
    lib.dg_moe_status_string.restype = c_char_p
    lib.dg_moe_last_error.argtypes = [c_void_p]
    lib.dg_moe_last_error.restype = c_char_p
    for name in EXPORTED:
        if name not in ("dg_moe_status_string", "dg_moe_last_error"):
            getattr(lib, name).restype = c_int
    status_of = [c_void_p, c_void_p, POINTER(c_uint), POINTER(c_uint)]
    heads = POINTER(dg_heads_t)
    lib.dg_rope_create.argtypes = [POINTER(dg_rope_config_t), POINTER(c_void_p)]
    lib.dg_rope_destroy.argtypes = [c_void_p]
    lib.dg_rope_apply.argtypes = [c_void_p, c_int, heads, heads, c_void_p, c_int, c_int, c_int,
                                  c_void_p]
    lib.dg_kv_create.argtypes = [POINTER(dg_kv_config_t), c_void_p, POINTER(c_void_p)]
    lib.dg_kv_destroy.argtypes = [c_void_p]
    lib.dg_kv_last_device_status.argtypes = status_of
    lib.dg_kv_append.argtypes = [c_void_p, c_int, c_void_p, heads, heads, heads, heads, c_int,
                                 POINTER(dg_kv_batch_t), c_void_p, c_int, c_void_p]
    lib.dg_kv_copy.argtypes = [c_void_p, c_void_p, c_int, c_void_p]
    lib.dg_kv_gather.argtypes = [c_void_p, c_void_p, c_int64, c_int, c_void_p, c_int64, c_int,
                                 c_void_p, c_int, c_void_p, c_int, c_void_p]
    lib.dg_kv_select.argtypes = [c_void_p, POINTER(dg_kv_select_t), c_void_p]
    lib.dg_kv_shared.argtypes = [c_void_p, POINTER(dg_kv_batch_t), c_void_p, c_int, c_void_p,
                                 c_void_p]
    lib.dg_kv_fork_workspace_size.argtypes = [c_int, POINTER(c_size_t)]
    lib.dg_kv_fork.argtypes = [POINTER(dg_kv_fork_t), c_void_p, c_size_t, c_void_p]
    lib.dg_kv_fork_last_device_status.argtypes = status_of
    lib.dg_attn_workspace_size.argtypes = [POINTER(dg_attn_config_t), c_void_p,
                                           POINTER(c_size_t)]
    lib.dg_attn_create.argtypes = [POINTER(dg_attn_config_t), c_void_p, c_void_p, c_size_t,
                                   POINTER(c_void_p)]
    lib.dg_attn_destroy.argtypes = [c_void_p]
    lib.dg_attn_forward.argtypes = [c_void_p, c_int, heads, heads, c_void_p,
                                    POINTER(dg_kv_batch_t), c_int, c_void_p]
    lib.dg_attn_shared_workspace_size.argtypes = [POINTER(dg_attn_config_t), c_void_p, c_int,
                                                  POINTER(c_size_t)]
    lib.dg_attn_forward_shared.argtypes = [c_void_p, c_int, heads, heads, c_void_p,
                                           POINTER(dg_kv_batch_t), POINTER(dg_attn_shared_t),
                                           c_int, c_void_p]
    lib.dg_attn_weights.argtypes = [c_void_p, c_int, heads, c_void_p, POINTER(dg_attn_weights_t),
                                    POINTER(dg_kv_batch_t), c_int, c_void_p]
    lib.dg_attn_last_device_status.argtypes = status_of
    for name in EXPORTED_ATTN:
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def dg_moe_status_string(status: int) -> str:
    return load_library().dg_moe_status_string(status).decode()


def _check(status: int, what: str, handle: int = None) -> None:
    if status != DG_OK:
        detail = ""
        if handle and status == DG_ERR_CUDA:
            detail = " [" + dg_moe_last_error(handle) + "]"
        raise DgError(status, what + detail)


def dg_moe_last_error(handle: int) -> str:
    return load_library().dg_moe_last_error(c_void_p(handle)).decode()


def dg_moe_workspace_size(cfg: dg_moe_config_t) -> int:
    n = c_size_t(0)
    _check(load_library().dg_moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "dg_moe_workspace_size")
    return n.value


def dg_moe_create(cfg: dg_moe_config_t, weights: dg_moe_weights_t, workspace: int,
                  workspace_bytes: int) -> int:
    h = c_void_p(0)
    _check(load_library().dg_moe_create(ctypes.byref(cfg), ctypes.byref(weights),
                                        c_void_p(workspace), workspace_bytes, ctypes.byref(h)),
           "dg_moe_create")
    return h.value


def dg_moe_forward(handle: int, h_in: int, h_out: int, n_tokens: int, layer_scalar: float,
                   stream: int, dbg: dg_moe_debug_t | None = None) -> None:
    _check(load_library().dg_moe_forward(c_void_p(handle), c_void_p(h_in), c_void_p(h_out),
                                         n_tokens, layer_scalar, c_void_p(stream),
                                         ctypes.byref(dbg) if dbg is not None else None),
           "dg_moe_forward", handle)


def dg_moe_forward_neighbours(handle: int, x: int, nb: dg_moe_neighbours_t, out: int,
                              n_tokens: int, layer_scalar: float, stream: int,
                              dbg: dg_moe_debug_t | None = None) -> None:
    _check(load_library().dg_moe_forward_neighbours(
        c_void_p(handle), c_void_p(x), ctypes.byref(nb) if nb is not None else None,
        c_void_p(out), n_tokens, layer_scalar, c_void_p(stream),
        ctypes.byref(dbg) if dbg is not None else None), "dg_moe_forward_neighbours", handle)


def dg_moe_forward_host(handle: int, h_in_host: int, h_out_host: int, n_tokens: int,
                        layer_scalar: float, stream: int) -> None:
    _check(load_library().dg_moe_forward_host(c_void_p(handle), c_void_p(h_in_host),
                                              c_void_p(h_out_host), n_tokens, layer_scalar,
                                              c_void_p(stream)),
           "dg_moe_forward_host", handle)


def dg_moe_destroy(handle: int) -> None:
    _check(load_library().dg_moe_destroy(c_void_p(handle)), "dg_moe_destroy")


def dg_moe_last_device_status(handle: int, stream: int):
    """(status, where, info) of the device status word; clears it."""
    where, info = c_uint(0), c_uint(0)
    s = load_library().dg_moe_last_device_status(c_void_p(handle), c_void_p(stream),
                                                 ctypes.byref(where), ctypes.byref(info))
    return s, where.value, info.value


def _kernel_names(fn, handle: int) -> list:
    n = c_int(0)
    _check(fn(c_void_p(handle), None, ctypes.byref(n)), fn.__name__)
    arr = (c_char_p * n.value)()
    _check(fn(c_void_p(handle), arr, ctypes.byref(n)), fn.__name__)
    return [a.decode() for a in arr]


def _set_profile_events(fn, handle: int, events) -> None:
    if events is None:
        _check(fn(c_void_p(handle), None, 0), fn.__name__)
        _EVENT_ARRAYS.pop(handle, None)
        return
    arr = (c_void_p * len(events))(*events)
    _check(fn(c_void_p(handle), arr, len(events)), fn.__name__)
    # keep the array alive as long as the handle may use it
    _EVENT_ARRAYS[handle] = arr


def dg_moe_kernel_names(handle: int) -> list:
    return _kernel_names(load_library().dg_moe_kernel_names, handle)


def dg_moe_set_profile_events(handle: int, events) -> None:
    """events: list of cudaEvent_t handles (ints), or None to switch off."""
    _set_profile_events(load_library().dg_moe_set_profile_events, handle, events)


def dg_moe_arm_wait_timeout_test(handle: int) -> None:
    """Arm the bounded-wait test for the handle's next forward (see
    include/dg_moe.h): one device wait runs out after 10 ms and reports
    DG_ERR_TIMEOUT through dg_moe_last_device_status."""
    _check(load_library().dg_moe_arm_wait_timeout_test(c_void_p(handle)),
           "dg_moe_arm_wait_timeout_test")


def dg_sc_mlp_kernel_names(handle: int) -> list:
    return _kernel_names(load_library().dg_sc_mlp_kernel_names, handle)


def dg_sc_mlp_set_profile_events(handle: int, events) -> None:
    _set_profile_events(load_library().dg_sc_mlp_set_profile_events, handle, events)


_EVENT_ARRAYS: dict = {}


def dg_moe_route_noalloc(cfg: dg_moe_config_t, weights: dg_moe_weights_t, h_in: int,
                         n_tokens: int, idx_out: int, w_out: int, stream: int) -> None:
    """Routing only, with the library's fixed device scratch (no allocation);
    see include/dg_moe.h."""
    _check(load_library().dg_moe_route_noalloc(ctypes.byref(cfg), ctypes.byref(weights),
                                               c_void_p(h_in), n_tokens, c_void_p(idx_out),
                                               c_void_p(w_out), c_void_p(stream)),
           "dg_moe_route_noalloc")


def dg_sc_mlp_workspace_size(cfg: dg_sc_mlp_config_t) -> int:
    n = c_size_t(0)
    _check(load_library().dg_sc_mlp_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "dg_sc_mlp_workspace_size")
    return n.value


def dg_sc_mlp_create(cfg: dg_sc_mlp_config_t, weights: dg_sc_mlp_weights_t, workspace: int,
                     workspace_bytes: int) -> int:
    h = c_void_p(0)
    _check(load_library().dg_sc_mlp_create(ctypes.byref(cfg), ctypes.byref(weights),
                                           c_void_p(workspace), workspace_bytes, ctypes.byref(h)),
           "dg_sc_mlp_create")
    return h.value


def dg_sc_mlp_forward(handle: int, embeds: int, signal: int, out: int, n_tokens: int,
                      stream: int) -> None:
    _check(load_library().dg_sc_mlp_forward(c_void_p(handle), c_void_p(embeds), c_void_p(signal),
                                            c_void_p(out), n_tokens, c_void_p(stream)),
           "dg_sc_mlp_forward")


def dg_sc_mlp_last_device_status(handle: int, stream: int) -> int:
    return load_library().dg_sc_mlp_last_device_status(c_void_p(handle), c_void_p(stream))


def dg_sc_mlp_destroy(handle: int) -> None:
    _check(load_library().dg_sc_mlp_destroy(c_void_p(handle)), "dg_sc_mlp_destroy")


# ---------------------------------------------------------------- dg_attn.h

def dg_rope_create(cfg: dg_rope_config_t) -> int:
    h = c_void_p(0)
    _check(load_library().dg_rope_create(ctypes.byref(cfg), ctypes.byref(h)), "dg_rope_create")
    return h.value


def dg_rope_destroy(handle: int) -> None:
    _check(load_library().dg_rope_destroy(handle), "dg_rope_destroy")


def dg_rope_apply(handle: int, dtype: int, x: dg_heads_t, out: dg_heads_t, positions: int,
                  n_tokens: int, n_heads: int, grad: int, stream: int) -> None:
    _check(load_library().dg_rope_apply(handle, dtype, x, out, positions, n_tokens, n_heads, grad,
                                        stream), "dg_rope_apply")


def dg_kv_create(cfg: dg_kv_config_t, status: int) -> int:
    h = c_void_p(0)
    _check(load_library().dg_kv_create(ctypes.byref(cfg), status, ctypes.byref(h)),
           "dg_kv_create")
    return h.value


def dg_kv_destroy(handle: int) -> None:
    _check(load_library().dg_kv_destroy(handle), "dg_kv_destroy")


def dg_kv_append(handle: int, layer: int, rope: int | None, k: dg_heads_t, v: dg_heads_t,
                 q: dg_heads_t | None, q_out: dg_heads_t | None, n_q_heads: int,
                 batch: dg_kv_batch_t, positions: int | None, n_tokens: int,
                 stream: int) -> None:
    _check(load_library().dg_kv_append(handle, layer, rope, k, v, q, q_out, n_q_heads, batch,
                                       positions, n_tokens, stream), "dg_kv_append")


def dg_kv_copy(handle: int, copies: int, n: int, stream: int) -> None:
    _check(load_library().dg_kv_copy(handle, copies, n, stream), "dg_kv_copy")


def dg_kv_gather(handle: int, src_table: int, src_stride: int, src_pages: int, dst_table: int,
                 dst_stride: int, dst_pages: int, cu: int, n_seqs: int, keep: int, n_keep: int,
                 stream: int) -> None:
    _check(load_library().dg_kv_gather(handle, src_table, src_stride, src_pages, dst_table,
                                       dst_stride, dst_pages, cu, n_seqs, keep, n_keep, stream),
           "dg_kv_gather")


def dg_kv_select(handle: int, s: dg_kv_select_t, stream: int) -> None:
    _check(load_library().dg_kv_select(handle, s, stream), "dg_kv_select")


def dg_kv_shared(handle: int, batch: dg_kv_batch_t, groups: int, n_groups: int, prefix: int,
                 stream: int) -> None:
    _check(load_library().dg_kv_shared(handle, batch, groups, n_groups, prefix, stream),
           "dg_kv_shared")


def dg_kv_fork_workspace_size(n_pages: int) -> int:
    n = c_size_t(0)
    _check(load_library().dg_kv_fork_workspace_size(n_pages, ctypes.byref(n)),
           "dg_kv_fork_workspace_size")
    return n.value


def dg_kv_fork(f: dg_kv_fork_t, workspace: int, workspace_bytes: int, stream: int) -> None:
    _check(load_library().dg_kv_fork(f, workspace, workspace_bytes, stream), "dg_kv_fork")


def dg_attn_workspace_size(cfg: dg_attn_config_t, kv: int) -> int:
    n = c_size_t(0)
    _check(load_library().dg_attn_workspace_size(ctypes.byref(cfg), kv, ctypes.byref(n)),
           "dg_attn_workspace_size")
    return n.value


def dg_attn_create(cfg: dg_attn_config_t, kv: int, workspace: int, workspace_bytes: int) -> int:
    h = c_void_p(0)
    _check(load_library().dg_attn_create(ctypes.byref(cfg), kv, workspace, workspace_bytes,
                                         ctypes.byref(h)), "dg_attn_create")
    return h.value


def dg_attn_destroy(handle: int) -> None:
    _check(load_library().dg_attn_destroy(handle), "dg_attn_destroy")


def dg_attn_forward(handle: int, layer: int, q: dg_heads_t, out: dg_heads_t, lse: int | None,
                    batch: dg_kv_batch_t, n_tokens: int, stream: int) -> None:
    _check(load_library().dg_attn_forward(handle, layer, q, out, lse, batch, n_tokens, stream),
           "dg_attn_forward")


def dg_attn_shared_workspace_size(cfg: dg_attn_config_t, kv: int, n_tokens: int) -> int:
    n = c_size_t(0)
    _check(load_library().dg_attn_shared_workspace_size(ctypes.byref(cfg), kv, n_tokens,
                                                        ctypes.byref(n)),
           "dg_attn_shared_workspace_size")
    return n.value


def dg_attn_forward_shared(handle: int, layer: int, q: dg_heads_t, out: dg_heads_t,
                           lse: int | None, batch: dg_kv_batch_t, shared: dg_attn_shared_t,
                           n_tokens: int, stream: int) -> None:
    _check(load_library().dg_attn_forward_shared(handle, layer, q, out, lse, batch, shared,
                                                 n_tokens, stream), "dg_attn_forward_shared")


def dg_attn_weights(handle: int, layer: int, q: dg_heads_t, lse: int, w: dg_attn_weights_t,
                    batch: dg_kv_batch_t, n_tokens: int, stream: int) -> None:
    _check(load_library().dg_attn_weights(handle, layer, q, lse, w, batch, n_tokens, stream),
           "dg_attn_weights")


def _device_status(fn, handle: int, stream: int):
    where, info = c_uint(0), c_uint(0)
    s = fn(handle, stream, ctypes.byref(where), ctypes.byref(info))
    return s, where.value, info.value


def dg_kv_last_device_status(handle: int, stream: int):
    """(status, where, info) of the cache's device status word; clears it."""
    return _device_status(load_library().dg_kv_last_device_status, handle, stream)


def dg_kv_fork_last_device_status(workspace: int, stream: int):
    return _device_status(load_library().dg_kv_fork_last_device_status, workspace, stream)


def dg_attn_last_device_status(handle: int, stream: int):
    return _device_status(load_library().dg_attn_last_device_status, handle, stream)
