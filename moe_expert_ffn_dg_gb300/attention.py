"""PyTorch-side holders of the attention half of a decoder layer: rotary
positions, the paged key/value cache and its page operations, and attention of
new tokens over the cache.

PyTorch only allocates device memory and supplies the CUDA stream; every step
runs in the CUDA library through the C ABI (``include/dg_attn.h``).  The cache and
the attention over it are for serving: autograd records nothing of their calls.
"""

from __future__ import annotations

import math

import torch

from . import binding as B
from .block import _Memory, _results, _settle, _stream

_DTYPES = {torch.bfloat16: B.DG_T_BF16, torch.float16: B.DG_T_FP16, torch.float32: B.DG_T_FP32}
_LAYOUTS = {"half": B.DG_ROPE_HALF, "interleaved": B.DG_ROPE_INTERLEAVED}
_SCALINGS = {"none": B.DG_ROPE_PLAIN, "linear": B.DG_ROPE_LINEAR, "base": B.DG_ROPE_BASE,
             "ramp": B.DG_ROPE_RAMP}


def _new(like: torch.Tensor, stream=None) -> torch.Tensor:
    """A contiguous tensor of the same shape for a call on `stream`."""
    return _results(lambda: (torch.empty(like.shape, dtype=like.dtype, device=like.device),),
                    like.device, stream)[0]


def _heads(t: torch.Tensor, dtype, device, dim: int, what: str) -> B.dg_heads_t:
    """A [tokens, heads, dim] tensor as the library takes it."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != dim or (stride[2] != 1 and dim > 1):
        raise ValueError(f"{what}: [tokens, heads, {dim}] with the last dimension contiguous")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what}: {dtype} on {device} expected, got {t.dtype} on {t.device}")
    return B.dg_heads_t(t.data_ptr(), stride[0], stride[1])


def _ints(t: torch.Tensor, device, shape: tuple, what: str) -> int:
    """Pointer of a contiguous int32 device tensor of the given shape."""
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous int32 on {device} expected")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {shape} expected, got {tuple(t.shape)}")
    return t.data_ptr()


def _weights(t: torch.Tensor, device, n: int, what: str):
    """Pointer and row stride of an fp32 [n, width] tensor with contiguous rows."""
    if t.dim() != 2 or t.shape[0] != n or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: [n_seqs, width] with contiguous rows")
    if t.dtype != torch.float32 or t.device != device:
        raise ValueError(f"{what}: fp32 on {device} expected, got {t.dtype} on {t.device}")
    return t.data_ptr(), t.stride(0) if n > 1 else t.shape[1]


class _Handle:
    """Owner of a C handle."""

    _destroy = None
    handle = None

    def close(self):
        if self.handle:
            type(self)._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Rope(_Handle):
    """Rotary positions of heads of ``head_dim`` elements, the first
    ``rot_dim`` of them rotated (default: all).  ``layout``: "half" pairs
    element i with i + rot_dim / 2, "interleaved" 2i with 2i + 1.  ``scaling``
    for contexts longer than the trained ``orig_len`` by ``factor``: "none",
    "linear", "base" (raised theta) or "ramp" (slow pairs stretched, fast ones
    kept, a ramp between ``beta_slow`` and ``beta_fast`` turns)."""

    _destroy = staticmethod(B.dg_rope_destroy)

    def __init__(self, head_dim: int, *, rot_dim: int = None, layout: str = "half",
                 theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 orig_len: float = 0.0, beta_slow: float = 1.0, beta_fast: float = 32.0,
                 amplitude: float = 1.0):
        if layout not in _LAYOUTS or scaling not in _SCALINGS:
            raise ValueError(f"layout {layout!r} or scaling {scaling!r} unknown")
        self.head_dim = head_dim
        self.cfg = B.dg_rope_config_t(head_dim, head_dim if rot_dim is None else rot_dim,
                                      _LAYOUTS[layout], _SCALINGS[scaling], theta, factor,
                                      orig_len, beta_slow, beta_fast, amplitude, 0)
        self.handle = B.dg_rope_create(self.cfg)

    def apply(self, x: torch.Tensor, positions: torch.Tensor, out: torch.Tensor = None,
              grad: bool = False, stream=None) -> torch.Tensor:
        """x [tokens, heads, head_dim] (bf16, fp16 or fp32) rotated by
        positions (int32 [tokens]); grad=True: the transposed rotation, which
        takes a gradient of the output to the gradient of the input.  out may
        be x.  Autograd records the call if x requires a gradient and no out is
        given."""
        if not x.is_cuda or x.dtype not in _DTYPES:
            raise ValueError("x: bf16, fp16 or fp32 on a GPU")
        if out is None:
            if x.requires_grad and torch.is_grad_enabled():
                return _Rotation.apply(x, self, positions, grad, stream)
            out = _new(x, stream)
        elif out.shape != x.shape:
            raise ValueError("out: of x's shape")
        B.dg_rope_apply(self.handle, _DTYPES[x.dtype],
                        _heads(x, x.dtype, x.device, self.head_dim, "x"),
                        _heads(out, x.dtype, x.device, self.head_dim, "out"),
                        _ints(positions, x.device, (x.shape[0],), "positions"), x.shape[0],
                        x.shape[1], int(grad), _stream(x.device, stream))
        return out


class _Rotation(torch.autograd.Function):
    """A rotation that autograd records: its gradient is the transposed one."""

    @staticmethod
    def forward(ctx, x, rope, positions, grad, stream):
        ctx.save_for_backward(positions)
        ctx.rope, ctx.grad = rope, grad
        return rope.apply(x, positions, grad=grad, stream=stream)

    @staticmethod
    def backward(ctx, g):
        if g.stride(2) != 1:  # a broadcast one
            g = g.contiguous()
        return ctx.rope.apply(g, *ctx.saved_tensors, grad=not ctx.grad), None, None, None, None


class KvBatch:
    """The sequences of a call: page_table [n_seqs, max_pages], lens [n_seqs]
    (tokens in the cache, this call's included) and cu [n_seqs + 1] (this
    call's tokens of sequence s are rows cu[s] .. cu[s + 1]), all int32.  The
    tensors may be rewritten between calls; their contents are read by the
    kernels."""

    def __init__(self, page_table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor):
        n, device = lens.shape[0], lens.device
        if page_table.dim() != 2 or page_table.shape[0] != n or page_table.dtype != torch.int32 \
                or page_table.device != device or (page_table.shape[1] > 1
                                                   and page_table.stride(1) != 1):
            raise ValueError("page_table: int32 [n_seqs, max_pages] with contiguous rows")
        self.page_table, self.lens, self.cu, self.device = page_table, lens, cu, device
        stride = page_table.stride(0) if n > 1 else page_table.shape[1]
        self.c = B.dg_kv_batch_t(page_table.data_ptr(), stride, _ints(lens, device, (n,), "lens"),
                                 _ints(cu, device, (n + 1,), "cu"), n, page_table.shape[1])


class KvShared(_Memory):
    """What the sequences of a batch's groups have in common (of
    :meth:`KvCache.shared`): prefix int32 [n_seqs], the tokens that lie in the
    same pages in all of a sequence's group.  It holds for the batch's tensors as
    they were then.  A plan may be dropped while calls with it are under way, on
    any stream."""

    def __init__(self, batch: KvBatch, groups: torch.Tensor, prefix: torch.Tensor):
        if groups.dim() != 1 or groups.shape[0] < 1:
            raise ValueError("groups: [n_groups + 1]")
        self.batch, self.groups, self.prefix = batch, groups, prefix
        self.device, n = batch.device, groups.shape[0]
        self.c = B.dg_attn_shared_t(_ints(groups, batch.device, (n,), "groups"),
                                    _ints(prefix, batch.device, (batch.c.n_seqs,), "prefix"),
                                    n - 1, None, 0)
        self._own(prefix, groups)


class KvKeep:
    """The tokens that stay (of :meth:`KvCache.select`): their places keep
    [n_seqs * budget] (-1 behind the last), cu [n_seqs + 1] and lens [n_seqs],
    all int32, and their weights [n_seqs, budget]."""

    __slots__ = ("keep", "cu", "lens", "weights")

    def __init__(self, keep, cu, lens, weights):
        self.keep, self.cu, self.lens, self.weights = keep, cu, lens, weights


class KvCache(_Handle, _Memory):
    """Paged key/value cache of several layers over the caller's pools
    [n_layers, n_pages, page_size, n_kv_heads, head_dim] (bf16 or fp16, the
    last dimension contiguous)."""

    _destroy = staticmethod(B.dg_kv_destroy)

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        if k_pages.dim() != 5 or k_pages.shape != v_pages.shape or \
                k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            raise ValueError("pools: two [layers, pages, page_size, kv_heads, head_dim] tensors "
                             "of one type on one device")
        if not k_pages.is_cuda or k_pages.stride(4) != 1 or v_pages.stride(4) != 1:
            raise ValueError("pools: on a GPU, last dimension contiguous")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.dtype, self.device = k_pages.dtype, k_pages.device
        (self.n_layers, self.n_pages, self.page_size, self.n_kv_heads,
         self.head_dim) = k_pages.shape
        self._status = torch.zeros(256, dtype=torch.uint8, device=self.device)
        self._own(self._status)
        pools = [B.dg_kv_pool_t(t.data_ptr(), *t.stride()[:4]) for t in (k_pages, v_pages)]
        self.cfg = B.dg_kv_config_t(self.n_layers, self.n_pages, self.page_size, self.n_kv_heads,
                                    self.head_dim, _DTYPES.get(self.dtype, -1), *pools, 0)
        _settle(self.device)
        self.handle = B.dg_kv_create(self.cfg, self._status.data_ptr())

    def append(self, k: torch.Tensor, v: torch.Tensor, batch: KvBatch, layer: int = 0,
               q: torch.Tensor = None, rope: Rope = None, positions: torch.Tensor = None,
               q_out: torch.Tensor = None, stream=None):
        """Write the new tokens' k and v [tokens, kv_heads, head_dim] into
        their pages of one layer, k rotated by ``rope`` on the way.  q [tokens,
        q_heads, head_dim], if given, is rotated too and returned (in q_out,
        which may be q).  positions: rotary positions, by default the tokens'
        places in the cache."""
        n = k.shape[0]
        if k.shape != (n, self.n_kv_heads, self.head_dim) or v.shape != k.shape:
            raise ValueError("k, v: [tokens, kv_heads, head_dim]")
        ck = _heads(k, self.dtype, self.device, self.head_dim, "k")
        cv = _heads(v, self.dtype, self.device, self.head_dim, "v")
        cq = co = None
        if q is not None:
            if q_out is None:
                q_out = _new(q, stream)
            if q.shape[0] != n or q_out.shape != q.shape:
                raise ValueError("q, q_out: one row a token")
            cq = _heads(q, self.dtype, self.device, self.head_dim, "q")
            co = _heads(q_out, self.dtype, self.device, self.head_dim, "q_out")
        B.dg_kv_append(self.handle, layer, rope.handle if rope is not None else None, ck, cv, cq,
                       co, q.shape[1] if q is not None else 0, self._batch(batch),
                       _ints(positions, self.device, (n,), "positions")
                       if positions is not None else None, n, self._use(stream))
        return q_out

    def _batch(self, batch: KvBatch):
        if batch.device != self.device:
            raise ValueError(f"batch on {batch.device}, cache on {self.device}")
        return batch.c

    def copy(self, copies: torch.Tensor, stream=None) -> None:
        """Copy pages, all layers: copies int32 [n, 3] rows (source page,
        destination page, tokens); rows with a negative source do nothing."""
        B.dg_kv_copy(self.handle, _ints(copies, self.device, (copies.shape[0], 3), "copies"),
                     copies.shape[0], self._use(stream))

    def gather(self, src_table: torch.Tensor, dst_table: torch.Tensor, cu: torch.Tensor,
               keep: torch.Tensor, stream=None) -> None:
        """Compact, all layers: token i of sequence s in the pages of dst_table
        becomes its token keep[cu[s] + i] in the pages of src_table.  The two
        tables' pages must differ."""
        n = cu.shape[0] - 1
        src = _ints(src_table, self.device, (n, src_table.shape[1]), "src_table")
        dst = _ints(dst_table, self.device, (n, dst_table.shape[1]), "dst_table")
        B.dg_kv_gather(self.handle, src, src_table.shape[1], src_table.shape[1], dst,
                       dst_table.shape[1], dst_table.shape[1],
                       _ints(cu, self.device, (n + 1,), "cu"), n,
                       _ints(keep, self.device, (keep.shape[0],), "keep"), keep.shape[0],
                       self._use(stream))

    def select(self, weights: torch.Tensor, lens: torch.Tensor, budget: int, first: int = 0,
               last: int = 0, out: KvKeep = None, stream=None) -> KvKeep:
        """Which tokens of each sequence stay when it is thinned to ``budget``:
        its first ``first`` and last ``last`` ones and, of the others, those
        with the largest weights (fp32 [n_seqs, width], of lens int32 [n_seqs]
        tokens), equal ones in the order of their places; all of them if there
        are no more.  keep and cu are what :meth:`gather` takes.  out.weights
        may be wider than the budget: what lies behind stays as it is."""
        n, dev = lens.shape[0], self.device
        w, stride = _weights(weights, dev, n, "weights")
        width = weights.shape[1]
        most = min(budget, width)
        if budget < 0 or first < 0 or last < 0 or first + last > budget:
            raise ValueError("budget: at least first + last, none of them negative")
        if budget >= width:  # all stay; the C call takes 32 bits
            budget, first, last = width, 0, 0
        if out is None:
            new = lens.new_empty
            out = KvKeep(*_results(lambda: (new(n * most), new(n + 1), new(n),
                                            weights.new_empty((n, most))), dev, stream))
            outputs = (out.keep.data_ptr(), out.cu.data_ptr(), out.lens.data_ptr(),
                       out.weights.data_ptr(), most)
        else:
            if out.weights.dim() != 2 or out.weights.shape[1] < most:
                raise ValueError(f"out.weights: [n_seqs, {most}] or wider")
            outputs = (_ints(out.keep, dev, (n * most,), "out.keep"),
                       _ints(out.cu, dev, (n + 1,), "out.cu"),
                       _ints(out.lens, dev, (n,), "out.lens"),
                       *_weights(out.weights, dev, n, "out.weights"))
        if n == 0:
            with torch.cuda.stream(stream):  # None: the current one
                out.cu.zero_()
        B.dg_kv_select(self.handle, B.dg_kv_select_t(
            w, stride, _ints(lens, dev, (n,), "lens"), n, width, budget, first, last, *outputs),
            self._use(stream))
        return out

    def shared(self, batch: KvBatch, groups: torch.Tensor, out: KvShared = None,
               stream=None) -> KvShared:
        """What the sequences groups[g] .. groups[g + 1] of the batch (int32
        [n_groups + 1], ascending) have in common, for every group: the tokens
        from the first on that lie in the same pages and that all of them had
        before this call's new ones.  For :meth:`PagedAttention.forward`."""
        sequences = self._batch(batch)
        if out is None:
            out = KvShared(batch, groups, *_results(
                lambda: (batch.lens.new_empty(batch.c.n_seqs),), self.device, stream))
            out._seen.add(_stream(self.device))  # the allocator knows of it
        elif out.batch is not batch or out.groups is not groups:
            raise ValueError("out: of this batch and these groups")
        c, raw = out.c, self._use(stream)
        if raw not in out._seen:
            out._use(stream)
        B.dg_kv_shared(self.handle, sequences, c.groups, c.n_groups, c.prefix, raw)
        return out

    def device_status(self, stream=None):
        """(status, where, info) of the device status word; clears it."""
        return B.dg_kv_last_device_status(self.handle, self._use(stream))


class KvFork:
    """What a fork step returns: the new table and lens, the pages' reference
    counts, the pages to copy (for :meth:`KvCache.copy`) and the number of
    pages missing (int32 [1]; 0: every sequence grew)."""

    __slots__ = ("table", "lens", "ref", "copies", "short")

    def __init__(self, table, lens, ref, copies, short):
        self.table, self.lens, self.ref, self.copies, self.short = table, lens, ref, copies, short


class KvPager(_Memory):
    """Bookkeeping of n_pages pages: which sequence holds which, shared ones
    counted.  The state (table, lens, ref) is the caller's; ``fork`` takes it
    one step further.  Calls of one instance share a workspace: they must not
    overlap."""

    def __init__(self, n_pages: int, page_size: int, device="cuda"):
        self.n_pages, self.page_size = n_pages, page_size
        if torch.device(device).type != "cuda":
            raise ValueError(f"pager on a GPU expected, not on {device}")
        self._bytes = B.dg_kv_fork_workspace_size(n_pages)
        # 4-byte elements: aligned as any allocation is
        self.workspace = torch.zeros((self._bytes + 3) // 4, dtype=torch.int32, device=device)
        self.device, self._ws = self.workspace.device, self.workspace.data_ptr()
        self._own(self.workspace)
        # zeroed before any stream uses it
        torch.cuda.current_stream(self.device).synchronize()

    def fork(self, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor,
             parent: torch.Tensor, grow: torch.Tensor, out: KvFork = None,
             stream=None) -> KvFork:
        """New sequence j continues old sequence parent[j] (-1: a new one) and
        gets room for grow[j] more tokens; old sequences without a child are
        freed, shared partly filled pages that grow are split (see
        ``include/dg_attn.h``).  out.ref may be ref."""
        dev, (n_old, row), n_new = self.device, table.shape, parent.shape[0]
        inputs = (_ints(table, dev, (n_old, row), "table"), _ints(lens, dev, (n_old,), "lens"),
                  _ints(ref, dev, (self.n_pages,), "ref"), _ints(parent, dev, (n_new,), "parent"),
                  _ints(grow, dev, (n_new,), "grow"))
        if out is None:
            new = lens.new_empty  # cheaper than views of one allocation
            out = KvFork(*_results(lambda: (new((n_new, row)), new(n_new), new(self.n_pages),
                                            new((n_new, 3)), new(1)), dev, stream))
            outputs = (out.table.data_ptr(), out.lens.data_ptr(), out.ref.data_ptr(),
                       out.copies.data_ptr(), out.short.data_ptr())
        else:
            outputs = (_ints(out.table, dev, (n_new, row), "out.table"),
                       _ints(out.lens, dev, (n_new,), "out.lens"),
                       _ints(out.ref, dev, (self.n_pages,), "out.ref"),
                       _ints(out.copies, dev, (n_new, 3), "out.copies"),
                       _ints(out.short, dev, (1,), "out.short"))
        f = B.dg_kv_fork_t(self.n_pages, self.page_size, row, n_old, n_new, *inputs, *outputs)
        B.dg_kv_fork(f, self._ws, self._bytes, self._use(stream))
        return out

    def device_status(self, stream=None):
        return B.dg_kv_fork_last_device_status(self._ws, self._use(stream))


class PagedAttention(_Handle, _Memory):
    """Attention of new tokens over a :class:`KvCache`.  A query at position p
    sees the keys p - left .. p + right of its sequence; negative: no limit
    (right=0: causal).  scale defaults to head_dim ** -0.5.  shared_tokens: new
    tokens that a call with shared prefixes may have (0: no such calls).  Calls
    of one instance share a workspace: they must not overlap."""

    _destroy = staticmethod(B.dg_attn_destroy)

    def __init__(self, cache: KvCache, n_q_heads: int, left: int = -1, right: int = 0,
                 scale: float = None, shared_tokens: int = 0):
        self.cache, self.n_q_heads, self.device = cache, n_q_heads, cache.device
        self.cfg = B.dg_attn_config_t(n_q_heads, left, right,
                                      1.0 / math.sqrt(cache.head_dim) if scale is None else scale,
                                      0)
        n = B.dg_attn_workspace_size(self.cfg, cache.handle)
        self.shared_tokens = shared_tokens
        self._pre_bytes, room = 0, (n + 1023) // 1024 * 1024
        if shared_tokens:
            self._pre_bytes = B.dg_attn_shared_workspace_size(self.cfg, cache.handle,
                                                              shared_tokens)
            n = room + self._pre_bytes
        self.workspace = torch.empty(n + 1024, dtype=torch.uint8, device=cache.device)
        self._own(self.workspace)
        ptr = (self.workspace.data_ptr() + 1023) // 1024 * 1024
        self._pre = ptr + room
        _settle(cache.device)
        self.handle = B.dg_attn_create(self.cfg, cache.handle, ptr, n)

    def forward(self, q: torch.Tensor, batch: KvBatch, layer: int = 0, out: torch.Tensor = None,
                lse: torch.Tensor = None, stream=None, shared: KvShared = None):
        """q [tokens, n_q_heads, head_dim] -> out of the same shape.  lse: an
        fp32 [tokens, n_q_heads] tensor that receives log sum exp of each
        query's scores; (out, lse) is returned then.  shared: what groups of the
        batch's sequences have in common (:meth:`KvCache.shared`), which is read
        once for all of a group."""
        c = self.cache
        if out is None:
            out = _new(q, stream)
        if q.dim() != 3 or q.shape[1] != self.n_q_heads or out.shape != q.shape:
            raise ValueError("q, out: [tokens, n_q_heads, head_dim]")
        if lse is not None and (lse.dtype != torch.float32 or lse.device != c.device
                                or not lse.is_contiguous()
                                or lse.shape != (q.shape[0], self.n_q_heads)):
            raise ValueError("lse: contiguous fp32 [tokens, n_q_heads]")
        args = (self.handle, layer, _heads(q, c.dtype, c.device, c.head_dim, "q"),
                _heads(out, c.dtype, c.device, c.head_dim, "out"),
                lse.data_ptr() if lse is not None else None, c._batch(batch))
        if shared is None:
            B.dg_attn_forward(*args, q.shape[0], self._use(stream))
        else:
            if shared.batch is not batch:
                raise ValueError("shared: of another batch")
            if q.shape[0] > self.shared_tokens:
                raise ValueError(f"{q.shape[0]} tokens with shared prefixes, room for "
                                 f"{self.shared_tokens} (shared_tokens)")
            s = shared.c
            shared._use(stream)
            B.dg_attn_forward_shared(*args, B.dg_attn_shared_t(
                s.groups, s.prefix, s.n_groups, self._pre, self._pre_bytes), q.shape[0],
                self._use(stream))
        return (out, lse) if lse is not None else out

    def weights(self, q: torch.Tensor, lse: torch.Tensor, batch: KvBatch, weights: torch.Tensor,
                layer: int = 0, decay: float = 1.0, fresh: bool = True, out: torch.Tensor = None,
                stream=None) -> torch.Tensor:
        """Attention weight that each cached token receives: out[s, j] = decay *
        weights[s, j] + the sum over heads and new tokens that see token j of
        exp(scale q k_j - lse), for every token of the batch's sequences.  lse:
        what :meth:`forward` gave for these q.  weights: fp32 [n_seqs, width];
        fresh: those of the call's own new tokens count as 0, whatever they
        hold (pass False for the layers after a step's first, if they share the
        weights).  out may be weights (the default)."""
        c = self.cache
        if q.dim() != 3 or q.shape[1] != self.n_q_heads:
            raise ValueError("q: [tokens, n_q_heads, head_dim]")
        if lse.dtype != torch.float32 or lse.device != c.device or not lse.is_contiguous() \
                or lse.shape != (q.shape[0], self.n_q_heads):
            raise ValueError("lse: contiguous fp32 [tokens, n_q_heads]")
        if out is None:
            out = weights
        if out.shape != weights.shape:
            raise ValueError("out: of weights' shape")
        n = batch.lens.shape[0]
        w, w_stride = _weights(weights, c.device, n, "weights")
        o, o_stride = _weights(out, c.device, n, "out")
        B.dg_attn_weights(self.handle, layer, _heads(q, c.dtype, c.device, c.head_dim, "q"),
                          lse.data_ptr(),
                          B.dg_attn_weights_t(w, o, w_stride, o_stride, weights.shape[1], decay,
                                              int(fresh)), c._batch(batch), q.shape[0],
                          self._use(stream))
        return out

    def device_status(self, stream=None):
        """(status, where, info) of the device status word; clears it."""
        return B.dg_attn_last_device_status(self.handle, self._use(stream))
