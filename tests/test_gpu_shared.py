"""Attention of sequences that share a prefix against a 64-bit implementation
that takes them one by one.  Tolerances: those of tests/test_gpu_attn.py, of the
same products; two parts of a row meet in fp32, which the terms there for sums
and for the exponential cover (their factors are off by 2^-21, their sums by three
half steps)."""

import math

import pytest
import torch

import attn_ref
from test_gpu_attn import BF, FP, _built, tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def make(groups, hq, hkv, d, ps, dtype, seed=0):
    """groups: lists of (common tokens, [(own tokens, new ones of them) of each
    sequence]).  Whole pages of what is common are the same pages; unwritten
    places hold NaN."""
    g = torch.Generator().manual_seed(seed)
    rows, lens, n, bounds, used = [], [], [], [0], 0
    for top, members in groups:
        k = top // ps
        shared = list(range(used, used + k))
        used += k
        for own, new in members:
            x = top + own
            more = -(-x // ps) - k
            rows.append(shared + list(range(used, used + more)))
            used += more
            lens.append(x)
            n.append(new)
        bounds.append(len(rows))
    order = torch.randperm(used + 2, generator=g)
    k = torch.full((used + 2, ps, hkv, d), math.nan, dtype=dtype)
    v = k.clone()
    table = torch.full((len(rows), max([1] + [len(r) for r in rows])), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        for i, page in enumerate(r):
            page = int(order[page])
            table[b, i] = page
            m = min(ps, lens[b] - i * ps)
            if torch.isnan(k[page, :m]).any():
                k[page, :m] = torch.randn(m, hkv, d, generator=g).to(dtype)
                v[page, :m] = torch.randn(m, hkv, d, generator=g).to(dtype)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    q = torch.randn(cu[-1], hq, d, generator=g).to(dtype)
    return q, k, v, table, lens, cu, bounds


def widened(table, k):
    """A page table with room for more than 256 MB of keys and values: below that
    sequences are taken one by one."""
    n, (_, ps, hkv, d) = table.shape[0], k.shape
    room = (256 << 20) // (n * ps * hkv * d * 4) + 1
    wide = torch.full((n, max(room, table.shape[1])), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    return wide


def handles(data, left=-1, right=0, wide=True, **kw):
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu, bounds = data
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    batch = pkg.KvBatch((widened(table, k) if wide else table).cuda(), i32(lens), i32(cu))
    attn = pkg.PagedAttention(cache, q.shape[1], left=left, right=right,
                              shared_tokens=max(q.shape[0], 1), **kw)
    return attn, q.cuda(), batch, i32(bounds)


def compare(data, out, lse, left=-1, right=0):
    q, k, v, table, lens, cu, _ = data
    d = q.shape[2]
    ref = attn_ref.attention(q, k, v, table, lens, cu, left, right, d ** -0.5)
    tol, ltol = tolerance(ref, q.dtype, d, max(lens))
    err = (out.double().cpu() - ref[0]).abs()
    assert not torch.isnan(err).any()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    some = ref[1] > -math.inf
    gl = lse.double().cpu()
    assert (gl[~some] == -math.inf).all()
    assert ((gl - ref[1]).abs()[some] <= ltol[some]).all()


def check(data, left=-1, right=0, prefixes=None):
    attn, q, batch, groups = handles(data, left, right)
    shared = attn.cache.shared(batch, groups)
    if prefixes is not None:
        assert shared.prefix.tolist() == prefixes
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    attn.forward(q, batch, out=out, lse=lse, shared=shared)
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0 and attn.cache.device_status()[0] == 0
    compare(data, out, lse, left, right)
    return shared.prefix.tolist()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_single_tokens(d, ps, dtype):
    """Groups of several sizes, one without a fork, one whose prefix is short."""
    got = check(make([(600, [(1, 1), (2, 1), (200, 1)]), (300, [(40, 1)]),
                      (16, [(3, 1), (90, 1)]), (1030, [(1, 1)] * 9)], 8, 2, d, ps, dtype))
    assert max(got) >= 1024 - 16


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 16, 128])
def test_heads_of_a_group(group, d):
    check(make([(300, [(5, 2), (1, 1), (0, 0), (7, 3)])], 2 * group, 2, d, 32, BF, 1))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("members", [2, 33, 70, 150])
def test_many_rows_of_a_group(members, d):
    """Tiles of both variants, ragged ends, parts of several CTAs."""
    check(make([(1600, [(i % 5 + 1, i % 3) for i in range(members)])], 8, 2, d, 64, BF, 2))


@pytest.mark.parametrize("rows", [30, 60, 128, 129, 300])
@pytest.mark.parametrize("d", [64, 256])
def test_rows_of_a_sequence(rows, d):
    """Chunks up to where a prefix is no longer taken together, and past it."""
    check(make([(500, [(rows, rows), (rows + 3, rows - 5)])], 2, 2, d, 16, FP, 3))


@pytest.mark.parametrize("left,right", [(-1, -1), (-1, 5), (40, 0), (0, 0), (1000, 3)])
def test_limits(left, right):
    check(make([(400, [(20, 6), (90, 30), (1, 1)]), (200, [(9, 9)] * 3)], 4, 2, 128, 16, BF, 4),
          left, right)


def test_prefix_lengths_around_a_tile():
    """Prefixes that end inside a page and a tile: the shortest past of a group
    whose rows go on alike."""
    import moe_expert_ffn_dg_gb300 as pkg
    for past in (127, 128, 129, 200, 255, 256, 257, 511):
        data = list(make([(640, [(1, 1), (30, 1), (5, 1)])], 4, 2, 128, 16, BF, 5))
        lens = list(data[4])
        lens[1] = past + 1  # its new token lies on a page of the others
        data[4] = lens
        got = check(tuple(data))
        assert got == [past] * 3 and pkg


def test_groups_leave_sequences_out():
    data = list(make([(300, [(3, 1)] * 3), (200, [(3, 1)] * 4), (500, [(9, 2)] * 2)], 4, 2, 64, 16,
                     BF, 6))
    for bounds in ([3, 7], [0, 2, 2, 5], [9, 9], [0, 1, 2, 3, 9], [4]):
        data[6] = bounds
        check(tuple(data))


def test_no_rows_and_no_groups():
    check(make([(300, [(0, 0)] * 3), (300, [(4, 1)] * 2)], 4, 2, 64, 16, BF, 7))
    attn, q, batch, groups = handles(make([(300, [(0, 0)] * 3)], 4, 2, 64, 16, BF, 7))
    shared = attn.cache.shared(batch, groups)
    assert attn.forward(q, batch, shared=shared).shape == (0, 4, 64)


def test_what_is_not_seen_may_hold_anything():
    """Rows outside every sequence are left as they were."""
    import moe_expert_ffn_dg_gb300 as pkg
    data = make([(300, [(3, 1)] * 3)], 4, 2, 64, 16, BF, 8)
    q, k, v, table, lens, cu, bounds = data
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    attn = pkg.PagedAttention(cache, 4, shared_tokens=8)
    wide = torch.full((8, 4, 64), math.nan, dtype=BF, device="cuda")
    wide[2:5] = q.cuda()
    batch = pkg.KvBatch(widened(table, k).cuda(), i32(lens), i32([c + 2 for c in cu]))
    out, lse = torch.full_like(wide, 7.0), torch.full((8, 4), 7.0, device="cuda")
    attn.forward(wide, batch, out=out, lse=lse, shared=cache.shared(batch, i32(bounds)))
    assert attn.device_status()[0] == 0
    compare(data, out[2:5], lse[2:5])
    for rows in (slice(0, 2), slice(5, 8)):
        assert (out[rows] == 7).all() and (lse[rows] == 7).all()


def test_non_finite_values_reach_the_rows_that_see_them():
    """An infinite score in the prefix, a NaN in one sequence's own tokens."""
    data = make([(300, [(3, 1)] * 3)], 2, 1, 64, 16, BF, 9)
    q, k, v, table, lens, cu, bounds = data
    k[int(table[1, 18]), 13] = math.nan  # token 301 of sequence 1 alone
    attn, qd, batch, groups = handles(data)
    lse = torch.empty(3, 2, device="cuda")
    out, _ = attn.forward(qd, batch, lse=lse, shared=attn.cache.shared(batch, groups))
    bad = torch.isnan(out).flatten(1).all(1)
    assert bad.tolist() == [False, True, False]
    assert torch.isnan(lse).all(1).tolist() == [False, True, False]
    k[int(table[0, 3]), 5] = math.nan  # token 53 of all
    attn, qd, batch, groups = handles(data)
    out = attn.forward(qd, batch, shared=attn.cache.shared(batch, groups))
    assert torch.isnan(out).all()


def test_large_scores():
    """Rows whose weights lie wholly in one of the two parts."""
    data = make([(300, [(9, 1)] * 4)], 4, 2, 128, 16, BF, 10)
    q, k, v, table, lens, cu, bounds = data
    q *= 20
    check(data)


def test_same_result_every_time_and_close_to_the_plain_call():
    data = make([(2000, [(i + 1, 1) for i in range(20)])], 8, 2, 128, 64, BF, 11)
    attn, q, batch, groups = handles(data)
    shared = attn.cache.shared(batch, groups)
    first = attn.forward(q, batch, shared=shared)
    for _ in range(5):
        assert torch.equal(attn.forward(q, batch, shared=shared), first)
    plain = attn.forward(q, batch)
    assert (plain.float() - first.float()).abs().max() <= 2 ** -6


def test_little_is_taken_one_by_one():
    """The same launches as without a plan, so the same bits; not so with room for
    more."""
    data = make([(2000, [(i + 1, 1) for i in range(20)])], 8, 2, 128, 64, BF, 11)
    attn, q, batch, groups = handles(data, wide=False)
    out = attn.forward(q, batch, shared=attn.cache.shared(batch, groups))
    assert torch.equal(out, attn.forward(q, batch))
    attn, q, batch, groups = handles(data)
    assert not torch.equal(attn.forward(q, batch, shared=attn.cache.shared(batch, groups)), out)


def test_captured_with_its_plan_and_replayed_on_new_lengths():
    """A step's graph: the common prefix is found again at every replay."""
    data = make([(700, [(40, 1)] * 5), (300, [(20, 1)] * 2)], 4, 2, 64, 16, BF, 12)
    attn, q, batch, groups = handles(data)
    shared = attn.cache.shared(batch, groups)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    attn.forward(q, batch, out=out, lse=lse, shared=shared)  # kernels are loaded
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.cache.shared(batch, groups, out=shared)
        attn.forward(q, batch, out=out, lse=lse, shared=shared)
    q_, k, v, table, lens, cu, bounds = data
    for cut in (0, 30, 500):
        new = [x - cut if b < 5 else x for b, x in enumerate(lens)]
        batch.lens.copy_(i32(new))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert attn.device_status()[0] == 0
        compare((q_, k, v, table, new, cu, bounds), out, lse)
    assert shared.prefix.tolist()[:5] == [239] * 5


def test_on_a_side_stream_and_two_at_once():
    data = [make([(700, [(40, 1)] * 5)], 4, 2, 64, 16, BF, 13),
            make([(1500, [(9, 2)] * 9)], 8, 2, 128, 64, BF, 14)]
    both = [handles(d) for d in data]
    plans = [a.cache.shared(b, g) for a, _, b, g in both]
    want = [a.forward(q, b, shared=s) for (a, q, b, _), s in zip(both, plans)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for (a, q, b, g), st in zip(both, streams):
            s = a.cache.shared(b, g, stream=st)
            outs.append(a.forward(q, b, shared=s, stream=st))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


def test_bad_prefixes_and_pages_are_reported():
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    data = make([(300, [(3, 1)] * 3)], 4, 2, 64, 16, BF, 15)
    attn, q, batch, groups = handles(data)
    shared = attn.cache.shared(batch, groups)
    shared.prefix.fill_(303)  # the new tokens lie in it
    attn.forward(q, batch, shared=shared)
    assert attn.device_status()[0] == B.DG_ERR_DEVICE_CHECK
    shared.prefix.fill_(1 << 30)
    attn.forward(q, batch, shared=shared)
    assert attn.device_status()[0] == B.DG_ERR_DEVICE_CHECK
    shared.prefix.fill_(-5)  # as none
    out, lse = attn.forward(q, batch, lse=torch.empty(3, 4, device="cuda"), shared=shared)
    assert attn.device_status()[0] == 0
    compare(data, out, lse)
    table = data[3].clone()
    table[:, 2] = 1 << 20
    bad = pkg.KvBatch(widened(table, data[1]).cuda(), batch.lens, batch.cu)
    attn.forward(q, bad, shared=attn.cache.shared(bad, groups))
    assert attn.device_status()[0] == B.DG_ERR_DEVICE_CHECK


def test_refusals():
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    data = make([(300, [(3, 1)] * 3)], 4, 2, 64, 16, BF, 16)
    attn, q, batch, groups = handles(data)
    shared = attn.cache.shared(batch, groups)
    other = pkg.KvBatch(batch.page_table, batch.lens, batch.cu)
    with pytest.raises(ValueError):
        attn.forward(q, other, shared=shared)
    small = pkg.PagedAttention(attn.cache, 4, shared_tokens=2)
    with pytest.raises(ValueError):
        small.forward(q, batch, shared=shared)
    with pytest.raises(ValueError):
        pkg.PagedAttention(attn.cache, 4).forward(q, batch, shared=shared)
    for a in ((groups, shared.prefix[:2]), (groups.long(), shared.prefix),
              (groups.cpu(), shared.prefix), (groups[:0], shared.prefix)):
        with pytest.raises(ValueError):
            pkg.KvShared(batch, *a)
    lib = B.load_library()
    x = B.dg_heads_t(q.data_ptr(), 256, 64)
    o = torch.empty_like(q)
    y = B.dg_heads_t(o.data_ptr(), 256, 64)
    good = dict(groups=groups.data_ptr(), prefix=shared.prefix.data_ptr(), n_groups=1,
                workspace=attn._pre, workspace_bytes=attn._pre_bytes)

    def go(**kw):
        return lib.dg_attn_forward_shared(attn.handle, 0, x, y, None, batch.c,
                                          B.dg_attn_shared_t(**{**good, **kw}), 3, None)
    assert go(n_groups=-1) == B.DG_ERR_INVALID_ARG and go(groups=None) == B.DG_ERR_INVALID_ARG
    assert go(prefix=None) == B.DG_ERR_INVALID_ARG
    assert go(groups=good["groups"] + 2) == B.DG_ERR_ALIGNMENT
    assert go(n_groups=1 << 20) == B.DG_ERR_UNSUPPORTED
    for kw in (dict(workspace=None), dict(workspace=attn._pre + 16),
               dict(workspace_bytes=good["workspace_bytes"] - 1)):
        assert go(**kw) == B.DG_ERR_WORKSPACE
    assert lib.dg_attn_forward_shared(attn.handle, 0, x, y, None, batch.c, None, 3, None) == \
        B.DG_ERR_INVALID_ARG
    assert go() == B.DG_OK
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
