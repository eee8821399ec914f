"""Attention weights of cached tokens against a 64-bit implementation.

Tolerance of a weight exp(s - t): a score s is an fp32 sum of D products (error up
to D 2^-23 sum |q k| scale, for any order and truncating adds); scale log2 e, the
product with it and the difference from t are rounded once each, in units of at
most (|s| + |t|) 2^-22 together, and the exponential by 2^-21.  So a weight is off by
a factor of at most e^d, d = D 2^-23 smax + 2^-21 (1 + smax + |t|).  Sums: 32 terms in
a row within a tile, pairs and a carried error beyond it, a store of partial
sums: 40 half steps; the decayed old weight and the last addition: 2^-22 of their
sizes."""

import math

import pytest
import torch

import attn_ref
from test_gpu_attn import BF, FP, _built, make  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def reference(q, k_pages, lse, w, table, lens, cu, left, right, scale, decay, fresh):
    """Weights and their tolerance, token by token."""
    G = q.shape[1] // k_pages.shape[2]
    out, tol = w.double().clone(), torch.zeros(w.shape, dtype=torch.float64)
    for b, kv in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if kv == 0:
            continue
        old = w[b, :kv].double().clone()
        if fresh:
            old[max(kv - n, 0):] = 0
        if decay == 0:
            old[:] = 0
        add = torch.zeros(kv, dtype=torch.float64)
        slack = torch.zeros(kv, dtype=torch.float64)
        k = attn_ref.cached(k_pages, table[b], kv)
        for i in range(n):
            p = kv - n + i
            lo = 0 if left < 0 else max(0, p - left)
            hi = kv if right < 0 else min(kv, p + right + 1)
            if hi <= lo:
                continue
            for h in range(q.shape[1]):
                qq, kk, t = q[cu[b] + i, h].double(), k[lo:hi, h // G], lse[cu[b] + i, h].double()
                x = torch.exp((kk @ qq) * scale - t)
                smax = (kk.abs() @ qq.abs()) * scale
                d = q.shape[2] * 2.0 ** -23 * smax + 2.0 ** -21 * (1 + smax + t.abs())
                add[lo:hi] += x
                slack[lo:hi] += x * torch.expm1(d)
        out[b, :kv] = decay * old + add
        tol[b, :kv] = slack + 40 * 2.0 ** -24 * add + 2.0 ** -22 * (add + decay * old.abs())
    return out, tol


def run(data, left=-1, right=0, decay=0.75, fresh=True, inplace=False, extra=3, lse=None):
    """Compare a call with the definition; returns the handle and its arguments."""
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu = data
    d, hq = q.shape[2], q.shape[1]
    scale = d ** -0.5
    g = torch.Generator().manual_seed(99)
    width = max(lens + [1]) + extra
    w = torch.rand(len(lens), width, generator=g)
    for b, kv in enumerate(lens):  # what a call must not read
        n = cu[b + 1] - cu[b]
        w[b, kv:] = math.nan
        if fresh:
            w[b, max(kv - n, 0):kv] = math.nan
    if lse is None:
        lse = attn_ref.attention(q, k, v, table, lens, cu, left, right, scale)[1].float()
    want, tol = reference(q, k, lse, w, table, lens, cu, left, right, scale, decay, fresh)
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    batch = pkg.KvBatch(table.cuda(), i32(lens), i32(cu))
    attn = pkg.PagedAttention(cache, hq, left=left, right=right)
    dev = w.cuda()
    out = dev if inplace else torch.full_like(dev, 7.0)
    qd, ld = q.cuda(), lse.cuda()
    got = attn.weights(qd, ld, batch, dev, decay=decay, fresh=fresh, out=None if inplace else out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr() and attn.device_status()[0] == 0
    res = got.double().cpu()
    for b, kv in enumerate(lens):
        err = (res[b, :kv] - want[b, :kv]).abs()
        assert not torch.isnan(err).any(), b
        assert (err <= tol[b, :kv]).all(), (b, float((err / tol[b, :kv].clamp(min=1e-300)).max()))
        tail = res[b, kv:]
        assert torch.isnan(tail).all() if inplace else (tail == 7).all()
    return attn, qd, ld, batch, dev, got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_single_tokens(d, ps, dtype):
    lens = [1, 2, 15, 127, 128, 129, 255, 256, 257, 300, 515]
    run(make([1] * len(lens), lens, 8, 2, d, ps, dtype))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 32, 128])
def test_chunks(d, ps, dtype):
    run(make([70, 0, 1, 33, 129], [70, 40, 200, 33, 260], 6, 2, d, ps, dtype, 1))


@pytest.mark.parametrize("left,right", [(-1, -1), (0, 0), (5, 0), (130, 0), (64, 3), (-1, 40),
                                        (10, -1), (200, 200)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows(d, left, right):
    run(make([40, 90, 1], [600, 90, 257], 4, 2, d, 32, BF, 2), left, right)


@pytest.mark.parametrize("group", [1, 3, 5, 7, 16, 17, 128])
def test_groups(group):
    run(make([9, 1], [40, 300], 2 * group, 2, 64, 16, BF, 3))
    run(make([1, 1, 1], [40, 300, 7], 2 * group, 2, 64, 16, FP, 4))


@pytest.mark.parametrize("decay,fresh", [(0.0, True), (1.0, True), (1.0, False), (0.5, False),
                                         (3.0, False)])
def test_decay_and_new_tokens(decay, fresh):
    data = make([5, 1, 0], [300, 20, 270], 4, 2, 128, 32, BF, 5)
    run(data, decay=decay, fresh=fresh)
    run(data, decay=decay, fresh=fresh, inplace=True)


def test_more_queries_than_keys():
    """Rows with negative positions, of an encoder memory or without a key."""
    run(make([40, 9], [7, 3], 4, 2, 64, 16, BF, 6), -1, -1)
    run(make([40, 9], [7, 3], 4, 2, 64, 16, BF, 6), -1, 0)


def test_no_tokens_and_no_keys():
    run(make([0, 0], [300, 10], 4, 2, 64, 16, BF, 7))
    run(make([0, 2, 0], [0, 2, 0], 4, 2, 64, 16, BF, 8))


def test_layers_of_a_step_add_up():
    """The first layer decays, the others add to what it wrote."""
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu = make([3, 1], [80, 300], 4, 2, 64, 16, BF, 9, garbage=0.0)
    pools = [torch.stack([x, x.flip(1)]).cuda() for x in (k, v)]
    cache = pkg.KvCache(*pools)
    batch = pkg.KvBatch(table.cuda(), i32(lens), i32(cu))
    attn = pkg.PagedAttention(cache, 4)
    w = torch.zeros(2, 400, device="cuda")
    want = torch.zeros(2, 400, dtype=torch.float64)
    bound = torch.zeros(2, 400, dtype=torch.float64)
    for layer in range(2):
        lse = torch.empty(4, 4, device="cuda")
        attn.forward(q.cuda(), batch, layer=layer, lse=lse)
        attn.weights(q.cuda(), lse, batch, w, layer=layer, fresh=layer == 0)
        one, tol = reference(q, pools[0][layer].cpu(), lse.cpu(), torch.zeros(2, 400), table, lens,
                             cu, -1, 0, 0.125, 1.0, True)
        want, bound = want + one, bound + tol
    err = (w.double().cpu() - want).abs()
    assert (err <= bound + 2.0 ** -23 * want).all()
    # every row of every head spreads a weight of one
    total = w.double().sum(1).cpu()
    assert torch.allclose(total, torch.tensor([3 * 4 * 2.0, 4 * 2.0], dtype=torch.float64),
                          rtol=1e-3)


def test_masked_places_may_hold_anything():
    """Keys that no token sees (NaN among them) and their rows' log-sums."""
    q, k, v, table, lens, cu = make([6, 2], [520, 300], 4, 2, 64, 16, BF, 10)
    want = attn_ref.attention(q, k, v, table, lens, cu, 40, 0, 0.125)[1].float()
    for b, first in ((0, 520 - 6 - 40), (1, 300 - 2 - 40)):
        for j in range(first):  # behind every window: page content, table entries of whole pages
            k[int(table[b, j // 16]), j % 16] = math.nan if j % 2 else math.inf
        table[b, :first // 16] = -7
    run((q, k, v, table, lens, cu), 40, 0, lse=want)


def test_long_sums_and_offsets():
    """Many tokens over few keys, and a cache whose pages lie far apart."""
    run(make([700], [700], 8, 1, 64, 64, BF, 11), -1, -1)


@pytest.mark.parametrize("left,right", [(1 << 27, 0), (0, 1 << 27), (1 << 27, 1 << 27)])
def test_limits_past_every_token(left, right):
    """Limits that a table of 2^27 places leaves standing, with 32 heads on one:
    rows times heads pass 32 bits before the tile bounds them."""
    q, k, v, table, lens, cu = make([3, 1], [300, 40], 64, 2, 64, 256, BF, 17)
    wide = torch.full((2, (1 << 19) + 8), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    run((q, k, v, wide, lens, cu), left, right)


def test_same_result_every_time():
    a = [run(make([70, 1], [3000, 900], 6, 2, 128, 64, BF, 12))[-1].clone() for _ in range(2)]
    assert torch.equal(a[0].nan_to_num(5), a[1].nan_to_num(5))


def test_strided_rows_and_views():
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu = make([3, 1], [80, 300], 4, 2, 64, 16, BF, 13)
    lse = attn_ref.attention(q, k, v, table, lens, cu, -1, 0, 0.125)[1].float()
    w = torch.rand(2, 310)
    want, tol = reference(q, k, lse, w, table, lens, cu, -1, 0, 0.125, 1.0, True)
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    attn = pkg.PagedAttention(cache, 4)
    batch = pkg.KvBatch(table.cuda(), i32(lens), i32(cu))
    wide = torch.zeros(4, 4, 72, dtype=BF, device="cuda")  # [heads, tokens, dim + 8]
    wide[..., :64] = q.transpose(0, 1).cuda()
    big = torch.full((2, 601), 5.0, device="cuda")
    src = torch.zeros(2, 333, device="cuda")
    src[:, 7:317] = w.cuda()
    attn.weights(wide[..., :64].transpose(0, 1), lse.cuda(), batch, src[:, 7:317],
                 out=big[:, 11:321])
    got = big.double().cpu()
    assert attn.device_status()[0] == 0
    for b, kv in enumerate(lens):
        assert ((got[b, 11:11 + kv] - want[b, :kv]).abs() <= tol[b, :kv]).all()
        assert (got[b, :11] == 5).all() and (got[b, 11 + kv:] == 5).all()


def test_captured_and_replayed():
    import moe_expert_ffn_dg_gb300 as pkg
    attn, q, lse, batch, w, out = run(make([70, 1], [3000, 900], 6, 2, 128, 64, BF, 14), decay=0.5)
    want, other = out.clone(), torch.full_like(out, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.weights(q, lse, batch, w, decay=0.5, out=other)
    for _ in range(3):
        other.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(other, want)
    side = torch.cuda.Stream()
    other.fill_(7.0)
    torch.cuda.synchronize()
    attn.weights(q, lse, batch, w, decay=0.5, out=other, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    assert isinstance(attn, pkg.PagedAttention)


def test_bad_pages_and_lengths_are_reported():
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    q, k, v, table, lens, cu = make([1, 1], [80, 300], 4, 2, 64, 16, BF, 15)
    lse = attn_ref.attention(q, k, v, table, lens, cu, -1, 0, 0.125)[1].float().cuda()
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    attn = pkg.PagedAttention(cache, 4)
    w = torch.zeros(2, 310, device="cuda")
    good = attn.weights(q.cuda(), lse, pkg.KvBatch(table.cuda(), i32(lens), i32(cu)), w.clone())
    assert attn.device_status()[0] == 0
    for page in (-1, 1 << 30):
        t = table.clone()
        t[1, 3] = page
        got = attn.weights(q.cuda(), lse, pkg.KvBatch(t.cuda(), i32(lens), i32(cu)), w.clone())
        assert attn.device_status()[0] == B.DG_ERR_DEVICE_CHECK
        assert torch.equal(got[0], good[0]) and torch.equal(got[1, 64:], good[1, 64:])
    # longer than its pages, longer than the weights' rows, negative
    for bad, width in (([80, 100000], 310), ([80, 300], 200), ([-5, 300], 310)):
        attn.weights(q.cuda(), lse, pkg.KvBatch(table.cuda(), i32(bad), i32(cu)),
                     torch.zeros(2, width, device="cuda"))
        assert attn.device_status()[0] == B.DG_ERR_DEVICE_CHECK


def test_refusals():
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu = make([1, 1], [80, 300], 4, 2, 64, 16, BF, 16)
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    attn = pkg.PagedAttention(cache, 4)
    batch = pkg.KvBatch(table.cuda(), i32(lens), i32(cu))
    q, lse, w = q.cuda(), torch.zeros(2, 4, device="cuda"), torch.zeros(2, 310, device="cuda")
    for a in ((q[:, :2], lse, w), (q, lse[:1], w), (q, lse.double(), w), (q, lse, w[:1]),
              (q, lse, w.half()), (q, lse, w.cpu()), (q, lse, w.t().contiguous().t()),
              (q.half(), lse, w)):
        with pytest.raises(ValueError):
            attn.weights(*a[:2], batch, a[2])
    with pytest.raises(ValueError):
        attn.weights(q, lse, batch, w, out=w[:, :300])
    for kw in (dict(decay=-0.5), dict(decay=math.nan), dict(decay=math.inf), dict(layer=1)):
        with pytest.raises(pkg.DgError):
            attn.weights(q, lse, batch, w, **kw)
