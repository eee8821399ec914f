"""Paged attention against a 64-bit implementation.

Tolerance, with u the half step of the element type (eps / 2): the weights are
rounded to that type before the product with V (u sum p |v|) and the output
once (u |o|).  A score is an fp32 sum of D products (error up to D 2^-23 sum
|q k| scale, for any order and truncating adds), and an error d of a score
moves p by a factor e^(2 d); sums over n keys add n 2^-23, and the exponential
2^-21.  fp16 weights below 2^-14 are off by up to 2^-25 absolutely (the largest
is at least 1)."""

import math

import pytest
import torch

import attn_ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import moe_expert_ffn_dg_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkg.build()
    pkg.load_library()


def make(n, lens, hq, hkv, d, ps, dtype, seed=0, spare=2, garbage=math.nan):
    """Pools whose unwritten places hold `garbage`, and shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-x // ps) for x in lens]
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=g).tolist()
    k = torch.full((pages, ps, hkv, d), garbage, dtype=dtype)
    v = torch.full((pages, ps, hkv, d), garbage, dtype=dtype)
    table = torch.full((len(lens), max(1, max(held))), -1, dtype=torch.int32)
    for b, x in enumerate(lens):
        for i in range(held[b]):
            pg = order.pop()
            table[b, i] = pg
            m = min(ps, x - i * ps)
            k[pg, :m] = torch.randn(m, hkv, d, generator=g).to(dtype)
            v[pg, :m] = torch.randn(m, hkv, d, generator=g).to(dtype)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    q = torch.randn(cu[-1], hq, d, generator=g).to(dtype)
    return q, k, v, table, lens, cu


def tolerance(ref, dtype, d, n):
    out, lse, mag, tot, smax = ref
    u = torch.finfo(dtype).eps / 2
    ds = d * 2.0 ** -23 * smax + 2.0 ** -22 * (1 + smax)
    rel = 2 * ds + n * 2.0 ** -23 + 2.0 ** -20
    tol = u * (mag + out.abs()) * (1 + rel) + rel * mag
    if dtype == FP:
        tol = tol + 2.0 ** -24 * (tot + 1)
    return tol, ds[..., 0] + n * 2.0 ** -23 + 2.0 ** -21 * (1 + lse.abs())


def check(data, left, right, scale=None, stream=None, heads_first=False):
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu = data
    d, hq, dtype = q.shape[2], q.shape[1], q.dtype
    scale = d ** -0.5 if scale is None else scale
    ref = attn_ref.attention(q, k, v, table, lens, cu, left, right, scale)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    batch = pkg.KvBatch(table.cuda(), torch.tensor(lens, **i32), torch.tensor(cu, **i32))
    attn = pkg.PagedAttention(cache, hq, left=left, right=right, scale=scale)
    qd = q.cuda()
    if heads_first:  # [heads, tokens, dim] in memory, inside a wider buffer
        wide = torch.zeros(hq, q.shape[0], d + 8, dtype=dtype, device="cuda")
        qd = wide[..., :d].transpose(0, 1)
        qd.copy_(q)
        out = torch.full_like(wide, 7.0)[..., :d].transpose(0, 1)
    else:
        out = torch.full_like(qd, 7.0)
    lse = torch.full((q.shape[0], hq), 7.0, device="cuda")
    attn.forward(qd, batch, out=out, lse=lse)
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    tol, ltol = tolerance(ref, dtype, d, max(lens) if lens else 0)
    got = out.double().cpu()
    assert not torch.isnan(got).any()
    err = (got - ref[0]).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    gl = lse.double().cpu()
    none = ref[1] == -math.inf
    assert (gl[none] == -math.inf).all() and (got[none] == 0).all()
    le = (gl - ref[1])[~none].abs()
    assert (le <= ltol[~none]).all(), float((le / ltol[~none]).max())
    return float((err / tol.clamp(min=1e-30)).max())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_single_tokens(d, ps, dtype):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 300, 511]
    check(make([1] * len(lens), lens, 8, 2, d, ps, dtype), -1, 0)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 32, 128])
def test_chunks(d, ps, dtype):
    """Chunks of several tiles, causal, ragged, empty ones among them."""
    check(make([70, 0, 1, 33, 129], [70, 40, 200, 33, 260], 6, 2, d, ps, dtype, 1), -1, 0)


@pytest.mark.parametrize("left,right", [(-1, -1), (0, 0), (5, 0), (130, 0), (64, 3), (-1, 40),
                                        (10, -1), (200, 200)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows(d, left, right):
    check(make([40, 90, 1], [300, 90, 257], 4, 2, d, 32, BF, 2), left, right)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 5), (7, 1), (48, 3), (128, 1), (100, 1)])
@pytest.mark.parametrize("n", [1, 9])
def test_head_groups(hq, hkv, n):
    check(make([n, n], [150, n], hq, hkv, 64, 16, BF, 3), -1, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_that_see_nothing(d):
    """More new tokens than cached ones (positions below zero), an empty
    cache, windows that end before the first key."""
    check(make([20, 3, 200], [5, 0, 100], 4, 2, d, 16, BF, 4), -1, 0)
    check(make([20, 3], [5, 0], 4, 2, d, 16, BF, 4), 2, -1)


@pytest.mark.parametrize("d", [128, 256])
def test_encoder_memory(d):
    """Cross attention: the cache length has nothing to do with the queries'."""
    check(make([150, 2], [37, 600], 4, 4, d, 64, FP, 5), -1, -1)


@pytest.mark.parametrize("garbage", [math.inf, -math.inf, 3e38])
def test_unwritten_places(garbage):
    dtype = BF
    for d in (64, 128, 256):
        check(make([5, 130], [21, 140], 4, 2, d, 64, dtype, 6, garbage=garbage), -1, 0)


def test_growing_scores():
    """Scores that climb along the keys move the running maximum at every
    tile; falling ones never do; huge ones saturate to one key."""
    for sign in (1.0, -1.0):
        q, k, v, table, lens, cu = make([3, 40], [700, 300], 4, 2, 128, 64, BF, 7)
        for b in range(2):
            for j in range(lens[b]):
                pg = int(table[b, j // 64])
                k[pg, j % 64] = (k[pg, j % 64].float() * 0.1 + sign * 0.05 * j / 10).to(BF)
        q = (q.float() * 0.2 + 0.5).to(BF)
        check((q, k, v, table, lens, cu), -1, -1, scale=0.5)
        check((q, k, v, table, lens, cu), -1, 0, scale=4.0)


def test_strided_queries_and_outputs():
    check(make([40, 1], [100, 77], 6, 2, 128, 32, BF, 8), -1, 0, heads_first=True)


def test_many_short_sequences():
    lens = [(7 * i) % 90 for i in range(700)]
    check(make([1] * 700, lens, 2, 1, 64, 16, BF, 9), -1, 0)


def test_long_sequence_is_split_and_joined():
    check(make([2], [9000], 2, 1, 64, 64, BF, 10), -1, 0)
    check(make([1, 130], [5000, 3000], 2, 2, 128, 16, FP, 11), -1, -1)


def test_pages_before_the_window_may_be_gone():
    data = make([4], [600], 4, 2, 128, 32, BF, 12)
    q, k, v, table, lens, cu = data
    gone = table[0, :15].long()  # keys 0 .. 479; the first query sees 596 - 100 on
    ref = attn_ref.attention(q, k, v, table, lens, cu, 100, 0, 128 ** -0.5)
    k[gone], v[gone] = math.nan, math.nan
    table = table.clone()
    table[0, :15] = -1
    import moe_expert_ffn_dg_gb300 as pkg
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    attn = pkg.PagedAttention(cache, 4, left=100, right=0)
    out = attn.forward(q.cuda(), pkg.KvBatch(table.cuda(), torch.tensor(lens, **i32),
                                             torch.tensor(cu, **i32)))
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    tol, _ = tolerance(ref, BF, 128, 600)
    assert ((out.double().cpu() - ref[0]).abs() <= tol).all()


def handles(data, left=-1, right=0, **kw):
    import moe_expert_ffn_dg_gb300 as pkg
    q, k, v, table, lens, cu = data
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = pkg.KvCache(k[None].cuda(), v[None].cuda())
    batch = pkg.KvBatch(table.cuda(), torch.tensor(lens, **i32), torch.tensor(cu, **i32))
    return (pkg.PagedAttention(cache, q.shape[1], left=left, right=right, **kw), q.cuda(), batch)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_replays_and_other_streams(d):
    """A captured call reads lens, cu and the table again at every replay; the
    same inputs give the same bits, on any stream."""
    attn, q, batch = handles(make([90, 1, 140], [700, 300, 140], 4, 2, d, 32, BF, 20))
    out = torch.zeros_like(q)
    attn.forward(q, batch, out=out)
    torch.cuda.synchronize()
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    alone = attn.forward(q, batch, stream=side)
    side.synchronize()
    assert torch.equal(alone, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.forward(q, batch, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # shorter caches, in the same tensors
    batch.lens.copy_(torch.tensor([500, 17, 140], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    again = attn.forward(q, batch)
    assert torch.equal(out, again) and not torch.equal(out, first)
    assert attn.device_status()[0] == 0


def test_rows_outside_every_sequence_are_left_alone():
    attn, q, batch = handles(make([3, 2], [50, 60], 4, 2, 64, 16, BF, 21))
    whole = attn.forward(q, batch)
    batch.cu.copy_(torch.tensor([1, 3, 4], dtype=torch.int32))
    out = torch.full_like(q, 5.0)
    attn.forward(q, batch, out=out)
    torch.cuda.synchronize()
    assert (out[[0, 4]] == 5.0).all() and not (out[1:4] == 5.0).all(-1).any()
    # rows 1, 2 are now the last two tokens of the first sequence, as before
    assert torch.equal(out[1:3], whole[1:3]) and attn.device_status()[0] == 0


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("n", [1, 200])
def test_bad_pages_and_lengths_are_reported(d, n):
    """A page id out of range reads as zeros, a length past the row is the
    row's, a negative one zero; the status word says so once."""
    from moe_expert_ffn_dg_gb300 import binding as B
    attn, q, batch = handles(make([n], [n + 100], 2, 1, d, 16, BF, 22))
    good = attn.forward(q, batch).clone()
    for bad in (-1, 10 ** 9):
        keep = batch.page_table[0, 2].clone()
        batch.page_table[0, 2] = bad
        out = attn.forward(q, batch)
        assert attn.device_status()[:2] == (B.DG_ERR_DEVICE_CHECK, 36)
        assert torch.isfinite(out).all()
        batch.page_table[0, 2] = keep
    for bad in (10 ** 9, -5):
        keep = batch.lens.clone()
        batch.lens.fill_(bad)
        # the row's last page may hold anything past the true length
        attn.forward(q, batch)
        assert attn.device_status()[:2] == (B.DG_ERR_DEVICE_CHECK, 37)
        batch.lens.copy_(keep)
    batch.cu.copy_(torch.tensor([0, n + 7], dtype=torch.int32))
    attn.forward(q, batch)
    assert attn.device_status()[:2] == (B.DG_ERR_DEVICE_CHECK, 37)
    batch.cu.copy_(torch.tensor([0, n], dtype=torch.int32))
    assert torch.equal(attn.forward(q, batch), good) and attn.device_status()[0] == 0


def test_layers_of_one_cache():
    import moe_expert_ffn_dg_gb300 as pkg
    data = make([5], [90], 2, 1, 128, 16, FP, 23)
    q, k, v, table, lens, cu = data
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = pkg.KvBatch(table.cuda(), torch.tensor(lens, **i32), torch.tensor(cu, **i32))
    zero = torch.zeros_like(k)
    cache = pkg.KvCache(torch.stack([zero, k]).cuda(), torch.stack([zero, v]).cuda())
    attn = pkg.PagedAttention(cache, 2)
    ref = attn_ref.attention(*data, -1, 0, 128 ** -0.5)
    tol, _ = tolerance(ref, FP, 128, 90)
    assert ((attn.forward(q.cuda(), batch, layer=1).double().cpu() - ref[0]).abs() <= tol).all()
    assert (attn.forward(q.cuda(), batch, layer=0) == 0).all()


def test_empty_calls():
    attn, q, batch = handles(make([0, 0], [30, 0], 2, 1, 64, 16, BF, 24))
    assert attn.forward(q, batch).shape == (0, 2, 64) and attn.device_status()[0] == 0


def test_refusals():
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    attn, q, batch = handles(make([4], [20], 4, 2, 64, 16, BF, 25))
    cache = attn.cache
    for kw, code in ((dict(n_q_heads=3), 1), (dict(n_q_heads=0), 1), (dict(n_q_heads=258), 3),
                     (dict(n_q_heads=4, scale=0.0), 1), (dict(n_q_heads=4, scale=math.nan), 1),
                     (dict(n_q_heads=4, scale=math.inf), 1), (dict(n_q_heads=4, scale=-1.0), 1)):
        with pytest.raises(B.DgError) as e:
            pkg.PagedAttention(cache, **kw)
        assert e.value.status == code
    wide = torch.zeros(4, 4, 72, dtype=BF, device="cuda")
    for bad in (lambda: attn.forward(q[:, :2], batch), lambda: attn.forward(q.half(), batch),
                lambda: attn.forward(q.cpu(), batch), lambda: attn.forward(q[..., :32], batch),
                lambda: attn.forward(q, batch, lse=torch.zeros(4, 4, device="cuda").half()),
                lambda: attn.forward(q, batch, lse=torch.zeros(4, 3, device="cuda")),
                lambda: pkg.KvBatch(batch.page_table.long(), batch.lens, batch.cu),
                lambda: pkg.KvBatch(batch.page_table, batch.lens, batch.cu[:1]),
                lambda: pkg.KvCache(cache.k_pages[0], cache.v_pages[0]),
                lambda: pkg.KvCache(cache.k_pages, cache.v_pages.half())):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: attn.forward(q, batch, layer=1), B.DG_ERR_INVALID_ARG),
                      (lambda: attn.forward(q, batch, out=q), B.DG_ERR_INVALID_ARG),
                      (lambda: attn.forward(wide[..., 1:65], batch), B.DG_ERR_ALIGNMENT),
                      (lambda: attn.forward(q[:, :1].expand(4, 4, 64), batch),
                       B.DG_ERR_UNSUPPORTED),
                      (lambda: pkg.KvCache(cache.k_pages.float(), cache.v_pages.float()),
                       B.DG_ERR_UNSUPPORTED)):
        with pytest.raises(B.DgError) as e:
            bad()
        assert e.value.status == code
    with pytest.raises(B.DgError) as e:  # a workspace too small or misaligned
        B.dg_attn_create(attn.cfg, cache.handle, attn.workspace.data_ptr() // 1024 * 1024, 1 << 20)
    assert e.value.status == B.DG_ERR_WORKSPACE
    with pytest.raises(B.DgError) as e:
        B.dg_attn_create(attn.cfg, cache.handle, 1024 * 1024 + 16, 1 << 30)
    assert e.value.status == B.DG_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_short_items_with_ragged_ends(d):
    """A CTA goes through many items of one or two key tiles each, every one of
    which ends inside a 16-key step (their cleared values follow one another
    closely)."""
    check(make([150, 141, 160], [152, 150, 163], 32, 2, d, 64, BF, 30), 90, 1)
    check(make([97, 150], [97, 331], 24, 3, d, 256, FP, 31), 30, 0)
