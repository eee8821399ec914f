"""Paged attention at values where it can go wrong: non-finite ones at places
that are seen, in items that one CTA holds whole and in items that several
share, and weights far below the largest one."""

import math

import pytest
import torch

from test_gpu_attn import BF, FP, _built, handles, make  # noqa: F401

pytestmark = pytest.mark.gpu


def run(data, left=-1, right=-1):
    attn, q, batch = handles(data, left, right)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out, lse = attn.forward(q, batch, lse=lse)
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    return out.cpu(), lse.cpu()


# one key tile (an item cannot be split) and two dozen (one tile a CTA)
@pytest.mark.parametrize("kv", [100, 3000])
@pytest.mark.parametrize("d,dtype", [(64, FP), (128, BF), (256, BF)])
@pytest.mark.parametrize("n", [1, 60])
def test_a_query_of_nan(n, d, dtype, kv):
    data = make([n], [kv], 8, 1, d, 64, dtype, 40)
    good = run(data)
    data[0][n - 1, 3, 5] = math.nan
    out, lse = run(data)
    assert out[n - 1, 3].isnan().all() and lse[n - 1, 3].isnan()
    rest = torch.ones(n, 8, dtype=torch.bool)
    rest[n - 1, 3] = False
    assert torch.equal(out[rest], good[0][rest]) and torch.equal(lse[rest], good[1][rest])


@pytest.mark.parametrize("first,count", [(0, 100), (1024, 128), (1000, 300), (2999, 1)])
@pytest.mark.parametrize("d,n", [(64, 1), (128, 1), (256, 1), (64, 60), (128, 60), (256, 60)])
def test_keys_of_nan(d, n, first, count):
    """A run of keys that fills a part, more than one, or less.  Queries whose
    window ends before or begins after it are not touched."""
    data = make([n], [3000], 4, 1, d, 64, BF, 41)
    q, k, v, table, lens, cu = data
    for left in (-1, 50):
        good = run(data, left, 0)
        bad = k.clone()
        for j in range(first, first + count):
            bad[int(table[0, j // 64]), j % 64, 0, 7] = math.nan
        out, lse = run((q, bad, v, table, lens, cu), left, 0)
        for i in range(n):
            p = 3000 - n + i
            sees = first <= p and (left < 0 or first + count > p - left)
            if sees:
                assert out[i].isnan().all() and lse[i].isnan().all(), i
            else:
                assert torch.equal(out[i], good[0][i]) and torch.equal(lse[i], good[1][i]), i


@pytest.mark.parametrize("kv", [100, 3000])
@pytest.mark.parametrize("n", [1, 60])
def test_infinite_scores_and_values(n, kv):
    """A score of +inf makes 0 / 0 of its row's weights; an infinite value
    reaches its column, with its sign, and nothing else."""
    data = make([n], [kv], 4, 1, 128, 64, BF, 42)
    q, k, v, table, lens, cu = data
    good = run(data)
    page, row = int(table[0, 77 // 64]), 77 % 64
    bad = v.clone()
    bad[page, row, 0, 9] = -math.inf
    out, lse = run((q, k, bad, table, lens, cu))
    assert (out[..., 9] == -math.inf).all() and torch.equal(lse, good[1])
    cols = [c for c in range(128) if c != 9]
    assert torch.equal(out[..., cols], good[0][..., cols])
    bad = k.clone()
    bad[page, row, 0] = math.inf * torch.sign(q[0, 2].float()).to(BF)
    out, lse = run((q, bad, v, table, lens, cu))
    assert out[0, 2].isnan().all() and not (lse[0, 2] == -math.inf)


@pytest.mark.parametrize("d,n", [(64, 1), (128, 1), (256, 1), (64, 150), (128, 150), (256, 40)])
def test_one_large_weight_before_a_long_tail(d, n):
    """fp16: the first key's weight is 2^26 times each other one's, and 131072 of
    those make up 2^-9 of the sum.  (Many sequences share the pages, so that a
    CTA runs through most of an item by itself.)

    Tolerance: a weight in fp16 is off by up to 2^-25 absolutely where it is
    small, which is 2^-32 of the largest weight (it lies at 2^7 or above): 2^-32
    a key, and half a step of the output (2^-11, relative).  The sums of 131072
    fp32 terms add 2^-23 a term relative to them (2^-6 of the tail), and scores
    up to 18 are off by 2^-24 of themselves a rounding: 2^-18 in all."""
    import moe_expert_ffn_dg_gb300 as pkg
    keys, seqs, ps = 131072, 160, 256
    pages = keys // ps
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(1, pages, ps, 1, d, dtype=FP, device="cuda")
    v = torch.ones(1, pages, ps, 1, d, dtype=FP, device="cuda")
    v[0, 0, 0] = 0
    scale = d ** -0.5
    # q k scale log2 e = 26 for the first key, 0 for the others
    q = torch.zeros(seqs * n, 2, d, dtype=FP, device="cuda")
    q[..., 1] = 4.0
    k[0, 0, 0, 0, 1] = 26 * math.log(2) / scale / 4
    cache = pkg.KvCache(k, v)
    table = torch.arange(pages, **i32).expand(seqs, pages).contiguous()
    batch = pkg.KvBatch(table, torch.full((seqs,), keys, **i32),
                        torch.arange(seqs + 1, **i32) * n)
    attn = pkg.PagedAttention(cache, 2, right=-1)
    lse = torch.zeros(seqs * n, 2, device="cuda")
    out, lse = attn.forward(q, batch, lse=lse)
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    top = 4.0 * float(k[0, 0, 0, 0, 1]) * scale
    tail = (keys - 1) * math.exp(-top)
    want = tail / (1 + tail)
    tol = 2.0 ** -11 * want + keys * 2.0 ** -32 + want * (2.0 ** -6 + 2.0 ** -18)
    err = (out.double() - want).abs().max()
    assert err <= tol, (float(err), tol, want)
    assert (lse.double() - (top + math.log1p(tail))).abs().max() <= 2.0 ** -18 * (1 + top)


@pytest.mark.parametrize("n", [1, 90])
def test_tables_with_a_row_stride(n):
    """Rows of a wider table, and of one whose first columns are another's: an
    append and an attention as with a table of their own."""
    import moe_expert_ffn_dg_gb300 as pkg
    data = make([n, 0, n], [400, 30, 290], 4, 2, 128, 32, BF, 43)
    attn, q, batch = handles(data)
    want = attn.forward(q, batch)
    table = batch.page_table
    wide = torch.full((3, 2 * table.shape[1] + 5), 10 ** 9, dtype=torch.int32, device="cuda")
    part = wide[:, 3:3 + table.shape[1]]
    part.copy_(table)
    other = pkg.KvBatch(part, batch.lens, batch.cu)
    assert part.stride(0) != part.shape[1]
    assert torch.equal(attn.forward(q, other), want)
    cache = attn.cache
    kv = torch.randn(2 * n, 4, 128, device="cuda").to(BF)
    got = []
    for b in (batch, other):
        cache.k_pages.zero_(), cache.v_pages.zero_()
        cache.append(kv[:, :2], kv[:, 2:], b, rope=pkg.Rope(128))
        got.append((cache.k_pages.clone(), cache.v_pages.clone()))
    assert got[0][0].any() and torch.equal(got[0][0], got[1][0])
    assert torch.equal(got[0][1], got[1][1])
    assert cache.device_status()[0] == 0 and attn.device_status()[0] == 0
