"""What forks share, and the choice of the tokens that stay, against plain
definitions.  Everything is whole numbers or copies: results are equal."""

import math
import random

import numpy as np
import pytest
import torch

from test_gpu_attn import BF, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


def a_cache(page=16, pages=4):
    import moe_expert_ffn_dg_gb300 as pkg
    return pkg.KvCache(*(torch.zeros(1, pages, page, 1, 64, dtype=BF, device="cuda")
                         for _ in range(2)))


# ------------------------------------------------------------------ select

def chosen(w, lens, budget, first, last):
    """keep, cu, weights by the definition, a token at a time."""
    budget = min(budget, w.shape[1])
    keep, cu = [], [0]
    for row, n in zip(w, lens):
        if n <= budget:
            some = list(range(n))
        else:
            some = list(range(first)) + list(range(n - last, n))
            mid = list(range(first, n - last))
            # NaN first, then by size (equal ones, 0 and -0 among them, by place)
            mid.sort(key=lambda j: (not math.isnan(row[j]), -row[j] if row[j] == row[j] else 0, j))
            some += mid[:budget - first - last]
        keep += sorted(some)
        cu.append(len(keep))
    return keep, cu


def check_select(w, lens, budget, first=0, last=0, cache=None, out=None):
    cache = cache or a_cache()
    w = np.asarray(w, np.float32)
    keep, cu = chosen(w, lens, budget, first, last)
    got = cache.select(torch.from_numpy(w).cuda(), i32(lens), budget, first=first, last=last, out=out)
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    most = min(budget, w.shape[1])
    assert got.cu.tolist() == cu and got.lens.tolist() == np.diff(cu).tolist()
    assert got.keep.shape == (len(lens) * most,)
    assert got.keep.tolist() == keep + [-1] * (len(lens) * most - len(keep))
    kept = got.weights.cpu().numpy()[:, :most]
    for b in range(len(lens)):
        some = keep[cu[b]:cu[b + 1]]
        want = np.zeros(most, np.float32)
        want[:len(some)] = w[b, some]
        assert np.array_equal(kept[b].view(np.uint32), want.view(np.uint32))
    return got


@pytest.mark.parametrize("width", [1, 7, 1000, 4096, 4097, 9000, 40000])
@pytest.mark.parametrize("seqs", [1, 5])
def test_select_sizes(seqs, width):
    rng = np.random.default_rng(width * 10 + seqs)
    lens = [width] + [int(x) for x in rng.integers(0, width + 1, seqs - 1)]
    w = rng.standard_normal((seqs, width)) ** 3
    for budget in sorted({0, 1, width // 3, width - 1, width, width + 9}):
        first = min(budget, 3)
        check_select(w, lens, budget, first, min(5, budget - first))
        check_select(w, lens, budget)


def test_select_many_short_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 65, 3000).tolist()
    check_select(rng.random((3000, 64)), lens, 20, 2, 3)


def test_select_rows_past_shared_memory():
    """A slice that is longer than what a CTA keeps of it."""
    rng = np.random.default_rng(4)
    w = np.exp(2 * rng.standard_normal((2, 300000)))
    check_select(w, [300000, 123457], 60000, 10, 1000)


@pytest.mark.parametrize("width", [20481, 45100, 61441, 90000, 110001, 131072, 170000, 400000])
def test_select_rows_of_several_blocks(width):
    """Two to eight blocks a row; in the last case none holds its slice."""
    rng = np.random.default_rng(width)
    w = np.exp(2 * rng.standard_normal((3, width)))
    w[1] = rng.integers(0, 50, width)  # equal ones on both sides of every border
    w[2, ::7] = math.nan
    lens = [width, width - 5, width // 3]
    check_select(w, lens, width // 9, 10, 100)
    check_select(w, lens, width // 2)


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "last digit", "nan", "inf", "negative"])
@pytest.mark.parametrize("width", [900, 20000])
def test_select_ties_and_special_values(kind, width):
    rng = np.random.default_rng(5)
    w = rng.standard_normal((2, width)).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":  # 0 and -0 are the same
        w = np.where(rng.random(w.shape) < 0.9, np.where(rng.random(w.shape) < 0.5, 0.0, -0.0), w)
    elif kind == "few":
        w = rng.choice(np.float32([1, 2, 3]), w.shape)
    elif kind == "last digit":  # bits of the last histogram alone
        w = (np.float32(1).view(np.uint32) + rng.integers(0, 700, w.shape, dtype=np.uint32)
             ).view(np.float32)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.1] = math.nan
        w.view(np.uint32)[0, ::17] |= 0xffc00000  # with the sign and other payloads
    elif kind == "inf":
        w[rng.random(w.shape) < 0.1] = math.inf
        w[rng.random(w.shape) < 0.6] = -math.inf
    else:
        w = -np.abs(w)
    for budget in (1, width // 10, width // 2, width - 1):
        check_select(w, [width, width - 3], budget)
        check_select(w, [width, width - 3], budget, min(2, budget), 0)


def test_select_leaves_what_it_must():
    """Rows of wider buffers, strided inputs, and NaN behind the sequences."""
    import moe_expert_ffn_dg_gb300 as pkg
    rng = np.random.default_rng(6)
    cache = a_cache()
    wide = torch.full((3, 700), 9.0, device="cuda")
    keep, cu, lens = i32([5] * 300), i32([5] * 4), i32([5] * 3)
    out = pkg.KvKeep(keep, cu, lens, wide[:, 50:250])
    w = torch.from_numpy(rng.random((3, 600), dtype=np.float32)).cuda()
    n = [600, 70, 0]
    for b in range(3):
        w[b, n[b]:] = math.nan
    got = cache.select(w[:, :550], i32([550, 70, 0]), 100, first=1, last=1, out=out)
    ref, ref_cu = chosen(w[:, :550].cpu().numpy(), [550, 70, 0], 100, 1, 1)
    assert got is out and keep.tolist() == ref + [-1] * (300 - len(ref)) and cu.tolist() == ref_cu
    assert (wide[:, :50] == 9).all() and (wide[:, 150:] == 9).all()
    assert (wide[1, 120:150] == 0).all() and (wide[2, 50:150] == 0).all()


def test_select_lens_out_of_range_are_reported():
    from moe_expert_ffn_dg_gb300 import binding as B
    cache = a_cache()
    w = torch.rand(2, 50, device="cuda")
    for bad, taken in (([51, 10], [50, 10]), ([20, -1], [20, 0])):
        got = cache.select(w, i32(bad), 30)
        assert cache.device_status()[0] == B.DG_ERR_DEVICE_CHECK
        want = cache.select(w, i32(taken), 30)
        assert cache.device_status()[0] == 0
        assert torch.equal(got.keep, want.keep) and torch.equal(got.cu, want.cu)


def test_select_captured_and_on_a_side_stream():
    cache = a_cache()
    w = torch.rand(9, 5000, device="cuda")
    lens = i32([5000, 0, 1, 3000, 4999, 700, 5000, 5000, 5000])
    want = cache.select(w, lens, 600, first=2, last=7)
    got = cache.select(w, lens, 600, first=2, last=7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.select(w, lens, 600, first=2, last=7, out=got)
    side = torch.cuda.Stream()
    for how in (graph.replay, lambda: cache.select(w, lens, 600, first=2, last=7, out=got,
                                                   stream=side)):
        for name in got.__slots__:
            getattr(got, name).fill_(3)
        torch.cuda.synchronize()
        how()
        torch.cuda.synchronize()
        for name in got.__slots__:
            assert torch.equal(getattr(got, name), getattr(want, name)), name


def test_select_budgets_past_32_bits_keep_all():
    w = np.arange(20, dtype=np.float32).reshape(2, 10)
    for budget, first, last in [(2**31, 0, 0), (2**32 + 3, 1, 1), (2**40, 2**33, 2**39),
                                (2**63, 0, 2**32 + 1), (11, 6, 5)]:
        check_select(w, [10, 4], budget, first, last)


def test_select_of_no_sequences_on_a_side_stream():
    cache, side = a_cache(), torch.cuda.Stream()
    out = cache.select(torch.zeros(0, 8, device="cuda"), i32([]), 4, stream=side)
    side.synchronize()
    assert out.cu.tolist() == [0] and out.keep.numel() == out.lens.numel() == 0


def test_select_refusals():
    import moe_expert_ffn_dg_gb300 as pkg
    cache = a_cache()
    w, lens = torch.rand(2, 50, device="cuda"), i32([50, 20])
    for a in ((w[:1], lens, 5), (w.half(), lens, 5), (w.cpu(), lens, 5), (w.t(), lens, 5),
              (w, lens.long(), 5), (w, lens, -1)):
        with pytest.raises(ValueError):
            cache.select(*a)
    for kw in (dict(first=3, last=3), dict(first=-1), dict(last=-1)):
        with pytest.raises(ValueError):
            cache.select(w, lens, 5, **kw)
    with pytest.raises(ValueError):
        cache.select(w, lens, 5, out=pkg.KvKeep(i32([0] * 10), i32([0] * 3), i32([0] * 2), w[:, :4]))
    with pytest.raises(pkg.DgError):  # in place
        cache.select(w, lens, 5, out=pkg.KvKeep(i32([0] * 10), i32([0] * 3), i32([0] * 2), w))
    empty = cache.select(w[:0], lens[:0], 5)
    assert empty.keep.numel() == 0 and empty.cu.tolist() == [0]


# ------------------------------------------------------------------ shared

def common(table, lens, cu, groups, page):
    out = [0] * len(lens)
    for a, b in zip(groups[:-1], groups[1:]):
        if b - a < 2:
            continue
        pages = 0
        while pages < table.shape[1] and len(set(table[a:b, pages].tolist())) == 1:
            pages += 1
        n = min([pages * page] + [lens[s] - (cu[s + 1] - cu[s]) for s in range(a, b)])
        out[a:b] = [n] * (b - a)
    return out


def check_shared(table, lens, n, groups, page, cache=None, strided=False):
    import moe_expert_ffn_dg_gb300 as pkg
    cache = cache or a_cache(page)
    cu = np.concatenate([[0], np.cumsum(n)])
    table = np.asarray(table, np.int32)
    t = i32(table)
    if strided:
        wide = torch.full((table.shape[0], table.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
        wide[:, 2:-3] = t
        t = wide[:, 2:-3]
    got = cache.shared(pkg.KvBatch(t, i32(lens), i32(cu)), i32(groups))
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    want = common(table, lens, cu, groups, page)
    assert got.prefix.tolist() == want
    return want


def forks(rng, groups, size, pages, page, tail):
    """Tables of sequences that begin alike."""
    rows, lens, n, bounds = [], [], [], [0]
    width = pages + tail // page + 2
    for _ in range(groups):
        k = rng.randint(0, pages)
        top = [rng.randint(0, 9) for _ in range(k)]
        for _ in range(rng.randint(0, size)):
            row = list(top)
            if row and rng.random() < 0.2:
                row[rng.randrange(k)] = 77  # ends the common part here
            x = rng.randint(0, tail) + (k * page if rng.random() < 0.8 else rng.randint(0, k * page))
            row += [rng.randint(0, 3) for _ in range(width - k)]
            rows.append(row[:width])
            lens.append(x)
            n.append(rng.randint(0, min(x, 5)))
        bounds.append(len(rows))
    return rows, lens, n, bounds


@pytest.mark.parametrize("page", [16, 64, 256])
def test_shared_of_forks(page):
    some = 0
    for seed in range(30):
        rng = random.Random(seed * 1000 + page)
        rows, lens, n, bounds = forks(rng, rng.randint(1, 7), rng.choice([1, 3, 40]),
                                      rng.choice([2, 40, 300]), page, rng.choice([0, 3, 500]))
        if rows:
            some += sum(check_shared(rows, lens, n, bounds, page, strided=seed % 2 == 1)) > 0
    assert some > 5


def test_shared_long_rows_and_large_groups():
    rng = np.random.default_rng(8)
    for members, pages, differ in ((2, 9000, 8999), (2, 9000, None), (700, 300, 299), (33, 129, 128)):
        table = np.tile(rng.integers(0, 1 << 20, pages), (members, 1))
        if differ is not None:
            table[members - 1, differ] += 1
        check_shared(table, [pages * 16] * members, [1] * members, [0, members], 16)


def test_shared_groups_leave_sequences_out():
    table = np.tile(np.arange(6), (9, 1))
    lens, n = [96] * 9, [1] * 9
    assert check_shared(table, lens, n, [2, 4, 4, 5, 8], 16) == [0, 0, 95, 95, 0, 95, 95, 95, 0]
    assert check_shared(table, lens, n, [9, 9], 16) == [0] * 9
    assert check_shared(table, lens, n, [0], 16) == [0] * 9


def test_shared_whole_pages_and_the_shortest_past():
    table = np.tile(np.arange(6), (3, 1))
    assert check_shared(table, [90, 50, 96], [1, 0, 30], [0, 3], 16) == [50] * 3
    assert check_shared(table, [90, 50, 96], [1, 50, 30], [0, 3], 16) == [0] * 3
    table[1, 2] = 9
    assert check_shared(table, [90, 50, 96], [1, 0, 30], [0, 3], 16) == [32] * 3


def test_shared_bad_groups_share_nothing():
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    cache = a_cache()
    table = i32(np.tile(np.arange(6), (9, 1)))
    batch = pkg.KvBatch(table, i32([96] * 9), i32(range(10)))
    for groups in ([0, 5, 3, 9], [-1, 9], [0, 10], [0, 4, 1 << 30]):
        got = cache.shared(batch, i32(groups))
        assert cache.device_status()[0] == B.DG_ERR_DEVICE_CHECK
        assert got.prefix.tolist() == [0] * 9
    # lengths out of range are clamped and recorded
    got = cache.shared(pkg.KvBatch(table, i32([96] * 8 + [1 << 29]), i32(range(10))), i32([0, 9]))
    assert cache.device_status()[0] == B.DG_ERR_DEVICE_CHECK and got.prefix.tolist() == [95] * 9
    got = cache.shared(pkg.KvBatch(table, i32([96] * 8 + [-1]), i32(range(10))), i32([0, 9]))
    assert cache.device_status()[0] == B.DG_ERR_DEVICE_CHECK and got.prefix.tolist() == [0] * 9


def test_shared_refusals_and_capture():
    import moe_expert_ffn_dg_gb300 as pkg
    cache = a_cache()
    batch = pkg.KvBatch(i32(np.tile(np.arange(6), (9, 1))), i32([96] * 9), i32(range(10)))
    for groups in (i32([0, 9]).long(), i32([0, 9]).cpu(), i32([])):
        with pytest.raises(ValueError):
            cache.shared(batch, groups)
    groups = i32([0, 9])
    got = cache.shared(batch, groups)
    for kw in (dict(groups=groups.clone(), batch=batch),
               dict(groups=groups, batch=pkg.KvBatch(batch.page_table, batch.lens, batch.cu))):
        with pytest.raises(ValueError):
            cache.shared(out=got, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.shared(batch, groups, out=got)
    got.prefix.zero_()
    graph.replay()
    assert got.prefix.tolist() == [95] * 9
