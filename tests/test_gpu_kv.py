"""The paged cache: append, page forks, page copies and compaction."""

import numpy as np
import pytest
import torch

import attn_ref
from test_gpu_rope import tolerance

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import moe_expert_ffn_dg_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkg.build()
    pkg.load_library()


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def pools(layers, pages, ps, h, d, dtype, seed=0, heads_first=False):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        t = torch.randn(layers, pages, ps, h, d, generator=g).to(dtype).cuda()
        if heads_first:  # [layer, page, head, token, d] in memory
            t = t.transpose(2, 3).contiguous().transpose(2, 3)
        out.append(t)
    return out


def tables(lens, ps, seed=0, spare=1):
    held = [-(-x // ps) for x in lens]
    order = np.random.default_rng(seed).permutation(sum(held) + spare).tolist()
    t = np.full((len(lens), max(1, max(held))), -1, np.int32)
    for b, n in enumerate(held):
        t[b, :n] = [order.pop() for _ in range(n)]
    return t, sum(held) + spare


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d,rot,layout", [(64, 64, "half"), (128, 32, "interleaved"),
                                          (256, 256, "half"), (64, 6, "half"), (128, 0, "half")])
@pytest.mark.parametrize("ps,heads_first", [(16, False), (64, True)])
def test_append(d, rot, layout, dtype, ps, heads_first):
    import moe_expert_ffn_dg_gb300 as pkg
    n, lens = [1, 0, 33, 5, 200], [1, 40, 33, 100, 230]
    table, pages = tables(lens, ps)
    k_pool, v_pool = pools(3, pages, ps, 2, d, dtype, heads_first=heads_first)
    want_k, want_v = k_pool.cpu().clone(), v_pool.cpu().clone()
    cu = np.concatenate([[0], np.cumsum(n)])
    g = torch.Generator().manual_seed(1)
    total = int(cu[-1])
    q = torch.randn(total, 6, d, generator=g).to(dtype)
    kv = torch.randn(total, 4, d, generator=g).to(dtype)  # k and v heads of one product
    cache = pkg.KvCache(k_pool, v_pool)
    rope = pkg.Rope(d, rot_dim=rot, layout=layout) if rot else None
    kvd = kv.cuda()
    q_out = cache.append(kvd[:, :2], kvd[:, 2:], pkg.KvBatch(i32(table), i32(lens), i32(cu)),
                         layer=1, q=q.cuda(), rope=rope)
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    pos = [lens[b] - n[b] + i for b in range(5) for i in range(n[b])]
    rk, rq = kv[:, :2].double(), q.double()
    tk, tq = torch.zeros_like(rk), torch.zeros_like(rq)
    if rot:
        rk, rq = (attn_ref.rotate(t, pos, rot, layout) for t in (rk, rq))
        tk = tolerance(kv[:, :2].double(), rk, pos, rot, layout, 1.0, dtype)
        tq = tolerance(q.double(), rq, pos, rot, layout, 1.0, dtype)
    assert ((q_out.double().cpu() - rq).abs() <= tq).all()
    got_k, got_v = k_pool.cpu(), v_pool.cpu()
    t = 0
    for b in range(5):
        for i in range(n[b]):
            pg, r = int(table[b, pos[t] // ps]), pos[t] % ps
            assert ((got_k[1, pg, r].double() - rk[t]).abs() <= tk[t]).all()
            want_k[1, pg, r] = got_k[1, pg, r]
            want_v[1, pg, r] = kv[t, 2:]
            t += 1
    # every other place is untouched
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v)


def test_append_positions_and_rows_outside():
    """Rotary positions of the caller's; rows outside every sequence and bad
    pages are left alone, the latter reported."""
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    k_pool, v_pool = pools(1, 4, 16, 1, 64, BF)
    before = k_pool.clone()
    cache = pkg.KvCache(k_pool, v_pool)
    k = torch.randn(6, 1, 64).to(BF).cuda()
    rope = pkg.Rope(64)
    pos = i32([5, 6, 7, 8, 9, 10])
    q_out = torch.full_like(k, 3.0)
    # rows 0 and 5 belong to no sequence
    cache.append(k, k, pkg.KvBatch(i32([[2], [0]]), i32([2, 10]), i32([1, 3, 5])), q=k, rope=rope,
                 positions=pos, q_out=q_out)
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    full = rope.apply(k, pos)
    assert torch.equal(q_out[1:5], full[1:5]) and (q_out[[0, 5]] == 3.0).all()
    want = before.clone()
    want[0, 2, 0:2] = full[1:3]
    want[0, 0, 8:10] = full[3:5]
    assert torch.equal(k_pool, want)
    # page ids past the pool, a token past its row, a negative position
    for table, lens in (([[9]], [2]), ([[-1]], [2]), ([[1]], [18]), ([[1]], [1])):
        cache.append(k[:2], k[:2], pkg.KvBatch(i32(table), i32(lens), i32([0, 2])), rope=rope)
        torch.cuda.synchronize()
        status = cache.device_status()
        assert status[0] == B.DG_ERR_DEVICE_CHECK and status[1] in (40, 41)
        assert cache.device_status()[0] == 0
    want[0, 1, 0] = rope.apply(k[:2], i32([-1, 0]))[1]  # the one good token of the last
    assert torch.equal(k_pool[:, [0, 2, 3]], want[:, [0, 2, 3]])
    assert torch.equal(k_pool[0, 1, 0], want[0, 1, 0])


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("ps,h,d", [(16, 1, 64), (64, 3, 128), (256, 8, 256)])
def test_copy(ps, h, d, heads_first):
    import moe_expert_ffn_dg_gb300 as pkg
    k_pool, v_pool = pools(2, 9, ps, h, d, FP, heads_first=heads_first)
    want_k, want_v = k_pool.clone(), v_pool.clone()
    rows = [(0, 5, ps), (0, 6, 1), (-1, -1, 0), (3, 7, ps - 1), (2, 8, 0), (-1, 4, ps)]
    for a, b, m in rows:
        if a >= 0:
            want_k[:, b, :m], want_v[:, b, :m] = want_k[:, a, :m], want_v[:, a, :m]
    cache = pkg.KvCache(k_pool, v_pool)
    cache.copy(i32(rows))
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    assert torch.equal(k_pool, want_k) and torch.equal(v_pool, want_v)
    cache.copy(i32([(1, 9, 3), (9, 1, 3), (1, -1, 3)]))  # out of range: nothing moves
    torch.cuda.synchronize()
    assert cache.device_status()[0] != 0
    assert torch.equal(k_pool, want_k) and torch.equal(v_pool, want_v)


@pytest.mark.parametrize("ps,h,d", [(16, 1, 64), (32, 5, 128), (128, 2, 256)])
def test_gather(ps, h, d):
    import moe_expert_ffn_dg_gb300 as pkg
    rng = np.random.default_rng(ps)
    src_len, keep_len = [100, 0, 300, 17, 1], [40, 0, 299, 0, 1]
    both, pages = tables(src_len + keep_len, ps)
    src, dst = both[:5], both[5:]
    k_pool, v_pool = pools(2, pages, ps, h, d, BF)
    want = [k_pool.clone(), v_pool.clone()]
    # the third sequence reversed and with repeats
    keep = [rng.permutation(a)[:b] if i != 2 else rng.integers(0, a, b)
            for i, (a, b) in enumerate(zip(src_len, keep_len))]
    for b in range(5):
        for i, s in enumerate(keep[b]):
            for w in want:
                w[:, dst[b, i // ps], i % ps] = w[:, src[b, s // ps], s % ps]
    cu = np.concatenate([[0], np.cumsum(keep_len)])
    cache = pkg.KvCache(k_pool, v_pool)
    cache.gather(i32(src), i32(dst), i32(cu), i32(np.concatenate(keep)))
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0
    assert torch.equal(k_pool, want[0]) and torch.equal(v_pool, want[1])
    for bad in ([-1], [both.shape[1] * ps]):
        cache.gather(i32(src[:1]), i32(dst[:1]), i32([0, 1]), i32(bad))
        torch.cuda.synchronize()
        assert cache.device_status()[0] != 0
    assert torch.equal(k_pool, want[0]) and torch.equal(v_pool, want[1])


def test_moves_past_32_bit_offsets():
    """A pool of more than 2^32 elements: pages at its far end."""
    import moe_expert_ffn_dg_gb300 as pkg
    ps, h, d = 256, 8, 128
    pages = (1 << 32) // (ps * h * d) + 40
    k_pool = torch.empty(1, pages, ps, h, d, dtype=BF, device="cuda")
    v_pool = torch.empty_like(k_pool)
    cache = pkg.KvCache(k_pool, v_pool)
    a, b = pages - 1, pages - 5
    new = torch.randn(200, 2 * h, d, dtype=BF, device="cuda")
    batch = pkg.KvBatch(i32([[a]]), i32([200]), i32([0, 200]))
    cache.append(new[:, :h], new[:, h:], batch)
    cache.copy(i32([(a, b, 200)]))
    cache.gather(i32([[b]]), i32([[pages - 9]]), i32([0, 200]), i32(np.arange(200)))
    q = torch.randn(1, h, d, dtype=BF, device="cuda")
    attn = pkg.PagedAttention(cache, h, left=-1, right=-1)
    outs = [attn.forward(q, pkg.KvBatch(i32([[p]]), i32([200]), i32([0, 1])))
            for p in (a, b, pages - 9)]
    torch.cuda.synchronize()
    assert cache.device_status()[0] == 0 and attn.device_status()[0] == 0
    for p in (a, b, pages - 9):
        assert torch.equal(k_pool[0, p, :200], new[:, :h])
        assert torch.equal(v_pool[0, p, :200], new[:, h:])
    s = torch.einsum("hd,khd->hk", q[0].double(), new[:, :h].double()) * d ** -0.5
    want = torch.einsum("hk,khd->hd", torch.softmax(s, -1), new[:, h:].double())
    mag = torch.einsum("hk,khd->hd", torch.softmax(s, -1), new[:, h:].double().abs())
    assert ((outs[0][0].double() - want).abs() <= 2.0 ** -8 * (mag + want.abs()) * 1.01).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------------ forks

def plain_fork(table, lens, ref, parent, grow, ps):
    """The definition, a sequence at a time."""
    row, ref = table.shape[1], ref.copy()
    held = [table[s, :-(-int(lens[s]) // ps)] for s in range(len(lens))]
    for h in held:
        np.subtract.at(ref, h, 1)
    rows = [list(held[p]) if p >= 0 else [] for p in parent]
    have = [int(lens[p]) if p >= 0 else 0 for p in parent]
    for r in rows:
        np.add.at(ref, r, 1)
    growing = {}
    for j, r in enumerate(rows):
        if grow[j] > 0 and have[j] % ps:
            growing.setdefault(r[-1], []).append(j)
    split = [have[j] % ps > 0 and grow[j] > 0 and
             (ref[r[-1]] > len(growing[r[-1]]) or growing[r[-1]][0] != j)
             for j, r in enumerate(rows)]
    want = [-(-(have[j] + int(grow[j])) // ps) for j in range(len(rows))]
    need = [want[j] - len(rows[j]) + split[j] for j in range(len(rows))]
    free = [i for i in range(len(ref)) if ref[i] == 0]
    short = max(0, sum(need) - len(free))
    if any(w > row for w in want) or any(have[j] + grow[j] > row * ps for j in range(len(rows))):
        short = -1
    copies = [(-1, -1, 0)] * len(rows)
    if short == 0:
        for j, r in enumerate(rows):
            got, free = free[:need[j]], free[need[j]:]
            ref[got] += 1
            if split[j]:
                copies[j] = (r[-1], got[0], have[j] % ps)
                ref[r[-1]] -= 1
                r.pop()
            r.extend(got)
            have[j] += int(grow[j])
    out = np.full((len(rows), row), -1, np.int64)
    for j, r in enumerate(rows):
        out[j, :len(r)] = r
    return out, have, ref, copies, short


def run_fork(table, lens, ref, parent, grow, ps, inplace=False, pager=None):
    import moe_expert_ffn_dg_gb300 as pkg
    table, ref = np.asarray(table), np.asarray(ref)
    pager = pager or pkg.KvPager(len(ref), ps)
    dref = i32(ref)
    out = None
    if inplace:
        n = len(parent)
        new = [torch.empty(s, dtype=torch.int32, device="cuda")
               for s in ((n, table.shape[1]), (n,), (n, 3), (1,))]
        out = pkg.KvFork(new[0], new[1], dref, new[2], new[3])
    f = pager.fork(i32(table), i32(lens), dref, i32(parent), i32(grow), out=out)
    torch.cuda.synchronize()
    want = plain_fork(table, lens, ref, parent, grow, ps)
    assert int(f.short[0]) == want[4]
    assert np.array_equal(f.ref.cpu().numpy(), want[2])
    assert f.lens.cpu().tolist() == want[1]
    assert f.copies.cpu().tolist() == [list(map(int, c)) for c in want[3]]
    assert np.array_equal(f.table.cpu().numpy(), want[0])
    assert pager.device_status()[0] == 0
    return [t.cpu().numpy() for t in (f.table, f.lens, f.ref)]


@pytest.mark.parametrize("slots,row,ps,pages,seed", [
    (1, 4, 16, 10, 0), (7, 9, 16, 200, 1), (40, 33, 32, 2000, 2), (300, 20, 256, 9000, 3),
    (1500, 6, 64, 20000, 4), (4096, 3, 16, 30001, 5), (5, 700, 16, 5000, 6)])
def test_fork_steps(slots, row, ps, pages, seed):
    """Several steps from an empty state, with whatever sharing they build up."""
    import moe_expert_ffn_dg_gb300 as pkg
    rng = np.random.default_rng(seed)
    pager = pkg.KvPager(pages, ps)
    table, lens = np.full((slots, row), -1, np.int32), np.zeros(slots, np.int32)
    ref = (rng.random(pages) < 0.01).astype(np.int32)
    for step in range(4):
        n = slots if step < 3 else max(1, slots // 2)
        parent = np.where(rng.random(n) < 0.5, np.arange(n) % slots,
                          rng.integers(0, slots, n)).astype(np.int32)
        parent[rng.random(n) < 0.15] = -1
        have = np.where(parent >= 0, lens[np.maximum(parent, 0)], 0)
        room = row * ps - have
        grow = np.minimum(rng.integers(0, max(2, row * ps // 4), n), room)
        grow[rng.random(n) < 0.2] = 0
        table, lens, ref = run_fork(table, lens, ref, parent, grow, ps, inplace=step % 2 == 1,
                                    pager=pager)


def test_fork_of_a_partly_filled_page():
    t = [[3, 5, -1, -1]]
    ref = np.zeros(12, np.int32)
    ref[[3, 5]] = 1
    run_fork(t, [20], ref, [0, 0, 0], [1, 1, 1], 16)      # the first child keeps it
    run_fork(t, [20], ref, [0, 0, 0], [0, 1, 1], 16)      # a child that stays: both others split
    run_fork(t, [20], ref, [0, 0], [0, 0], 16)            # nobody grows
    run_fork(t, [32], ref, [0, 0], [1, 1], 16)            # full page: nothing to split
    ref[5] = 2                                            # held elsewhere too
    run_fork(t, [20], ref, [0], [5], 16)
    run_fork(t, [20], ref, [-1], [1], 16)                 # freed, a new one in its place
    run_fork(t, [20], ref, [], [], 16)                    # freed, nothing else


def test_fork_without_enough_pages_or_room():
    t = [[0, 1, -1], [1, -1, -1]]
    ref = np.array([1, 2, 0, 0], np.int32)
    run_fork(t, [30, 16], ref, [0, 1, 0], [2, 40, 1], 16)
    run_fork(t, [30, 16], ref, [0, 1], [2, 32], 16)       # just enough
    run_fork(t, [30, 16], ref, [0, 1], [18, 33], 16)      # a row outgrown
    run_fork(t, [30, 16], ref, [0, 1], [2 ** 31 - 1, 0], 16)


def test_fork_bad_inputs_are_reported():
    import moe_expert_ffn_dg_gb300 as pkg
    from moe_expert_ffn_dg_gb300 import binding as B
    pager = pkg.KvPager(8, 16)
    ref = i32([1] * 4 + [0] * 4)

    def go(table, lens, parent, grow, r=ref):
        f = pager.fork(i32(table), i32(lens), r, i32(parent), i32(grow))
        torch.cuda.synchronize()
        return f, pager.device_status()[0]
    f, s = go([[0, 99]], [20], [0, -1], [0, 1])
    assert s == B.DG_ERR_DEVICE_CHECK and f.table.tolist() == [[0, -1], [4, -1]]
    f, s = go([[0, 1]], [20], [7], [1])
    assert s == B.DG_ERR_DEVICE_CHECK and f.lens.tolist() == [1]
    f, s = go([[0, 1]], [-3], [0], [-1])
    assert s == B.DG_ERR_DEVICE_CHECK and f.lens.tolist() == [0]
    f, s = go([[0, 1]], [1000], [0], [0])
    assert s == B.DG_ERR_DEVICE_CHECK and f.lens.tolist() == [32]
    f, s = go([[0, 1]], [32], [-1], [0], i32([1, 0] + [1] * 6))  # a count below zero
    assert s == B.DG_ERR_DEVICE_CHECK
    f, s = go([[0, 1]], [20], [0], [1])
    assert s == 0


def test_steps_in_a_graph():
    """Fork, split copies, append and gather captured once and replayed on new
    contents of the same tensors."""
    import moe_expert_ffn_dg_gb300 as pkg
    ps, pages = 16, 40
    k_pool, v_pool = pools(2, pages, ps, 2, 64, BF, seed=5)
    cache, pager = pkg.KvCache(k_pool, v_pool), pkg.KvPager(pages, ps)
    table = i32([[3, 5, -1, -1], [7, -1, -1, -1]])
    lens, parent, grow = i32([20, 16]), i32([0, 0]), i32([3, 5])
    ref = i32(np.bincount([3, 5, 7], minlength=pages))
    kv = torch.randn(8, 4, 64, dtype=BF, device="cuda")
    cu = i32([0, 3, 8])
    rope = pkg.Rope(64)

    def step(out=None):
        f = pager.fork(table, lens, ref, parent, grow, out=out)
        cache.copy(f.copies)
        cache.append(kv[:, :2], kv[:, 2:], pkg.KvBatch(f.table, f.lens, cu), layer=1, rope=rope)
        return f
    f = step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (k_pool, v_pool, f.table, f.lens, f.ref, f.copies)]
    assert f.copies.tolist() == [[-1, -1, 0], [5, 0, 4]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(f)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (k_pool, v_pool, f.table, f.lens, f.ref, f.copies)):
        assert torch.equal(a, b)
    parent.copy_(i32([1, 0]))  # another step: nothing is shared, nothing split
    graph.replay()
    torch.cuda.synchronize()
    assert (f.copies[:, 0] == -1).all() and f.lens.tolist() == [19, 25]
    assert int(f.short[0]) == 0
    assert cache.device_status()[0] == 0 and pager.device_status()[0] == 0
