"""Paged attention of calls large enough that beginning an item counts in the
split of the work (small ones never reach that), against 64 bits.  Tolerances
are those of the small tests."""

import random

import pytest
import torch

import test_attn_schedule as schedule
from test_gpu_attn import BF, FP, _built, make, tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return schedule.library(tmp_path_factory.mktemp("schedule"))


def plain(q, k, v, table, lens, cu, left, right, scale):
    """As attn_ref.attention, a sequence at a time on the GPU in 64 bits."""
    hkv, d = k.shape[2], k.shape[3]
    group = q.shape[1] // hkv
    out, mag, tot = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64, device="cuda")
    smax = torch.zeros(*q.shape[:2], 1, dtype=torch.float64, device="cuda")
    for b, kv in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        if not n or not kv:
            continue
        pages = table[b, :-(-kv // k.shape[1])].long()
        kk = k[pages].flatten(0, 1)[:kv].double().transpose(0, 1)
        vv = v[pages].flatten(0, 1)[:kv].double().transpose(0, 1)
        qq = q[rows].double().view(n, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * n, d)
        at = torch.arange(n, device="cuda")[:, None] + kv - n
        j = torch.arange(kv, device="cuda")[None]
        seen = torch.ones(n, kv, dtype=torch.bool, device="cuda")
        if left >= 0:
            seen &= j >= at - left
        if right >= 0:
            seen &= j <= at + right
        seen = seen.repeat(group, 1)
        s = (qq @ kk.mT * scale).masked_fill(~seen, -torch.inf)
        t = torch.logsumexp(s, -1, keepdim=True)
        w = torch.exp(s - t.masked_fill(t == -torch.inf, 0.0))

        def back(x):
            return x.view(hkv, group, n, -1).permute(2, 0, 1, 3).flatten(1, 2)
        out[rows], mag[rows] = back(w @ vv), back(w @ vv.abs())
        tot[rows] = back(seen.double() @ vv.abs())
        lse[rows] = back(t)[..., 0]
        sm = (qq.abs() @ kk.abs().mT * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
        smax[rows] = back(sm)
    return out, lse, mag, tot, smax


# head size, type, key/value heads, query heads a group, page; sequences, most
# new tokens, most cached ones; a table wide enough for caches past the L2
CASES = {
    "few rows, 64": (64, FP, 8, 4, 16, 70, 1, 900, False),
    "few rows, 128": (128, BF, 8, 3, 64, 70, 1, 900, False),
    "few rows, 256": (256, BF, 8, 2, 32, 70, 1, 900, False),
    "many rows, 64": (64, BF, 4, 4, 64, 18, 260, 4000, False),
    "many rows, 128": (128, FP, 4, 4, 128, 18, 260, 4000, False),
    "many rows, 128, teams": (128, BF, 4, 4, 256, 2, 900, 5000, True),
    "many rows, 256": (256, BF, 8, 4, 64, 18, 60, 4000, False),
    "many rows, 256, teams of pairs": (256, FP, 8, 4, 64, 8, 260, 3500, False),
}


@pytest.mark.parametrize("left,right", [(-1, 0), (1900, 3), (-1, -1)])
@pytest.mark.parametrize("name", CASES)
def test_items_whose_beginnings_count(name, left, right, lib):
    import moe_expert_ffn_dg_gb300 as pkg
    d, dtype, hkv, group, ps, seqs, new, past, wide = CASES[name]
    rng = random.Random(name)
    # ragged, an empty chunk, an empty cache and a short one among them
    n = [rng.randint(max(1, new * 2 // 3), new) for _ in range(seqs)]
    lens = [rng.randint(past // 2, past) for _ in range(seqs)]
    if seqs > 2:
        n[1], lens[2], lens[3] = 0, 0, min(n[3], 17)
    q, k, v, table, lens, cu = make(n, lens, hkv * group, hkv, d, ps, dtype, 50)
    if wide:
        table = torch.nn.functional.pad(table, (0, 600 - table.shape[1]), value=-1)
    cap = table.shape[1] * ps
    rows = sum(n) * group // seqs
    many = name.startswith("many")
    assert many == (rows > (32 if d == 256 else 128))
    nq, team, over = schedule.rule(d, many, rows, cap * hkv * d * 4)
    assert (team > (2 if d == 256 else 1)) == ("teams" in name)
    ctas = min(160, torch.cuda.get_device_properties(0).multi_processor_count)
    bad, used = schedule.go(lib, nq, team, over, lens, n, hkv, group, left, right, ctas, cap)
    assert bad == 0 and used == over  # the beginnings count
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    table = table.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = pkg.KvCache(k[None], v[None])
    attn = pkg.PagedAttention(cache, hkv * group, left=left, right=right)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out, lse = attn.forward(q, pkg.KvBatch(table, torch.tensor(lens, **i32),
                                           torch.tensor(cu, **i32)), lse=lse)
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    ref = plain(q, k, v, table, lens, cu, left, right, d ** -0.5)
    tol, ltol = tolerance(ref, dtype, d, max(lens))
    err = (out.double() - ref[0]).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    none = ref[1] == -torch.inf
    assert (lse[none] == -torch.inf).all() and (out[none] == 0).all()
    assert ((lse.double() - ref[1])[~none].abs() <= ltol[~none]).all()
