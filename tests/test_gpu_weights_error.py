"""How far attention weights are from 64 bits, by their root mean square.

The tensor core adds to its fp32 accumulator towards zero, 16 products at a time, so
scores lie nearer to zero than they should, and the loss does not average out over
the rows that a weight sums.  `model` works that out for the inputs at hand: sums of
16 exact products, cut to 24 bits after each addition, one or two accumulators a
score; the factor scale log2 e and the scaled log-sum rounded to fp32, as the kernel
does.  A kernel may be off by sqrt(2) times that, and by 2^-22, the exponential's
error, beside it.  Twice as many accumulators lose half as much, so at head size 256,
where two are paid for, one is over the bound (checked of the model, for the inputs of
a test).  With the attention's own log-sums the same bound holds against the softmax:
what its scores lose, and with them its log-sums, falls out of the difference for the
most part where both have one accumulator (head sizes 64 and 128)."""

import re

import numpy as np
import pytest
import torch

from test_attn_sources import CSRC
from test_gpu_attn import BF, FP, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def accumulators(d):
    src = open(f"{CSRC}/dg_weights.cu").read()
    at, more, one = re.search(r"kAccs = D == (\d+) \? (\d+) : (\d+);", src).groups()
    return int(more) if d == int(at) else int(one)


def cut(x):
    """To 24 bits, towards zero."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def near(x):
    return x.astype(np.float32).astype(np.float64)


def model(q, k, lse, accs):
    """Weights of the keys, q [rows, d], k [keys, d], lse [rows]."""
    d = q.shape[1]
    parts = []
    for a in np.split(np.arange(d), accs):
        s = np.zeros((q.shape[0], k.shape[0]))
        for c in np.split(a, len(a) // 16):
            s = cut(s + q[:, c] @ k[:, c].T)
        parts.append(s)
    s = near(sum(parts))
    scale2 = float(np.float32(np.float32(d ** -0.5) * np.float32(1.4426950408889634)))
    off = near(np.float64(np.float32(-1.4426950408889634)) * lse)
    return np.exp2(near(s * scale2 + off[:, None]))


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("tokens", [2, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_error(d, tokens, dtype):
    """Many rows a sequence, or eight (the kernel's two widths): 512 in all, 4 query
    heads on one, every sequence over the same 1500 tokens."""
    import moe_expert_ffn_dg_gb300 as pkg
    g = torch.Generator().manual_seed(d + tokens)
    seqs, kv, group, ps = 128 // tokens, 1500, 4, 64
    q = (3 * torch.randn(seqs * tokens, group, d, generator=g)).to(dtype)
    pages = -(-kv // ps)
    k = torch.randn(1, pages, ps, 1, d, generator=g).to(dtype)
    rows = q.double().numpy().reshape(-1, d)
    keys = k.double().numpy().reshape(-1, d)[:kv]
    exact = rows @ keys.T * float(np.float32(d ** -0.5))
    lse = np.log(np.exp(exact).sum(1))
    lse32 = lse.astype(np.float32)

    def sums(w):  # rows of a sequence
        return w.reshape(seqs, -1, kv).sum(1)
    want = sums(np.exp(exact - lse32[:, None].astype(np.float64)))

    def lost(accs):
        return rms(sums(model(rows, keys, lse32.astype(np.float64), accs)) - want) / rms(want)
    accs = accumulators(d)
    bound = 2 ** 0.5 * lost(accs) + 2.0 ** -22
    if accs > 1:
        assert bound < lost(accs // 2)

    table = torch.arange(pages, dtype=torch.int32).repeat(seqs, 1).cuda()
    cache = pkg.KvCache(k.cuda(), torch.zeros_like(k).cuda())
    batch = pkg.KvBatch(table, torch.full((seqs,), kv, dtype=torch.int32, device="cuda"),
                        torch.arange(0, seqs * tokens + 1, tokens, dtype=torch.int32, device="cuda"))
    attn = pkg.PagedAttention(cache, group, right=-1)
    w = torch.zeros(seqs, kv, device="cuda")
    qd = q.cuda()
    attn.weights(qd, torch.from_numpy(lse32.reshape(-1, group)).cuda(), batch, w, decay=0.0)
    err = rms(w.double().cpu().numpy() - want) / rms(want)
    assert err <= bound, (err, bound)
    own = torch.empty(seqs * tokens, group, device="cuda")
    attn.forward(qd, batch, lse=own)
    attn.weights(qd, own, batch, w, decay=0.0)
    want = sums(np.exp(exact - lse[:, None]))
    beside = rms(w.double().cpu().numpy() - want) / rms(want)
    print(f"{d} {tokens} {dtype}: {err:.2g} of {bound:.2g}, own log-sums {beside:.2g}")
    assert beside <= bound, (beside, bound)
    assert attn.device_status()[0] == 0
