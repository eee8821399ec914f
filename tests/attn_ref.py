"""Plain 64-bit implementations of the attention half, on the CPU, one token
and one page at a time where that is plainest."""

import math

import numpy as np
import torch


def frequencies(rot, theta=1e4, scaling="none", factor=1.0, orig_len=0.0, slow=1.0, fast=32.0):
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        g = np.clip((orig_len * f / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        f = g * f + (1 - g) * f / factor
    return f


def rotate(x, positions, rot, layout, amplitude=1.0, grad=False, **kw):
    """x [T, H, D] float64 tensor, positions a list of ints."""
    y = x.clone()
    f = frequencies(rot, **kw)
    a = np.array([[math.remainder(p * w, 2 * math.pi) for w in f] for p in positions])
    c = torch.from_numpy(np.cos(a) * amplitude)[:, None]
    s = torch.from_numpy(np.sin(a) * amplitude * (-1 if grad else 1))[:, None]
    i = torch.arange(rot // 2)
    lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def cached(pages, table_row, n):
    """The first n tokens of a sequence, [n, kv_heads, dim] float64."""
    ps = pages.shape[1]
    return torch.stack([pages[int(table_row[j // ps]), j % ps] for j in range(n)]).double() \
        if n else torch.zeros(0, *pages.shape[2:], dtype=torch.float64)


def attention(q, k_pages, v_pages, table, lens, cu, left, right, scale):
    """out, lse, and the sums a tolerance needs: sum p |v|, sum |v| over what a
    query sees, and the largest sum |q k| scale of a query."""
    T, H, D = q.shape
    G = H // k_pages.shape[2]
    out, mag, tot = (torch.zeros(T, H, D, dtype=torch.float64) for _ in range(3))
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    smax = torch.zeros(T, H, 1, dtype=torch.float64)
    for b in range(len(lens)):
        n, kv = cu[b + 1] - cu[b], lens[b]
        k, v = cached(k_pages, table[b], kv), cached(v_pages, table[b], kv)
        for i in range(n):
            p = kv - n + i
            lo = 0 if left < 0 else max(0, p - left)
            hi = kv if right < 0 else min(kv, p + right + 1)
            if hi <= lo:
                continue
            for h in range(H):
                qq, kk, vv = q[cu[b] + i, h].double(), k[lo:hi, h // G], v[lo:hi, h // G]
                s = (kk @ qq) * scale
                t = torch.logsumexp(s, 0)
                w = torch.exp(s - t)
                r = cu[b] + i
                out[r, h], lse[r, h] = w @ vv, t
                mag[r, h], tot[r, h] = w @ vv.abs(), vv.abs().sum(0)
                smax[r, h] = (kk.abs() @ qq.abs()).max() * scale
    return out, lse, mag, tot, smax
