"""Serving of forked and thinned sequences over the paged cache: the prefix
that forks share and attention that reads it once, the attention weight that
every cached token received, and the choice of the tokens that stay when a cache
is thinned.  Each case below is one call of one of them.

``own`` False computes the operators from elementary torch operations in 32
bits; ``own`` True makes the calls of the package.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # a step of eight candidates forked from one conversation: what they share
        _case("shared_small", "shared", groups=1, size_lo=8, size_hi=8, n_lo=1, n_hi=1,
              prefix_lo=1000, prefix_hi=1000, tail_lo=0, tail_hi=90, page=64, row=32, lens=31),
        # the same for a full server: 512 sequences of 40 prompts
        _case("shared_server", "shared", groups=40, size_lo=1, size_hi=25, n_lo=1, n_hi=4,
              prefix_lo=0, prefix_hi=24000, tail_lo=0, tail_hi=900, page=64, row=512, lens=32),
        # four candidates of a short conversation, one token each: latency
        _case("prefix_few", "prefix", groups=1, size_lo=4, size_hi=4, n_lo=1, n_hi=1,
              prefix_lo=2000, prefix_hi=2000, tail_lo=3, tail_hi=70, q_heads=16, kv_heads=4,
              dim=64, page=16, lens=33, dtype="fp16"),
        # a decode step of 64 samples of one long prompt
        _case("prefix_samples", "prefix", groups=1, size_lo=64, size_hi=64, n_lo=1, n_hi=1,
              prefix_lo=16000, prefix_hi=16000, tail_lo=10, tail_hi=600, q_heads=32, kv_heads=8,
              dim=128, page=64, lens=34, dtype="bf16"),
        # prompts with different numbers of samples, one to four tokens each
        # (drafted ones among them), some prompts without a fork
        _case("prefix_ragged", "prefix", groups=12, size_lo=1, size_hi=14, n_lo=1, n_hi=4,
              prefix_lo=300, prefix_hi=9000, tail_lo=0, tail_hi=400, q_heads=16, kv_heads=8,
              dim=256, page=64, lens=35, dtype="bf16"),
        # 128 sequences behind one document, four drafted tokens each
        _case("prefix_document", "prefix", groups=1, size_lo=128, size_hi=128, n_lo=4, n_hi=4,
              prefix_lo=65536, prefix_hi=65536, tail_lo=50, tail_hi=500, q_heads=32, kv_heads=8,
              dim=128, page=128, lens=36, dtype="bf16"),
        # weights that the tokens of one short conversation got in a step
        _case("weights_token", "weights", seqs=1, n_lo=1, n_hi=1, past_lo=776, past_hi=776,
              q_heads=16, kv_heads=4, dim=64, page=16, left=-1, right=0, decay=0.9, lens=37,
              dtype="fp16"),
        # the same for a serving step of 64 ragged sequences
        _case("weights_step", "weights", seqs=64, n_lo=1, n_hi=1, past_lo=1000, past_hi=16000,
              q_heads=32, kv_heads=8, dim=128, page=64, left=-1, right=0, decay=0.98, lens=38,
              dtype="bf16"),
        # canvases of 256 tokens weigh their prompts before those are thinned
        _case("weights_canvases", "weights", seqs=8, n_lo=256, n_hi=256, past_lo=500,
              past_hi=8000, q_heads=16, kv_heads=8, dim=256, page=64, left=-1, right=-1,
              decay=1.0, lens=39, dtype="bf16"),
        # a chunk of a long prompt: 4096 tokens behind 12288
        _case("weights_chunk", "weights", seqs=1, n_lo=4096, n_hi=4096, past_lo=12288,
              past_hi=12288, q_heads=32, kv_heads=8, dim=128, page=128, left=-1, right=0,
              decay=1.0, lens=40, dtype="bf16"),
        # eight conversations cut to their 512 most attended tokens
        _case("select_small", "select", seqs=8, len_lo=100, len_hi=1500, width=2048, budget=512,
              first=4, last=32, lens=41),
        # 48 long ones cut to 16384 tokens
        _case("select_long", "select", seqs=48, len_lo=8000, len_hi=131072, width=131072,
              budget=16384, first=16, last=256, lens=42),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["shared", "prefix", "prefix", "prefix", "weights", "weights", "weights",
                     "select", "select"])
    dt = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    seed = rng.randrange(1 << 30)
    if op == "shared":
        top = _log_int(rng, 1, 16000)
        tail = _log_int(rng, 1, 2000)
        return dict(op=op, groups=_log_int(rng, 1, 60), size_lo=rng.choice([0, 1, 2]),
                    size_hi=rng.randint(2, 12), n_lo=rng.choice([0, 1]), n_hi=rng.randint(1, 5),
                    prefix_lo=rng.choice([0, top // 2, top]), prefix_hi=top, tail_lo=0,
                    tail_hi=tail, page=page, row=-(-(top + tail + 8) // page) + rng.randint(0, 9),
                    lens=seed)
    if op == "prefix":
        groups = rng.choice([1, 1, 2, 3, 5, 9])
        size = _log_int(rng, 2, max(2, 96 // groups))
        top = _log_int(rng, 16, 20000 // groups)
        n = rng.choice([1, 1, 1, 2, 3, 5, 9])
        return dict(op=op, groups=groups, size_lo=rng.choice([size, 1, 0]), size_hi=size,
                    n_lo=rng.choice([n, n, 0]), n_hi=n, prefix_lo=rng.choice([0, top // 2, top]),
                    prefix_hi=top, tail_lo=0, tail_hi=_log_int(rng, 1, 1500),
                    q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), kv_heads=kv, dim=dim,
                    page=page, lens=seed, dtype=dt)
    if op == "weights":
        kind = rng.choice(["step", "canvas", "chunk"])
        if kind == "step":
            seqs, n, past = _log_int(rng, 1, 200), 1, _log_int(rng, 16, 8000)
        elif kind == "canvas":
            seqs, n, past = rng.randint(1, 8), rng.choice([32, 256]), _log_int(rng, 16, 6000)
        else:
            seqs, n, past = rng.randint(1, 4), _log_int(rng, 3, 1500), _log_int(rng, 1, 8000)
        return dict(op=op, seqs=seqs, n_lo=rng.choice([n, n, max(0, n // 3)]), n_hi=n,
                    past_lo=rng.choice([0, past // 4, past]), past_hi=past,
                    q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), kv_heads=kv, dim=dim,
                    page=page, left=rng.choice([-1, -1, rng.randint(0, 300), 1023]),
                    right=-1 if kind == "canvas" else rng.choice([0, 0, -1, 7]),
                    decay=rng.choice([0.0, 0.9, 1.0]), lens=seed, dtype=dt)
    seqs = _log_int(rng, 1, 200)
    width = _log_int(rng, 16, min(131072, 4000000 // seqs))
    budget = _log_int(rng, 1, width)
    first = rng.choice([0, 0, min(4, budget)])
    return dict(op=op, seqs=seqs, len_lo=rng.choice([0, 1, width // 2]), len_hi=width, width=width,
                budget=budget, first=first, last=rng.choice([0, min(64, budget - first)]),
                lens=seed)


# ------------------------------------------------------------------ inputs

def _chunks(case):
    """New tokens and total lengths of the sequences of a case, and for forks
    the prompt's length of each and the bounds of the groups: a function of the
    case alone."""
    rng = random.Random(case["lens"])
    if case["op"] == "weights":
        n = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
        past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
        return n, [a + b for a, b in zip(n, past)], None, None
    n, lens, prompt, bounds = [], [], [], [0]
    for _ in range(case["groups"]):
        top = rng.randint(case["prefix_lo"], case["prefix_hi"])
        for _ in range(rng.randint(case["size_lo"], case["size_hi"])):
            n.append(rng.randint(case["n_lo"], case["n_hi"]))
            prompt.append(top)
            lens.append(top + rng.randint(case["tail_lo"], case["tail_hi"]) + n[-1])
        bounds.append(len(n))
    if not n:  # one sequence at least
        n, lens, prompt, bounds[-1] = [1], [case["prefix_hi"] + 1], [case["prefix_hi"]], 1
    return n, lens, prompt, bounds


def _tables(case, lens, prompt, bounds, nrng):
    """Page table of sequences that hold their prompt's whole pages in common
    (a part of a page is every sequence's own), and the number of pages."""
    page = case["page"]
    need = [-(-x // page) for x in lens]
    width = max(case.get("row", 0), max(need), 1)
    table = np.full((len(lens), width), -1, np.int64)
    at = 0
    for g in range(len(bounds) - 1):
        a, b = bounds[g], bounds[g + 1]
        if a == b:
            continue
        k = prompt[a] // page
        table[a:b, :k] = np.arange(at, at + k)
        at += k
        for s in range(a, b):
            table[s, k:need[s]] = np.arange(at, at + need[s] - k)
            at += need[s] - k
    pages = at + 3
    order = nrng.permutation(pages)
    return np.where(table >= 0, order[table], -1), pages


def _gpu(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device="cuda")


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _attended(case, gen, pages, total):
    """Queries, and keys of which one in fifty draws much of the attention, as
    the tokens do that are worth keeping."""
    d, kvh, group = case["dim"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    u = torch.nn.functional.normalize(_randn(gen, kvh, d), dim=-1)
    k = _randn(gen, pages, case["page"], kvh, d)
    pull = torch.rand(pages, case["page"], kvh, 1, generator=gen, device="cuda") < 0.02
    k += pull * (1.2 * math.sqrt(d)) * u
    q = _randn(gen, total, kvh, group, d) + 3.0 * u[:, None]
    dt = _T[case["dtype"]]
    return q.reshape(total, case["q_heads"], d).to(dt), k.to(dt)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    nrng = np.random.default_rng(seed)
    op, s = case["op"], {"case": case}
    if op == "select":
        rng = random.Random(case["lens"])
        lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
        s["lens"] = _gpu(lens)
        w = torch.exp(2.5 * _randn(gen, case["seqs"], case["width"]) - 6.0)
        # tokens that nothing has attended to yet, and equal small weights
        r = torch.rand(case["seqs"], case["width"], generator=gen, device="cuda")
        s["weights"] = torch.where(r < 0.1, 0.0, torch.where(r < 0.2, 2.0 ** -12, w))
        return s
    n, lens, prompt, bounds = _chunks(case)
    if op == "shared":
        # how long a prompt is, another each time
        for a, b in zip(bounds[:-1], bounds[1:]):
            cut = int(nrng.integers(0, prompt[a] // 2 + 1)) if a < b else 0
            for i in range(a, b):
                lens[i], prompt[i] = lens[i] - cut, prompt[i] - cut
    total = sum(n)
    s["lens"], s["cu"] = _gpu(lens), _gpu(np.concatenate([[0], np.cumsum(n)]))
    if op == "weights":
        table, pages = _tables(case, lens, [0] * len(n), list(range(len(n) + 1)), nrng)
    else:
        table, pages = _tables(case, lens, prompt, bounds, nrng)
        s["groups"] = _gpu(bounds)
    s["table"], s["pages"] = _gpu(table), pages
    if op == "shared":
        s["k_pages"] = torch.zeros(1, pages, case["page"], 1, 64, dtype=torch.bfloat16,
                                   device="cuda")
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        return s
    s["q"], k = _attended(case, gen, pages, total)
    s["k_pages"] = k[None]
    s["lse"] = torch.full((total, case["q_heads"]), -math.inf, device="cuda")
    if op == "prefix":
        s["v_pages"] = _randn(gen, *s["k_pages"].shape).to(k.dtype)
        s["out"] = torch.empty_like(s["q"])
        return s
    s["v_pages"] = torch.empty_like(s["k_pages"])
    for b, rows, z in _scores(s):
        s["lse"][rows] = torch.logsumexp(z, -1).permute(2, 0, 1).flatten(1)
        del z
    s["weights"] = torch.exp(_randn(gen, len(n), max(max(lens), 1) + 5))
    s["out"] = torch.zeros_like(s["weights"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import moe_expert_ffn_dg_gb300 as pkg
    if case["op"] == "select":
        # the pools are not touched: any cache of the server will do
        pool = torch.zeros(1, 1, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
        s["cache"] = pkg.KvCache(pool, torch.zeros_like(pool))
        return s
    s["cache"] = pkg.KvCache(s["k_pages"], s["v_pages"])
    s["batch"] = pkg.KvBatch(s["table"], s["lens"], s["cu"])
    if case["op"] == "prefix":
        s["attn"] = pkg.PagedAttention(s["cache"], n_q_heads=case["q_heads"], right=0,
                                       shared_tokens=s["q"].shape[0])
        # found once a step, used in all of its layers
        s["shared"] = s["cache"].shared(s["batch"], s["groups"])
    if case["op"] == "weights":
        s["attn"] = pkg.PagedAttention(s["cache"], n_q_heads=case["q_heads"], left=case["left"],
                                       right=case["right"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "shared":
            return s["cache"].shared(s["batch"], s["groups"]).prefix
        if op == "prefix":
            return s["attn"].forward(s["q"], s["batch"], out=s["out"], lse=s["lse"],
                                     shared=s["shared"])
        if op == "weights":
            return s["attn"].weights(s["q"], s["lse"], s["batch"], s["weights"],
                                     decay=case["decay"], out=s["out"])
        f = s["cache"].select(s["weights"], s["lens"], case["budget"], first=case["first"],
                              last=case["last"])
        return {"keep": f.keep, "cu": f.cu, "lens": f.lens, "weights": f.weights}
    return {"shared": _plain_shared, "prefix": _plain_prefix, "weights": _plain_weights,
            "select": _plain_select}[op](s)


def _plain_shared(s):
    page, n = s["case"]["page"], s["lens"].shape[0]
    table, groups = s["table"], s["groups"].long()
    seq = torch.arange(n, device="cuda")
    g = torch.searchsorted(groups[1:], seq, right=True)
    first = groups[g]
    same = torch.cumprod((table == table[first]).int(), 1).sum(1) * page
    past = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).clamp(min=0)
    least = torch.full((groups.shape[0] - 1,), 1 << 30, dtype=torch.long, device="cuda")
    least.scatter_reduce_(0, g, torch.minimum(same, past.long()), "amin")
    alone = (groups[1:] - groups[:-1])[g] < 2
    return torch.where(alone, 0, least[g]).int()


def _scores(s):
    """Scaled scores of the sequences that have new tokens, one at a time,
    [kv_heads, group, tokens, keys], -inf where a token does not look."""
    case = s["case"]
    n, lens, _, _ = _chunks(case)
    kvh, d = case["kv_heads"], case["dim"]
    group, page, at = case["q_heads"] // kvh, case["page"], 0
    for b, (nb, kb) in enumerate(zip(n, lens)):
        if nb and kb:
            rows = s["table"][b, :-(-kb // page)].long()
            i = torch.arange(nb, device="cuda")[:, None] + (kb - nb)
            j = torch.arange(kb, device="cuda")[None]
            left, right = case.get("left", -1), case.get("right", 0)
            hide = torch.zeros(nb, kb, dtype=torch.bool, device="cuda")
            if left >= 0:
                hide |= j < i - left
            if right >= 0:
                hide |= j > i + right
            k = s["k_pages"][0, rows].flatten(0, 1)[:kb].float().transpose(0, 1)
            q = s["q"][at:at + nb].float().view(nb, kvh, group, d).permute(1, 2, 0, 3)
            z = (q.reshape(kvh, group * nb, d) @ k.mT).view(kvh, group, nb, kb)
            z *= 1.0 / math.sqrt(d)
            yield b, slice(at, at + nb), z.masked_fill_(hide, -math.inf)
        at += nb


def _plain_prefix(s):
    case = s["case"]
    _, lens, _, _ = _chunks(case)
    kvh, d, page = case["kv_heads"], case["dim"], case["page"]
    for b, rows, z in _scores(s):
        pages = s["table"][b, :-(-lens[b] // page)].long()
        v = s["v_pages"][0, pages].flatten(0, 1)[:lens[b]].float().transpose(0, 1)
        top = z.amax(-1, keepdim=True)
        z = torch.exp(z - top)
        l = z.sum(-1, keepdim=True)
        o = (z.flatten(1, 2) @ v).view(*z.shape[:3], d) / l
        s["out"][rows] = o.permute(2, 0, 1, 3).flatten(1, 2).to(s["out"].dtype)
        s["lse"][rows] = (top + torch.log(l)).permute(2, 0, 1, 3).flatten(1)
    return s["out"], s["lse"]


def _plain_weights(s):
    case = s["case"]
    n, lens, _, _ = _chunks(case)
    kvh = case["kv_heads"]
    group = case["q_heads"] // kvh
    at = torch.arange(s["weights"].shape[1], device="cuda")[None]
    old = at < (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None]
    held = at < s["lens"][:, None]
    new = torch.where(old, case["decay"] * s["weights"], 0.0)
    for b, rows, z in _scores(s):
        lse = s["lse"][rows].view(-1, kvh, group).permute(1, 2, 0)[..., None]
        # a row that sees nothing has a log-sum of -inf, and weighs nothing
        z = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse))
        new[b, :lens[b]] += z.flatten(0, 2).sum(0)
    s["out"].copy_(torch.where(held, new, s["out"]))
    return s["out"]


def _plain_select(s):
    case = s["case"]
    seqs, width = s["weights"].shape
    budget = min(case["budget"], width)
    lens = s["lens"].long()
    at = torch.arange(width, device="cuda")[None]
    # held back: behind the end; taken first: the first and last tokens
    rank = torch.where(at < lens[:, None], 1, 0)
    sure = (at < case["first"]) | (at >= lens[:, None] - case["last"])
    rank = torch.where(sure & (rank > 0), 2, rank)
    # by weight, then stably by rank: equal weights in the order of their places
    order = torch.sort(s["weights"], dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(rank.gather(1, order), dim=1, descending=True,
                                       stable=True).indices)
    count = torch.clamp(lens, max=budget)
    taken = torch.zeros(seqs, width, dtype=torch.bool, device="cuda")
    taken.scatter_(1, order, torch.arange(width, device="cuda")[None] < count[:, None])
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(count, 0)
    row, place = torch.nonzero(taken, as_tuple=True)
    keep = torch.full((seqs * budget,), -1, dtype=torch.int32, device="cuda")
    keep[:place.shape[0]] = place.int()
    weights = torch.zeros(seqs, budget, device="cuda")
    weights[row, torch.arange(place.shape[0], device="cuda") - cu[row]] = s["weights"][row, place]
    return {"keep": keep, "cu": cu, "lens": count.int(), "weights": weights}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    return {"shared": _exact_shared, "prefix": _exact_prefix, "weights": _exact_weights,
            "select": _exact_select}[case["op"]](s)


def _exact_shared(s):
    page = s["case"]["page"]
    table, cu = s["table"].cpu().numpy(), s["cu"].tolist()
    bounds = s["groups"].tolist()
    past = [x - (cu[i + 1] - cu[i]) for i, x in enumerate(s["lens"].tolist())]
    out = np.zeros(len(past), np.int64)
    for a, b in zip(bounds[:-1], bounds[1:]):
        if b - a < 2:
            continue
        differ = np.nonzero((table[a:b] != table[a]).any(0))[0]
        pages = int(differ[0]) if len(differ) else table.shape[1]
        out[a:b] = min([pages * page] + past[a:b])
    return _gpu(out)


def _places(s, b, length):
    """Rows of the pool, tokens in a line, that hold a sequence."""
    page = s["case"]["page"]
    t = torch.arange(length, device="cuda")
    return s["table"][b].long()[t // page] * page + t % page


def _too_long(case, per_pair):
    n, lens, _, _ = _chunks(case)
    return per_pair * case["dim"] * case["q_heads"] * sum(a * b for a, b in zip(n, lens)) > 8e12


def _exact_heads(s):
    """(sequence, rows, head, scores) in 64 bits, hidden ones -inf."""
    case = s["case"]
    n, lens, _, _ = _chunks(case)
    flat = (-1, case["kv_heads"], case["dim"])
    group = case["q_heads"] // case["kv_heads"]
    lo = 0
    for b in range(len(n)):
        rows = torch.arange(lo, lo + n[b], device="cuda")
        lo += n[b]
        if not n[b] or not lens[b]:
            continue
        where = _places(s, b, lens[b])
        ahead = torch.arange(lens[b], device="cuda")[None] - \
            torch.arange(lens[b] - n[b], lens[b], device="cuda")[:, None]
        hide = torch.zeros_like(ahead, dtype=torch.float64)
        if case.get("left", -1) >= 0:
            hide[ahead < -case["left"]] = -math.inf
        if case.get("right", 0) >= 0:
            hide[ahead > case.get("right", 0)] = -math.inf
        for e in range(case["q_heads"]):
            if e % group == 0:
                k = s["k_pages"][0].view(flat)[where, e // group].double()
            z = torch.matmul(s["q"][rows, e].double(), k.T).div_(case["dim"] ** 0.5)
            yield b, rows, e, z.add_(hide)


def _exact_prefix(s):
    case = s["case"]
    if _too_long(case, 4.0):
        return None
    _, lens, _, _ = _chunks(case)
    group = case["q_heads"] // case["kv_heads"]
    out = s["q"].double().zero_()
    lse = s["lse"].double()
    for b, rows, e, z in _exact_heads(s):
        v = s["v_pages"][0].view(-1, case["kv_heads"], case["dim"])[_places(s, b, lens[b]),
                                                                   e // group].double()
        t = torch.logsumexp(z, -1)
        out[rows, e] = torch.exp(z - t[:, None]) @ v
        lse[rows, e] = t
    return out, lse


def _exact_weights(s):
    case = s["case"]
    if _too_long(case, 2.0):
        return None
    n, lens, _, _ = _chunks(case)
    out = s["out"].double()
    for b in range(len(n)):
        out[b, :lens[b] - n[b]] = s["weights"][b, :lens[b] - n[b]].double() * case["decay"]
        out[b, lens[b] - n[b]:lens[b]] = 0
    for b, rows, e, z in _exact_heads(s):
        t = s["lse"][rows, e].double()
        some = t > -math.inf
        out[b, :lens[b]] += torch.exp(z[some] - t[some, None]).sum(0)
    return out


def _exact_select(s):
    case = s["case"]
    w = s["weights"].cpu().numpy()
    budget = min(case["budget"], w.shape[1])
    keep = np.full(w.shape[0] * budget, -1, np.int64)
    kept = np.zeros((w.shape[0], budget))
    cu = [0]
    for b, length in enumerate(s["lens"].tolist()):
        if length <= budget:
            some = np.arange(length)
        else:
            a, z = case["first"], length - case["last"]
            # descending weight, then ascending place
            mid = a + np.lexsort((np.arange(a, z), -w[b, a:z]))[:budget - a - case["last"]]
            some = np.concatenate([np.arange(a), np.sort(mid), np.arange(z, length)])
        keep[cu[-1]:cu[-1] + len(some)] = some
        kept[b, :len(some)] = w[b, some]
        cu.append(cu[-1] + len(some))
    return {"keep": _gpu(keep), "cu": _gpu(cu), "lens": _gpu(np.diff(cu)),
            "weights": _gpu(kept, torch.float64)}


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "select":
        rng = random.Random(case["lens"])
        lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
        out = case["seqs"] * min(case["budget"], case["width"])
        return {"bytes": 4 * sum(lens) + 8 * out + 12 * case["seqs"], "flops": 0}
    n, lens, prompt, bounds = _chunks(case)
    page = case["page"]
    if op == "shared":
        # the rows up to the first page that differs
        some = [b - a > 1 for a, b in zip(bounds[:-1], bounds[1:]) for _ in range(a, b)]
        return {"bytes": 4 * sum(p // page + 1 for p, m in zip(prompt, some) if m) + 12 * len(n),
                "flops": 0}
    row = 2 * case["kv_heads"] * case["dim"]  # bytes of a token's keys
    q = sum(n) * case["q_heads"]
    pairs = keys = 0
    for a, b in zip(n, lens):
        if not a or not b:
            continue
        i = np.arange(b - a, b)
        left, right = case.get("left", -1), case.get("right", 0)
        lo = np.maximum(0, i - left) if left >= 0 else np.zeros_like(i)
        hi = np.minimum(b - 1, i + right) if right >= 0 else np.full_like(i, b - 1)
        seen = np.maximum(0, hi - lo + 1)
        pairs += int(seen.sum())
        if seen.any():
            keys += int(hi.max() - lo[seen > 0].min() + 1)
    if op == "prefix":
        # a prompt's whole pages once for all of its sequences
        for a, b in zip(bounds[:-1], bounds[1:]):
            active = sum(1 for i in range(a, b) if n[i])
            if active > 1:
                keys -= (active - 1) * (prompt[a] // page * page)
        return {"bytes": 4 * q * case["dim"] + 2 * keys * row + 4 * q,
                "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    return {"bytes": 2 * q * case["dim"] + 4 * q + keys * row + 8 * sum(lens),
            "flops": 2 * pairs * case["q_heads"] * case["dim"]}
