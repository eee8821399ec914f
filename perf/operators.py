"""The attention half of a decoder layer next to the routed feed-forward
block: rotary positions, the append of a chunk to a paged key/value cache,
attention over that cache, and the page operations (forking, freeing and
reserving, copying, compacting).  Each case below is one call of one of them.

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
        # one decode step of four sequences: 16 query heads rotated, nothing else
        _case("rope_step", "rope", tokens=4, heads=16, dim=128, rot=128, layout="half",
              scaling="none", factor=1.0, orig_len=0, amplitude=1.0, theta=1e4, far=4096,
              grad=False, dtype="bf16"),
        # gradient of the rotation of a batch of 64 canvases (16384 tokens), half
        # of each head rotated, pairs interleaved, positions far past the trained length
        _case("rope_grad_batch", "rope", tokens=16384, heads=24, dim=256, rot=128,
              layout="interleaved", scaling="ramp", factor=32.0, orig_len=8192, amplitude=1.3466,
              theta=1e6, far=262144, grad=True, dtype="fp16"),
        # one new token of each of 64 sequences enters the cache
        _case("append_step", "append", seqs=64, n_lo=1, n_hi=1, past_lo=100, past_hi=4000,
              q_heads=16, kv_heads=8, dim=128, rot=128, layout="half", page=16, layers=1,
              lens=11, dtype="fp16"),
        # 64 committed canvases of 256 tokens enter the cache at head size 256
        _case("append_canvases", "append", seqs=64, n_lo=256, n_hi=256, past_lo=0, past_hi=255,
              q_heads=16, kv_heads=8, dim=256, rot=256, layout="half", page=64, layers=1,
              lens=12, dtype="bf16"),
        # one token of one short conversation: latency
        _case("attn_one_token", "attn", seqs=1, n_lo=1, n_hi=1, past_lo=776, past_hi=776,
              q_heads=16, kv_heads=4, dim=64, page=16, left=-1, right=0, lens=13, dtype="fp16"),
        # a serving step: one token each of 64 ragged sequences
        _case("attn_step_batch", "attn", seqs=64, n_lo=1, n_hi=1, past_lo=1000, past_hi=16000,
              q_heads=32, kv_heads=8, dim=128, page=64, left=-1, right=0, lens=14, dtype="bf16"),
        # one denoise step: 8 canvases of 256 tokens, every token sees its whole
        # prompt and canvas
        _case("attn_canvases", "attn", seqs=8, n_lo=256, n_hi=256, past_lo=500, past_hi=8000,
              q_heads=16, kv_heads=8, dim=256, page=64, left=-1, right=-1, lens=15,
              dtype="bf16"),
        # a long prompt taken in chunks: 4096 new tokens behind 12288 cached ones
        _case("attn_long_chunk", "attn", seqs=1, n_lo=4096, n_hi=4096, past_lo=12288,
              past_hi=12288, q_heads=32, kv_heads=8, dim=128, page=128, left=-1, right=0,
              lens=16, dtype="bf16"),
        # bookkeeping of a small step: 8 sequences, two forked, one dropped
        _case("fork_small", "fork", slots=8, new_slots=9, row=64, page=16, pages=1000,
              len_hi=900, grow_hi=40, mix=21),
        # beam reordering and growth of a full server
        _case("fork_server", "fork", slots=512, new_slots=512, row=512, page=64, pages=262144,
              len_hi=30000, grow_hi=300, mix=22),
        # the pages that a fork split, copied in all 30 layers
        _case("copy_split_pages", "copy", pairs=64, page=64, kv_heads=8, dim=128, layers=30,
              pages=192, mix=23, dtype="bf16"),
        # caches thinned to about half of their tokens, into fresh pages
        _case("compact_half", "gather", seqs=16, src_lo=1000, src_hi=6000, keep=0.5, page=32,
              kv_heads=8, dim=128, layers=4, mix=24, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "fork", "copy", "gather"])
    dt = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        scaling = rng.choice(["none", "linear", "base", "ramp"])
        rot = rng.choice([dim, dim // 2, dim // 4, 6, dim - 2])
        tokens = _log_int(rng, 1, 16000)
        return dict(op=op, tokens=tokens, heads=rng.randint(1, 24), dim=dim, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                    factor=rng.choice([2.0, 8.0, 32.0]), orig_len=8192,
                    amplitude=rng.choice([1.0, 1.25]), theta=rng.choice([1e4, 5e5]),
                    far=rng.choice([1000, 100000, 1000000]), grad=rng.random() < 0.5, dtype=dt)
    if op == "append":
        seqs = _log_int(rng, 1, 128)
        n_hi = _log_int(rng, 1, max(1, 8192 // seqs))
        return dict(op=op, seqs=seqs, n_lo=rng.choice([0, 1]) if seqs > 8 else 1, n_hi=n_hi, past_lo=0,
                    past_hi=rng.randint(1, 1000), q_heads=kv * rng.randint(1, 6), kv_heads=kv,
                    dim=dim, rot=rng.choice([0, dim, dim // 2]),
                    layout=rng.choice(["half", "interleaved"]), page=page,
                    layers=rng.randint(1, 2), lens=rng.randrange(1 << 30), dtype=dt)
    if op == "attn":
        kind = rng.choice(["step", "canvas", "chunk"])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        if kind == "step":
            seqs, n, past = _log_int(rng, 1, 200), 1, _log_int(rng, 16, 8000)
        elif kind == "canvas":
            seqs, n, past = rng.randint(1, 8), 256, _log_int(rng, 16, 6000)
        else:
            seqs, n, past = rng.randint(1, 4), _log_int(rng, 3, 1500), _log_int(rng, 1, 8000)
        return dict(op=op, seqs=seqs, n_lo=rng.choice([n, n, max(0, n // 3)]), n_hi=n,
                    past_lo=rng.choice([0, past // 4, past]), past_hi=past, q_heads=kv * group,
                    kv_heads=kv, dim=dim, page=page,
                    left=rng.choice([-1, -1, rng.randint(0, 300), 1023]),
                    right=-1 if kind == "canvas" else rng.choice([0, 0, -1, 7]),
                    lens=rng.randrange(1 << 30), dtype=dt)
    if op == "fork":
        slots = _log_int(rng, 1, 400)
        row = _log_int(rng, 4, 400)
        return dict(op=op, slots=slots, new_slots=max(1, int(slots * rng.uniform(0.3, 1.5))),
                    row=row, page=page, pages=max(8, int(slots * row * rng.uniform(0.8, 1.5))),
                    len_hi=max(1, row * page * 3 // 4), grow_hi=max(1, row * page // 5),
                    mix=rng.randrange(1 << 30))
    if op == "copy":
        return dict(op=op, pairs=_log_int(rng, 1, 60), page=rng.choice([16, 32, 64]), kv_heads=kv,
                    dim=dim, layers=rng.randint(1, 8), pages=200, mix=rng.randrange(1 << 30),
                    dtype=dt)
    return dict(op=op, seqs=rng.randint(1, 16), src_lo=rng.choice([0, 1, 100]),
                src_hi=_log_int(rng, 100, 4000), keep=rng.uniform(0.05, 0.95), page=page,
                kv_heads=kv, dim=dim, layers=rng.randint(1, 3), mix=rng.randrange(1 << 30),
                dtype=dt)


# ------------------------------------------------------------------ inputs

def _chunks(case):
    """New tokens and total lengths of the sequences of an append or an
    attention case: a function of the case alone."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    return n, [a + b for a, b in zip(n, past)]


def _rows(lens, page, pages, gen_order):
    """A page table whose rows take the pages in the order given."""
    width = max(1, max(-(-x // page) for x in lens))
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for s, x in enumerate(lens):
        k = -(-x // page)
        table[s, :k] = gen_order[at:at + k]
        at += k
    assert at <= pages
    return table


def _gpu(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device="cuda")


def _randn(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype) \
        if math.prod(shape) < 1 << 28 else \
        torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    nrng = np.random.default_rng(seed)
    op, s = case["op"], {"case": case}
    if op == "rope":
        dt = _T[case["dtype"]]
        s["x"] = _randn(gen, case["tokens"], case["heads"], case["dim"], dtype=dt)
        s["pos"] = _gpu(nrng.integers(0, case["far"], case["tokens"]))
        s["out"] = torch.empty_like(s["x"])
    elif op in ("append", "attn"):
        dt = _T[case["dtype"]]
        n, lens = _chunks(case)
        page, kvh, d = case["page"], case["kv_heads"], case["dim"]
        used = sum(-(-x // page) for x in lens)
        pages = used + 3
        s["table"] = _gpu(_rows(lens, page, pages, nrng.permutation(pages)))
        s["lens"] = _gpu(lens)
        s["cu"] = _gpu(np.concatenate([[0], np.cumsum(n)]))
        total = sum(n)
        layers = case.get("layers", 1)
        s["k_pages"] = _randn(gen, layers, pages, page, kvh, d, dtype=dt)
        s["v_pages"] = _randn(gen, layers, pages, page, kvh, d, dtype=dt)
        s["q"] = _randn(gen, total, case["q_heads"], d, dtype=dt)
        s["q_out"] = torch.empty_like(s["q"])
        if op == "append":
            s["k"] = _randn(gen, total, kvh, d, dtype=dt)
            s["v"] = _randn(gen, total, kvh, d, dtype=dt)
        else:
            s["lse"] = torch.empty(total, case["q_heads"], device="cuda")
    elif op == "fork":
        s.update(_fork_inputs(case, seed))
    elif op == "copy":
        dt = _T[case["dtype"]]
        shape = (case["layers"], case["pages"], case["page"], case["kv_heads"], case["dim"])
        s["k_pages"] = _randn(gen, *shape, dtype=dt)
        s["v_pages"] = _randn(gen, *shape, dtype=dt)
        r = np.random.default_rng(case["mix"])
        order = nrng.permutation(case["pages"])
        # sources may repeat (a page split several ways), destinations do not;
        # every eighth row or so is empty, as rows of a fork without a split are
        half = case["pages"] // 2
        rows = np.stack([order[nrng.integers(0, half, case["pairs"])],
                         order[half:half + case["pairs"]],
                         r.integers(1, case["page"] + 1, case["pairs"])], 1)
        rows[r.random(case["pairs"]) < 0.125] = (-1, -1, 0)
        s["copies"] = _gpu(rows)
    else:
        dt = _T[case["dtype"]]
        src, keep = _kept(case)
        page = case["page"]
        pages = sum(-(-x // page) for x in src) + sum(-(-x // page) for x in keep) + 2
        order = nrng.permutation(pages)
        s["src"] = _gpu(_rows(src, page, pages, order))
        s["dst"] = _gpu(_rows(keep, page, pages, order[sum(-(-x // page) for x in src):]))
        s["cu"] = _gpu(np.concatenate([[0], np.cumsum(keep)]))
        picks = [np.sort(nrng.choice(a, b, replace=False)) for a, b in zip(src, keep) if b]
        s["keep"] = _gpu(np.concatenate(picks) if picks else np.zeros(0))
        shape = (case["layers"], pages, page, case["kv_heads"], case["dim"])
        s["k_pages"] = _randn(gen, *shape, dtype=dt)
        s["v_pages"] = _randn(gen, *shape, dtype=dt)
    return s


def _kept(case):
    r = random.Random(case["mix"])
    src = [r.randint(case["src_lo"], case["src_hi"]) for _ in range(case["seqs"])]
    return src, [int(x * case["keep"]) for x in src]


def _fork_inputs(case, seed):
    r = np.random.default_rng([case["mix"], seed])
    slots, page, row, pages = case["slots"], case["page"], case["row"], case["pages"]
    order = r.permutation(pages).tolist()
    table = np.full((slots, row), -1, np.int32)
    lens = np.zeros(slots, np.int32)
    at = 0
    for j in range(slots):
        x = int(r.integers(0, case["len_hi"] + 1))
        k = -(-x // page)
        first = 0
        how = r.random()
        if j and how < 0.3:
            # the same beginning as the sequence before: whole pages shared
            first = min(int(lens[j - 1]) // page, k, int(r.integers(0, row)))
            table[j, :first] = table[j - 1, :first]
        elif j and how < 0.4:
            # a copy of the sequence before, its last page shared too
            x, k = int(lens[j - 1]), -(-int(lens[j - 1]) // page)
            first = k
            table[j, :k] = table[j - 1, :k]
        take = min(k - first, len(order) - at)
        k = first + take
        x = min(x, k * page)
        table[j, first:k] = order[at:at + take]
        table[j, k:] = -1
        lens[j] = x
        at += take
    held = [table[j, :-(-int(lens[j]) // page)] for j in range(slots)]
    ref = np.bincount(np.concatenate(held), minlength=pages).astype(np.int32)
    ref[r.integers(0, pages, max(1, pages // 200))] += 1     # pinned elsewhere
    n = case["new_slots"]
    parent = np.where(r.random(n) < 0.6, np.arange(n) % slots, r.integers(0, slots, n))
    parent[r.random(n) < 0.1] = -1                            # new conversations
    grow = r.integers(0, case["grow_hi"] + 1, n)
    grow[r.random(n) < 0.1] = 0
    have = np.where(parent >= 0, lens[np.maximum(parent, 0)], 0)
    grow = np.minimum(grow, row * page - have)
    return {"table": _gpu(table), "lens": _gpu(lens), "ref": _gpu(ref), "parent": _gpu(parent),
            "grow": _gpu(grow)}


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import moe_expert_ffn_dg_gb300 as pkg
    op = case["op"]
    if op == "rope" or (op == "append" and case["rot"]):
        s["rope"] = _rope(pkg, case)
    if op in ("append", "attn", "copy", "gather"):
        s["cache"] = pkg.KvCache(s["k_pages"], s["v_pages"])
    if op in ("append", "attn"):
        s["batch"] = pkg.KvBatch(s["table"], s["lens"], s["cu"])
    if op == "attn":
        s["attn"] = pkg.PagedAttention(s["cache"], n_q_heads=case["q_heads"], left=case["left"],
                                       right=case["right"])
    if op == "fork":
        s["pager"] = pkg.KvPager(n_pages=case["pages"], page_size=case["page"], device="cuda")
    return s


def _rope(pkg, case):
    return pkg.Rope(case["dim"], rot_dim=case["rot"], layout=case["layout"],
                    theta=case.get("theta", 1e4), scaling=case.get("scaling", "none"),
                    factor=case.get("factor", 1.0), orig_len=case.get("orig_len", 0),
                    amplitude=case.get("amplitude", 1.0))


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "rope":
            return s["rope"].apply(s["x"], s["pos"], out=s["out"], grad=case["grad"])
        if op == "append":
            last = case["layers"] - 1
            q = s["cache"].append(s["k"], s["v"], s["batch"], layer=last, q=s["q"],
                                  rope=s.get("rope"), q_out=s["q_out"])
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if op == "attn":
            return s["attn"].forward(s["q"], s["batch"], out=s["q_out"], lse=s["lse"])
        if op == "fork":
            f = s["pager"].fork(s["table"], s["lens"], s["ref"], s["parent"], s["grow"])
            return {"table": f.table, "lens": f.lens, "ref": f.ref, "copies": f.copies,
                    "short": f.short}
        if op == "copy":
            s["cache"].copy(s["copies"])
        else:
            s["cache"].gather(s["src"], s["dst"], s["cu"], s["keep"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return {"rope": _plain_rope_case, "append": _plain_append, "attn": _plain_attn,
            "fork": _plain_fork, "copy": _plain_copy, "gather": _plain_gather}[op](s)


def _freq(case):
    """Angular frequencies in 64 bits."""
    rot, theta, factor = case["rot"], case.get("theta", 1e4), case.get("factor", 1.0)
    scaling = case.get("scaling", "none")
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        turns = case["orig_len"] * f / (2 * math.pi)
        g = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = g * f + (1 - g) * f / factor
    return f


def _plain_rotate(x, pos, case, grad=False):
    rot = case["rot"]
    ang = pos.double()[:, None] * _freq(case)[None]     # far positions: 64-bit angles
    amp = case.get("amplitude", 1.0)
    c = (ang.cos() * amp).float()[:, None]
    si = (ang.sin() * amp).float()[:, None]
    if grad:
        si = -si
    f = x.float()
    if case["layout"] == "half":
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        y = torch.cat([a * c - b * si, b * c + a * si, f[..., rot:]], -1)
    else:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        y = torch.cat([torch.stack([a * c - b * si, b * c + a * si], -1).flatten(-2),
                       f[..., rot:]], -1)
    return y.to(x.dtype)


def _plain_rope_case(s):
    return _plain_rotate(s["x"], s["pos"], s["case"], s["case"]["grad"])


def _where(s, total):
    """Sequence and cache position of every new token."""
    tok = torch.arange(total, device="cuda")
    cu, lens = s["cu"].long(), s["lens"].long()
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return seq, lens[seq] - (cu[seq + 1] - tok)


def _plain_append(s):
    case = s["case"]
    q, k = s["q"], s["k"]
    seq, pos = _where(s, q.shape[0])
    if case["rot"]:
        q, k = _plain_rotate(q, pos, case), _plain_rotate(k, pos, case)
    page = s["table"].long()[seq, pos // case["page"]]
    last = case["layers"] - 1
    s["k_pages"][last, page, pos % case["page"]] = k
    s["v_pages"][last, page, pos % case["page"]] = s["v"]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attn(s):
    case = s["case"]
    n, lens = _chunks(case)
    page, kvh, d = case["page"], case["kv_heads"], case["dim"]
    group = case["q_heads"] // kvh
    out = torch.zeros_like(s["q"])
    lse = torch.full((s["q"].shape[0], case["q_heads"]), -math.inf, device="cuda")
    at = 0
    for b, (nb, kb) in enumerate(zip(n, lens)):
        if nb and kb:
            rows = s["table"][b, :-(-kb // page)].long()
            i = torch.arange(nb, device="cuda")[:, None] + (kb - nb)
            j = torch.arange(kb, device="cuda")[None]
            seen = torch.ones(nb, kb, dtype=torch.bool, device="cuda")
            if case["left"] >= 0:
                seen &= j >= i - case["left"]
            if case["right"] >= 0:
                seen &= j <= i + case["right"]
            k = s["k_pages"][0, rows].flatten(0, 1)[:kb].float().transpose(0, 1)
            v = s["v_pages"][0, rows].flatten(0, 1)[:kb].float().transpose(0, 1)
            q = s["q"][at:at + nb].float().view(nb, kvh, group, d).permute(1, 2, 0, 3)
            z = (q.reshape(kvh, group * nb, d) @ k.mT).view(kvh, group, nb, kb)
            z = torch.where(seen, z * (1.0 / math.sqrt(d)), -math.inf)
            top = z.amax(-1, keepdim=True)
            z = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            l = z.sum(-1, keepdim=True)
            o = (z.view(kvh, group * nb, kb) @ v).view(kvh, group, nb, d)
            o = o / torch.where(l == 0, 1.0, l)
            out[at:at + nb] = o.permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
            lse[at:at + nb] = (top + torch.log(l)).permute(2, 0, 1, 3).reshape(nb, -1)
        at += nb
    return out, lse


def _plain_fork(s):
    case = s["case"]
    page, pages, row = case["page"], case["pages"], case["row"]
    table, lens, parent, grow = (s[k].long() for k in ("table", "lens", "parent", "grow"))
    n = parent.shape[0]
    dev = table.device
    held = (lens + page - 1) // page
    col = torch.arange(row, device=dev)
    old = col[None] < held[:, None]
    child = torch.zeros(table.shape[0] + 1, dtype=torch.long, device=dev)
    child.scatter_add_(0, torch.where(parent >= 0, parent, table.shape[0]), torch.ones_like(parent))
    ref = torch.zeros(pages + 1, dtype=torch.long, device=dev)
    ref[:pages] = s["ref"]
    ref.scatter_add_(0, torch.where(old, table, pages).flatten(),
                     ((child[:-1, None] - 1) * old).flatten())
    have = torch.where(parent >= 0, lens[parent.clamp(min=0)], 0)
    k = (have + page - 1) // page
    base = table[parent.clamp(min=0)]
    part = (grow > 0) & (have % page != 0)
    last = torch.where(part, base.gather(1, (k - 1).clamp(min=0)[:, None])[:, 0], pages)
    j = torch.arange(n, device=dev)
    count = torch.zeros(pages + 1, dtype=torch.long, device=dev)
    count.scatter_add_(0, last, torch.ones_like(last))
    first = torch.full((pages + 1,), n, dtype=torch.long, device=dev)
    first.scatter_reduce_(0, last, j, "amin")
    split = part & ((ref[last] > count[last]) | (first[last] != j))
    want = (have + grow + page - 1) // page
    need = want - k + split
    total = need.sum()
    free = ref[:pages] == 0
    short = (total - free.sum()).clamp(min=0)
    ok = short == 0
    rank = torch.cumsum(free, 0) - 1
    order = torch.zeros(pages + 1, dtype=torch.long, device=dev)
    order.scatter_(0, torch.where(free, rank, pages), torch.arange(pages, device=dev))
    split, grow = split & ok, grow * ok
    want = torch.where(ok, want, k)
    start = torch.cumsum(need, 0) - need
    stay = k - split.long()
    fresh = order[(start[:, None] + col[None] - stay[:, None]).clamp(0, pages)]
    new = torch.where(col[None] < stay[:, None], base,
                      torch.where(col[None] < want[:, None], fresh, -1))
    ref.scatter_add_(0, last, -split.long())
    ref[:pages] += (free & (rank < total) & ok).long()
    dst = new.gather(1, (k - 1).clamp(min=0)[:, None])[:, 0]
    copies = torch.stack([torch.where(split, last, -1), torch.where(split, dst, -1),
                          torch.where(split, have % page, 0)], 1)
    return {"table": new.int(), "lens": (have + grow).int(), "ref": ref[:pages].int(),
            "copies": copies.int(), "short": short.int()[None]}


def _plain_copy(s):
    c = s["copies"].long()
    page = s["case"]["page"]
    # an empty row repeats the first one that is not
    at = torch.where(c[:, 0] >= 0, torch.arange(c.shape[0], device="cuda"),
                     torch.argmax((c[:, 0] >= 0).int()))
    c = c[at]
    t = torch.arange(page, device="cuda")
    live = (t[None] < c[:, 2:3])[None, :, :, None, None]
    src, dst = c[:, 0].clamp(min=0), c[:, 1].clamp(min=0)
    for p in (s["k_pages"], s["v_pages"]):
        p[:, dst] = torch.where(live, p[:, src], p[:, dst])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_gather(s):
    page = s["case"]["page"]
    keep, cu = s["keep"].long(), s["cu"].long()
    i = torch.arange(keep.shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], i, right=True)
    to = i - cu[seq]
    sp, dp = s["src"].long()[seq, keep // page], s["dst"].long()[seq, to // page]
    for p in (s["k_pages"], s["v_pages"]):
        p[:, dp, to % page] = p[:, sp, keep % page]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rotate(s["x"], s["pos"].cpu().numpy(), case, -1.0 if case["grad"] else 1.0)
    if op == "append":
        n, lens = _chunks(case)
        pos = np.concatenate([np.arange(k - m, k) for m, k in zip(n, lens)]).astype(np.int64)
        seq = np.repeat(np.arange(len(n)), n)
        table = s["table"].cpu().numpy()
        flat = table[seq, pos // case["page"]].astype(np.int64) * case["page"] + pos % case["page"]
        flat = torch.from_numpy(flat).cuda()
        q, k = s["q"].double(), s["k"].double()
        if case["rot"]:
            q = _exact_rotate(s["q"], pos, case, 1.0)
            k = _exact_rotate(s["k"], pos, case, 1.0)
        out = {"q": q}
        for name, new in (("k_pages", k), ("v_pages", s["v"].double())):
            pool = s[name].double()
            pool[-1].view(-1, case["kv_heads"], case["dim"])[flat] = new
            out[name] = pool
        return out
    if op == "attn":
        return _exact_attn(s)
    if op == "fork":
        return _exact_fork(s)
    pools = {k: s[k].double() for k in ("k_pages", "v_pages")}
    if op == "copy":
        for a, b, m in s["copies"].tolist():
            if a >= 0:
                for k in pools:
                    pools[k][:, b, :m] = s[k][:, a, :m].double()
        return pools
    page, cu = case["page"], s["cu"].tolist()
    src, dst = s["src"].cpu().numpy(), s["dst"].cpu().numpy()
    keep = s["keep"].cpu().numpy().astype(np.int64)
    for b in range(case["seqs"]):
        kb = keep[cu[b]:cu[b + 1]]
        at = np.arange(len(kb))
        f = torch.from_numpy(src[b, kb // page].astype(np.int64) * page + kb % page).cuda()
        t = torch.from_numpy(dst[b, at // page].astype(np.int64) * page + at % page).cuda()
        for k in pools:
            w = (case["layers"], -1, case["kv_heads"], case["dim"])
            pools[k].view(w)[:, t] = s[k].view(w)[:, f].double()
    return pools


def _exact_rotate(x, pos, case, sign):
    """The rotation as a product of complex numbers."""
    rot = case["rot"]
    theta, factor = float(case.get("theta", 1e4)), float(case.get("factor", 1.0))
    how = case.get("scaling", "none")
    if how == "base":
        theta *= factor ** (rot / (rot - 2.0))
    f = []
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        if how == "linear":
            w /= factor
        elif how == "ramp":
            turns = case["orig_len"] * w / (2.0 * math.pi)
            g = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            w = w * g + w * (1.0 - g) / factor
        f.append(w)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(f)[None]
    z = torch.from_numpy(np.exp(1j * sign * a) * case.get("amplitude", 1.0)).cuda()[:, None]
    y = x.double()
    if case["layout"] == "half":
        w = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    else:
        w = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
    return y


def _exact_attn(s):
    case = s["case"]
    n, lens = _chunks(case)
    if 4.0 * case["dim"] * case["q_heads"] * sum(a * b for a, b in zip(n, lens)) > 8e12:
        return None
    page, group = case["page"], case["q_heads"] // case["kv_heads"]
    out = s["q"].double().zero_()
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    ends = np.cumsum(n)
    for b in range(case["seqs"]):
        if not n[b] or not lens[b]:
            continue
        lo = int(ends[b]) - n[b]
        token = torch.arange(lens[b], device="cuda")
        where = s["table"][b].long()[token // page] * page + token % page
        delta = token[None] - token.new_tensor(range(lens[b] - n[b], lens[b]))[:, None]
        hide = torch.zeros_like(delta, dtype=torch.float64)
        if case["left"] >= 0:
            hide[delta < -case["left"]] = -math.inf
        if case["right"] >= 0:
            hide[delta > case["right"]] = -math.inf
        flat = (-1, case["kv_heads"], case["dim"])
        for e in range(case["q_heads"]):
            k = s["k_pages"][0].view(flat)[where, e // group].double()
            v = s["v_pages"][0].view(flat)[where, e // group].double()
            z = torch.matmul(s["q"][lo:lo + n[b], e].double(), k.T).div_(case["dim"] ** 0.5)
            z += hide
            t = torch.logsumexp(z, -1)
            some = t > -math.inf
            w = torch.exp(z[some] - t[some, None])
            rows = torch.nonzero(some)[:, 0] + lo
            out[rows, e] = w @ v
            lse[lo:lo + n[b], e] = t
    return out, lse


def _exact_fork(s):
    case = s["case"]
    page = case["page"]
    table, lens, ref, parent, grow = (s[k].cpu().numpy().astype(np.int64)
                                      for k in ("table", "lens", "ref", "parent", "grow"))
    ref = ref.copy()
    rows = []
    for j in range(table.shape[0]):
        ref[table[j, :-(-lens[j] // page)]] -= 1
    for p in parent:
        rows.append([] if p < 0 else table[p, :-(-lens[p] // page)].tolist())
        ref[rows[-1]] += 1
    have = [0 if p < 0 else int(lens[p]) for p in parent]
    users = {}
    for j, r in enumerate(rows):
        if grow[j] > 0 and have[j] % page:
            users.setdefault(r[-1], []).append(j)
    split = set()
    for p, js in users.items():
        split.update(js if ref[p] > len(js) else js[1:])
    free = np.nonzero(ref == 0)[0].tolist()
    need = [-(-(have[j] + int(grow[j])) // page) - len(r) + (j in split)
            for j, r in enumerate(rows)]
    short = max(0, sum(need) - len(free))
    copies = np.tile(np.array([-1, -1, 0], np.int64), (len(rows), 1))
    if not short:
        nxt = iter(free)
        for j, r in enumerate(rows):
            got = [next(nxt) for _ in range(need[j])]
            ref[got] += 1
            if j in split:
                copies[j] = (r[-1], got[0], have[j] % page)
                ref[r.pop()] -= 1
            r += got
            have[j] += int(grow[j])
    new = np.full((len(rows), case["row"]), -1, np.int64)
    for j, r in enumerate(rows):
        new[j, :len(r)] = r
    return {"table": _gpu(new), "lens": _gpu(have), "ref": _gpu(ref), "copies": _gpu(copies),
            "short": _gpu([short])}


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if op in ("append", "attn"):
        n, lens = _chunks(case)
        q = sum(n) * case["q_heads"] * case["dim"]
        kv = case["kv_heads"] * case["dim"]
    if op == "append":
        return {"bytes": 4 * q + 8 * sum(n) * kv,
                "flops": 3 * sum(n) * (case["q_heads"] + case["kv_heads"]) * case["rot"]}
    if op == "attn":
        keys = pairs = 0
        for a, b in zip(n, lens):
            if not a or not b:
                continue
            i = np.arange(b - a, b)
            lo = np.maximum(0, i - case["left"]) if case["left"] >= 0 else np.zeros_like(i)
            hi = np.minimum(b - 1, i + case["right"]) if case["right"] >= 0 \
                else np.full_like(i, b - 1)
            seen = np.maximum(0, hi - lo + 1)
            pairs += int(seen.sum())
            if seen.any():
                keys += int(hi.max() - lo[seen > 0].min() + 1)
        return {"bytes": 4 * q + 4 * keys * kv + 4 * sum(n) * case["q_heads"],
                "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    if op == "fork":
        # the held part of the old rows, about half of the longest; whole new rows
        cells = case["slots"] * case["len_hi"] // (2 * case["page"]) \
            + case["new_slots"] * case["row"]
        return {"bytes": 4 * (cells + 2 * case["pages"] + case["slots"] + 6 * case["new_slots"]),
                "flops": 0}
    row = 2 * 2 * case["layers"] * case["kv_heads"] * case["dim"]
    if op == "copy":
        r = np.random.default_rng(case["mix"])
        m = r.integers(1, case["page"] + 1, case["pairs"])
        m = m[r.random(case["pairs"]) >= 0.125]
        return {"bytes": 2 * row * int(m.sum()), "flops": 0}
    _, keep = _kept(case)
    return {"bytes": (2 * row + 4) * sum(keep), "flops": 0}
