"""The example layer: what it leaves in the cache, and its attention half
against a plain one over dense keys and values."""

import os
import sys

import pytest
import torch

import attn_ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples"))


@pytest.fixture(scope="module")
def ran():
    import moe_expert_ffn_dg_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkg.build()
    pkg.load_library()
    import canvas_layer
    out = canvas_layer.run(prompt_chunks=(40, 27), canvases=2, canvas=96, steps=2)
    torch.cuda.synchronize()
    return out


def test_state_of_the_cache(ran):
    layer, server, log, short = ran
    assert int(short) == 0
    assert server.lens.tolist() == [163, 163, 82]
    ref = server.ref.cpu()
    held = torch.zeros_like(ref)
    for row, n in zip(server.table.cpu(), server.lens.tolist()):
        held[row[:-(-n // 64)].long()] += 1
    assert torch.equal(ref, held)
    # 67 prompt tokens: the first page is shared, the second was split
    assert server.table[0, 0] == server.table[1, 0] and server.table[0, 1] != server.table[1, 1]
    for s in (server.cache, server.pager, layer.causal, layer.canvas, layer.moe):
        assert s.device_status()[0] == 0
    # the thinned copy holds every other token of the first candidate
    for pages in (server.cache.k_pages, server.cache.v_pages):
        rows = [pages[0, server.table[s].clamp(min=0).long()].flatten(0, 1) for s in (0, 2)]
        assert torch.equal(rows[1][:82], rows[0][:163:2])


def test_attention_half(ran):
    """The last canvases' attention, from the layer's own bf16 projections: the
    prompt's tokens and the canvas's, in one dense sequence each."""
    layer, server, log, _ = ran
    d, hq = 128, layer.q_heads
    hkv = server.cache.n_kv_heads
    x, batch, causal, _ = log[-1]
    got = layer.attention(x, batch, causal)          # appends the same rows again

    def qkv(t):
        return (t @ layer.w_qkv.T).view(t.shape[0], hq + 2 * hkv, d).cpu()
    prompt = torch.cat([qkv(a[0]) for a in log[:2]])
    canvases = qkv(x).split(96)
    out = []
    for c in canvases:
        seq = torch.cat([prompt, c])
        rot = attn_ref.rotate(seq[:, :hq + hkv].double(), list(range(163)), d, "half")
        k = rot[:, hq:].to(torch.bfloat16).double()
        q = rot[67:, :hq].to(torch.bfloat16).double()
        v = seq[:, hq + hkv:].double()
        g = hq // hkv
        s = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(g, 1)) * d ** -0.5
        o = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v.repeat_interleave(g, 1))
        out.append(o.reshape(96, hq * d))
    ref = torch.cat(out) @ layer.w_o.double().cpu().T
    # roundings to bf16 (2^-8 each, relative to sums of magnitudes): q and k may
    # differ by one step from these (a tie of the rotation), the weights, o, the
    # projection's output; the sums over 163 keys and 512 columns average them,
    # so the RMS of the error stays below three of them
    err = (got.double().cpu() - ref).pow(2).mean().sqrt()
    assert err <= 3 * 2.0 ** -8 * ref.pow(2).mean().sqrt(), float(err)
