"""Rotary positions against a 64-bit implementation.

Tolerance: the output is rounded once (half a step of its type, relative).
Before that, fp32: the angle is off by at most 2^-25 half turns, sincospi by 2
steps, three roundings of products and sums, the amplitude's and its product's:
together below 2^-20 of amplitude (|a| + |b|) for the pair (a, b).  The 64-bit
side's own angle p f is off by up to |p| 2^-51."""

import numpy as np
import pytest
import torch

import attn_ref

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import moe_expert_ffn_dg_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkg.build()
    pkg.load_library()


def tolerance(x, ref, positions, rot, layout, amplitude, dtype):
    i = torch.arange(rot // 2)
    lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    pair = torch.zeros_like(ref)
    both = x[..., lo].abs() + x[..., hi].abs()
    pair[..., lo], pair[..., hi] = both, both
    far = torch.tensor([abs(p) for p in positions], dtype=torch.float64)[:, None, None]
    tol = pair * amplitude * (2.0 ** -20 + far * 2.0 ** -51)
    tiny = 2.0 ** -25 if dtype == FP else 0.0
    return tol + (torch.finfo(dtype).eps / 2) * (ref.abs() + tol) + tiny


def run(t, h, d, rot, layout, dtype, positions, grad=False, strided=0, inplace=False, seed=0,
        **kw):
    import moe_expert_ffn_dg_gb300 as pkg
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=g).to(dtype)
    amplitude = kw.pop("amplitude", 1.0)
    rope = pkg.Rope(d, rot_dim=rot, layout=layout, amplitude=amplitude, **kw)
    xd = x.cuda()
    if strided:  # heads inside wider rows, off by `strided` elements
        wide = torch.zeros(t, h, d + 2 * strided, dtype=dtype, device="cuda")
        xd = wide[..., strided:strided + d]
        xd.copy_(x)
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    out = rope.apply(xd, pos, out=xd if inplace else None, grad=grad)
    torch.cuda.synchronize()
    names = {"orig_len": "orig_len", "beta_slow": "slow", "beta_fast": "fast"}
    ref = attn_ref.rotate(x.double(), positions, rot, layout, amplitude, grad,
                          **{names.get(a, a): b for a, b in kw.items()})
    err = (out.double().cpu() - ref).abs()
    tol = tolerance(x.double(), ref, positions, rot, layout, amplitude, dtype)
    assert (err <= tol).all(), float((err - tol).max())
    assert torch.equal(out[..., rot:].cpu(), x[..., rot:])
    return x, out


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 6), (80, 80), (256, 256), (96, 32),
                                   (10, 10), (512, 512), (7, 4)])
def test_heads(d, rot, layout, dtype):
    run(5, 3, d, rot, layout, dtype, [0, 1, 17, 4095, 100000])


@pytest.mark.parametrize("scaling", ["linear", "base", "ramp"])
@pytest.mark.parametrize("grad", [False, True])
def test_scaled(scaling, grad):
    kw = dict(orig_len=4096.0) if scaling == "ramp" else {}
    run(7, 2, 128, 128, "half", F32, [0, 3, 4096, 65535, 131071, 1 << 20, 5], grad,
        scaling=scaling, factor=32.0, theta=5e5, amplitude=1.25, **kw)


def test_ramp_borders():
    run(3, 2, 64, 64, "interleaved", F32, [9, 999, 70000], scaling="ramp", factor=8.0,
        orig_len=2048.0, beta_slow=0.0, beta_fast=4.0)


def test_far_and_negative_positions():
    run(6, 2, 128, 128, "half", F32, [2 ** 31 - 1, -1, -2 ** 31, -12345, 10 ** 9, 2 ** 24 + 1])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("strided", [0, 1, 8])
def test_in_place_and_strides(layout, strided):
    run(9, 5, 64, 32, layout, BF, list(range(9)), strided=strided, inplace=True)
    run(9, 5, 64, 32, layout, BF, list(range(9)), strided=strided)


@pytest.mark.parametrize("t,h,d", [(1, 1, 64), (1, 40, 256), (700, 1, 64), (3000, 2, 32),
                                   (33, 17, 48)])
def test_token_and_head_counts(t, h, d):
    rng = np.random.default_rng(t)
    run(t, h, d, d, "half", BF, rng.integers(0, 10000, t).tolist())


def test_no_tokens():
    import moe_expert_ffn_dg_gb300 as pkg
    x = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    out = pkg.Rope(64).apply(x, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert out.shape == x.shape


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_by_differences(layout):
    """The rotation is linear: <g, y(x + e) - y(x - e)> / 2 = <grad, e> up to
    fp32 rounding of the dot products (2^-18 of the sums of magnitudes)."""
    import moe_expert_ffn_dg_gb300 as pkg
    rng = torch.Generator().manual_seed(3)
    rope = pkg.Rope(64, rot_dim=48, layout=layout, amplitude=1.3)
    pos = torch.tensor([0, 7, 900, 40000], dtype=torch.int32, device="cuda")
    x, e, g = (torch.randn(4, 3, 64, generator=rng).cuda() for _ in range(3))
    dy = (rope.apply(x + e, pos).double() - rope.apply(x - e, pos).double()) / 2
    dx = rope.apply(g, pos, grad=True).double()
    a, b = (dy * g.double()).sum(), (dx * e.double()).sum()
    mag = (x.abs().double() + e.abs().double()).mul(g.abs().double()).sum() * 2.6
    assert abs(a - b) <= 2.0 ** -18 * mag


def test_gradient_undoes_a_rotation():
    import moe_expert_ffn_dg_gb300 as pkg
    rope = pkg.Rope(128)
    x = torch.randn(50, 4, 128, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    back = rope.apply(rope.apply(x, pos), pos, grad=True)
    assert (back - x).abs().max() <= 2.0 ** -18 * x.abs().max() * 2


def test_wrapper_refusals():
    import moe_expert_ffn_dg_gb300 as pkg
    rope = pkg.Rope(64)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(2, 3, 64, dtype=BF, device="cuda")
    for bad in (lambda: pkg.Rope(64, layout="other"), lambda: pkg.Rope(64, scaling="other"),
                lambda: rope.apply(x[..., :32], pos), lambda: rope.apply(x.double(), pos),
                lambda: rope.apply(x, pos.long()), lambda: rope.apply(x, pos[:1]),
                lambda: rope.apply(x, pos, out=x.float()),
                lambda: rope.apply(x.transpose(1, 2).contiguous().transpose(1, 2), pos)):
        with pytest.raises(ValueError):
            bad()
