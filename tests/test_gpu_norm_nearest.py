"""Norm and rotation: the output is the nearest bf16 of the formula's value, bit for bit, near-ties among the
values; and the FP4 form agrees with the head quantizer where values are infinite or NaN.

The reference is the formula in 64 bits, rounded once.  Without a norm its products are exact and their sum is
rounded to 53 bits, as the kernel's: all bits are equal.  With one the kernel's root is within 2^-23 (four roundings
in a sum of eight squares, halved): bits are equal unless the value lies within that of a tie."""
import math

import pytest

from tests.test_gpu_norm_extreme_rows import assert_bits, nearest, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,norm,rot", [(700, 40, 128, "token", 128), (515, 24, 128, "head", 64), (300, 5, 64, "token", 32),
                                            (64, 3, 64, "head", 0), (1000, 7, 128, "none", 128), (33, 2, 64, "none", 48)])
def test_bits(fb, T, H, D, norm, rot, layout):
    import torch

    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    w = None if norm == "none" else 1 + 0.3 * torch.randn(H * D if norm == "token" else D, generator=g, device="cuda")
    a = torch.rand(T, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 2 * math.pi
    table = (torch.stack([a.cos(), a.sin()], 2) * 1.1).float().reshape(T, rot) if rot else None
    got = fb.qk_norm_rope(x, norm=norm, q_weight=w, eps=1e-6, table=table, layout=layout)
    assert_bits(got, reference(x, w, 1e-6, norm, table, layout), exact=norm == "none")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_near_ties(fb, layout):
    """Products x c and x s on a tie of bf16 and an fp32 step to either side of it, in every pair's place."""
    import torch

    T, H, D = 900, 2, 128
    g = torch.Generator(device="cuda").manual_seed(8)
    # odd multiples of half a bf16 step in [1, 2), moved by -1, 0 or 1 steps of fp32
    half = 1 + (2 * torch.randint(0, 128, (T, D), generator=g, device="cuda").double() + 1) * 2.0 ** -8
    table = (half + torch.randint(-1, 2, (T, D), generator=g, device="cuda").double() * 2.0 ** -23).float()
    x = torch.zeros(T, H, D, device="cuda", dtype=torch.bfloat16)
    pick = torch.randint(0, 3, (T, H, D // 2), generator=g, device="cuda")
    power = 2.0 ** torch.randint(-9, 9, (T, H, D // 2), generator=g, device="cuda").float()
    i = torch.arange(D // 2, device="cuda")
    iu, iv = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + D // 2)
    x[..., iu] = torch.where(pick != 1, power, 0.0).bfloat16()
    x[..., iv] = torch.where(pick != 0, -power, 0.0).bfloat16()
    ref = reference(x, None, 0.0, "none", table, layout)
    want, _ = nearest(ref)
    got = fb.qk_norm_rope(x, norm="none", table=table, layout=layout)
    assert bool((got == want).all())
    # with a norm of ones and a weight of a power of two: the same values again
    one = torch.ones(T, H, D, device="cuda", dtype=torch.bfloat16)
    got = fb.qk_norm_rope(one, norm="head", eps=0.0, table=table, layout=layout)
    ref = reference(one, None, 0.0, "head", table, layout)
    want, tie = nearest(ref)
    assert bool(((got == want) | tie).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("norm,rot,layout", [("none", 0, "half"), ("none", 128, "interleaved"), ("head", 128, "half"),
                                             ("token", 64, "half"), ("token", 48, "interleaved")])
def test_non_finite_values_in_fp4(fb, fmt, norm, rot, layout):
    """Infinities and NaN alone, in pairs and in whole blocks: codes and scales of the head quantizer."""
    import torch

    T, H = 260, 3
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(T, H, 128, generator=g, device="cuda").bfloat16()
    nan, inf = float("nan"), float("inf")
    x[3, 0, 5], x[4, 1, 70], x[5, 2, 127] = nan, inf, -inf
    x[6, 0, 0:32], x[7, 1, 32:64], x[8, 2, 64:128] = nan, inf, -inf
    x[9, 0, 16], x[9, 0, 17], x[10, 1, 0:128:2], x[11], x[12] = nan, inf, nan, nan, inf
    x[13, 0, 40:48], x[13, 0, 48], x[14], x[15, 1] = nan, 3.0, 0.0, 3.3e38
    a = torch.rand(T, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 2 * math.pi
    table = torch.stack([a.cos(), a.sin()], 2).float().reshape(T, rot) if rot else None
    for gv in ((0.002, 1e-30, 1e30) if fmt == "nvfp4" else (None,)):
        gl = None if gv is None else torch.tensor([gv], device="cuda")
        kw = dict(norm=norm, table=table, layout=layout)
        bf = fb.qk_norm_rope(x, **kw)
        codes, sf = fb.qk_norm_rope_quantize_heads(x, fmt=fmt, g_q=gl, **kw)
        want = fb.quantize_heads(bf.reshape(T, H * 128), H, fmt, gl)
        assert torch.equal(codes, want[0]) and torch.equal(sf, want[1]), gv
