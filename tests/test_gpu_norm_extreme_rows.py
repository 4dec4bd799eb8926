"""The norm where eps is 0 and a row's values are small or large: its squares are taken in 64 bits where fp32
loses them, and the result is the nearest bf16 as everywhere.

Where squares are taken in fp32, a sum of eight of them carries four roundings of 2^-24, which the root halves: it
is within 2^-23.  So bits are equal unless the formula's value lies within 2^-23 of itself (2^-15 in units of a last
place of 8 bits, whose values are below 2^8) from a tie; the 64-bit reference itself is within 2^-49."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def nearest(ref):
    """(ref rounded once to bf16, True where a tie is nearer than 2^-23 of the value)."""
    import torch

    e = torch.frexp(ref)[1].clamp(min=-125)
    t = torch.ldexp(ref, 8 - e)
    tie = ((t - t.floor()) - 0.5).abs() < 2.0 ** -15
    return torch.ldexp(torch.round(t), e - 8).to(torch.bfloat16), tie


def reference(x, w, eps, norm, table, layout):
    import torch

    T, H, D = x.shape
    y = x.double()
    if norm != "none":
        dims = 2 if norm == "head" else (1, 2)
        y = y / torch.sqrt((y * y).mean(dims, keepdim=True) + eps)
    if w is not None:
        y = y * (w.double().view(H, D) if norm == "token" else w.double())
    if table is not None:
        R = table.shape[1]
        c, s = table.double().view(T, 1, R // 2, 2).unbind(3)
        i = torch.arange(R // 2, device="cuda")
        iu, iv = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + R // 2)
        u, v = y[..., iu], y[..., iv]
        y = y.clone()
        y[..., iu], y[..., iv] = u * c - v * s, u * s + v * c
    return y


def assert_bits(got, ref, exact=False):
    """Equal bits (zeros of either sign), ties apart unless `exact`."""
    import torch

    want, tie = nearest(ref)
    tie &= not exact
    nan = ref.isnan()
    wrong = (got.view(torch.int16) != want.view(torch.int16)) & ~tie & ~nan & ~((got == 0) & (want == 0))
    assert not bool(wrong.any()), (int(wrong.sum()), got[wrong][:4], ref[wrong][:4])
    assert torch.equal(got.isnan(), nan)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("norm,rot,H,D", [("head", 128, 3, 128), ("token", 128, 3, 128), ("token", 0, 2, 64), ("head", 32, 5, 64)])
def test_rows_of_any_size(fb, norm, rot, H, D, layout):
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)
    T = 240
    scale = torch.logspace(-39, 37, T, device="cuda", dtype=torch.float64)[:, None, None]
    x = (torch.randn(T, H, D, generator=g, device="cuda", dtype=torch.float64) * scale).bfloat16()
    w = 1 + 0.3 * torch.randn(H * D if norm == "token" else D, generator=g, device="cuda")
    a = torch.rand(T, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 2 * math.pi
    table = torch.stack([a.cos(), a.sin()], 2).float().reshape(T, rot) if rot else None
    got = fb.qk_norm_rope(x, norm=norm, q_weight=w, eps=0.0, table=table, layout=layout)
    assert_bits(got, reference(x, w, 0.0, norm, table, layout))


@pytest.mark.parametrize("norm", ["head", "token"])
@pytest.mark.parametrize("size", [3e-41, 1e-25, 1e-19, 1.0, 1e20, 2e38])
def test_one_value_among_zeros(fb, norm, size):
    """A row with one value, and a row of zeros beside it (0 / 0)."""
    import torch

    x = torch.zeros(3, 2, 128, device="cuda", dtype=torch.bfloat16)
    x[0, 0, 17], x[0, 1, 3], x[2, 0, 5], x[2, 1, 127] = size, -size, -size, size
    got = fb.qk_norm_rope(x, norm=norm, eps=0.0)
    assert_bits(got, reference(x, None, 0.0, norm, None, "half"))


def test_a_head_does_not_see_its_neighbours(fb):
    """A head of tiny values changes no bit of the heads beside it."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(50, 8, 64, generator=g, device="cuda").bfloat16()
    clean = fb.qk_norm_rope(x, norm="head", eps=0.0)
    x[:, 3] *= 1e-30
    got = fb.qk_norm_rope(x, norm="head", eps=0.0)
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(got[:, keep], clean[:, keep])
    assert_bits(got, reference(x, None, 0.0, "head", None, "half"))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantized_form(fb, fmt):
    """The FP4 form of such rows is the head quantizer's of the bf16 form."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(7)
    T, H = 130, 4
    x = (torch.randn(T, H, 128, generator=g, device="cuda") * torch.logspace(-35, 35, T, device="cuda")[:, None, None]).bfloat16()
    gl = torch.tensor([0.003], device="cuda") if fmt == "nvfp4" else None
    for norm in ("head", "token"):
        bf = fb.qk_norm_rope(x, norm=norm, eps=0.0)
        assert_bits(bf, reference(x, None, 0.0, norm, None, "half"))
        codes, sf = fb.qk_norm_rope_quantize_heads(x, fmt=fmt, norm=norm, eps=0.0, g_q=gl)
        want = fb.quantize_heads(bf.reshape(T, H * 128), H, fmt, gl)
        assert torch.equal(codes, want[0]) and torch.equal(sf, want[1])
