"""Rotary tables, the norm and rotation of queries and keys, and decoded FP4 heads against
their formulas in 64 bits.

Tolerances: a bf16 output is the nearest bf16 of a value whose root is within 2^-24, so it is
within 2^-8 (half a bf16 step) of the exact value, relative, plus 2^-23 for the root and its
product with the rounding.  The FP4 form has to give the head quantizer's codes bit for bit."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def make(T, H, D, seed, scale=1.0):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, H, D, generator=g, device="cuda") * scale).bfloat16()


def make_table(T, rot, seed=0, amplitude=1.0):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    a = torch.rand(T, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 2 * math.pi
    return (torch.stack([a.cos(), a.sin()], 2) * amplitude).float().reshape(T, rot)


def weights(n, seed):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    return 1 + 0.3 * torch.randn(n, generator=g, device="cuda")


def reference(x, w, eps, norm, table, layout):
    """The formula in 64 bits."""
    import torch

    T, H, D = x.shape
    y = x.double()
    if norm == "head":
        y = y / torch.sqrt((y * y).mean(2, keepdim=True) + eps)
    elif norm == "token":
        y = y / torch.sqrt((y * y).mean((1, 2), keepdim=True) + eps)
    if w is not None:
        y = y * (w.double().view(H, D) if norm == "token" else w.double())
    if table is None:
        return y
    R = table.shape[1]
    c, s = table.double().view(T, 1, R // 2, 2).unbind(3)
    i = torch.arange(R // 2, device=x.device)
    iu, iv = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + R // 2)
    out = y.clone()
    out[..., iu] = y[..., iu] * c - y[..., iv] * s
    out[..., iv] = y[..., iu] * s + y[..., iv] * c
    return out


def assert_nearest(got, ref):
    err = (got.double() - ref).abs()
    tol = ref.abs() * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133
    assert bool((err <= tol).all()), float((err / tol).max())


CASES = [
    # T, Hq, Hk, D, norm, rot, layout
    (1, 40, 40, 128, "token", 128, "interleaved"),
    (1, 3, 1, 64, "head", 64, "half"),
    (2, 1, 1, 128, "token", 16, "interleaved"),
    (129, 5, 2, 128, "head", 128, "half"),
    (300, 24, 8, 64, "token", 32, "half"),
    (777, 7, 7, 128, "none", 96, "interleaved"),
    (1000, 128, 1, 128, "token", 128, "half"),
    (5000, 40, 40, 128, "token", 128, "interleaved"),
    (64, 12, 12, 128, "head", 0, "interleaved"),
    (3000, 9, 3, 128, "none", 64, "half"),
]


@pytest.mark.parametrize("T,Hq,Hk,D,norm,rot,layout", CASES)
def test_norm_rope_matches_formula(fb, T, Hq, Hk, D, norm, rot, layout):
    q, k = make(T, Hq, D, 1, 2.0), make(T, Hk, D, 2, 0.05)
    table = make_table(T, rot, amplitude=1.2) if rot else None
    n = (lambda H: H * D) if norm == "token" else (lambda H: D)
    qw, kw = (None, None) if norm == "none" else (weights(n(Hq), 1), weights(n(Hk), 2))
    qo, ko = fb.qk_norm_rope(q, k, norm=norm, q_weight=qw, k_weight=kw, eps=1e-6, table=table, layout=layout)
    assert_nearest(qo, reference(q, qw, 1e-6, norm, table, layout))
    assert_nearest(ko, reference(k, kw, 1e-6, norm, table, layout))


def test_queries_alone_and_no_weights(fb):
    q, table = make(33, 6, 128, 3), make_table(33, 128)
    alone = fb.qk_norm_rope(q, norm="head", table=table)
    assert_nearest(alone, reference(q, None, 1e-6, "head", table, "interleaved"))


def test_strided_slices_in_place_and_neighbours(fb):
    """Q and K slices of one projection, in place: the values between them stay as they were."""
    import torch

    T, Hq, Hk, D = 257, 8, 2, 128
    qkv = make(T, Hq + 2 * Hk, D, 5)
    before = qkv.clone()
    table = make_table(T, 64)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    fb.qk_norm_rope(q, k, norm="head", table=table, layout="half", q_out=q, k_out=k)
    assert_nearest(q, reference(before[:, :Hq], None, 1e-6, "head", table, "half"))
    assert_nearest(k, reference(before[:, Hq:Hq + Hk], None, 1e-6, "head", table, "half"))
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_rounding_is_to_the_nearest_everywhere(fb):
    """Values rotated by angles that cancel, and magnitudes from tiny to large."""
    import torch

    T, H, D = 4096, 4, 128
    x = make(T, H, D, 11) * torch.logspace(-6, 6, T, device="cuda").bfloat16()[:, None, None]
    x[..., 1::2] = x[..., 0::2]
    table = torch.full((T, D), math.sqrt(0.5), device="cuda")
    out = fb.qk_norm_rope(x, norm="none", table=table)
    ref = reference(x, None, 0.0, "none", table, "interleaved")
    assert_nearest(out, ref)
    assert bool((out[..., 0::2] == 0).all())


def test_zero_rows_and_non_finite_rows_stay_apart(fb):
    """A token of zeros gives zeros; a NaN or infinity changes its own token alone."""
    import torch

    for norm in ("head", "token"):
        x = make(9, 2, 128, 13)
        x[2] = 0
        clean = fb.qk_norm_rope(x, norm=norm)
        x[4, 1, 7], x[6, 0, 100] = float("nan"), float("inf")
        got = fb.qk_norm_rope(x, norm=norm)
        rest = [t for t in range(9) if t not in (4, 6)]
        assert torch.equal(got[rest], clean[rest])
        assert bool((got[2] == 0).all())
        assert bool(got[4, 1].isnan().all()) and bool(got[6, 0, 100].isnan())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,Hq,Hk,norm,rot,layout", [
    (1, 2, 1, "head", 128, "interleaved"), (127, 3, 3, "token", 64, "half"), (128, 40, 40, "token", 128, "interleaved"),
    (1021, 6, 2, "head", 128, "half"), (260, 4, 1, "none", 0, "half"), (515, 5, 5, "head", 48, "interleaved")])
def test_quantized_heads_are_the_quantizer_s(fb, fmt, T, Hq, Hk, norm, rot, layout):
    """Codes and scales, padding included, bit for bit those of quantize_heads over the bf16 form."""
    import torch

    q, k = make(T, Hq, 128, 21), make(T, Hk, 128, 22, 3.0)
    table = make_table(T, rot) if rot else None
    n = (lambda H: H * 128) if norm == "token" else (lambda H: 128)
    qw, kw = (None, None) if norm == "none" else (weights(n(Hq), 3), weights(n(Hk), 4))
    kwargs = dict(norm=norm, q_weight=qw, k_weight=kw, table=table, layout=layout)
    g = [torch.tensor([v], device="cuda") for v in (0.002, 0.004)] if fmt == "nvfp4" else [None, None]
    bf = fb.qk_norm_rope(q, k, **kwargs)
    got = fb.qk_norm_rope_quantize_heads(q, k, fmt=fmt, g_q=g[0], g_k=g[1], **kwargs)
    for x, H, gl, (codes, sf) in zip(bf, (Hq, Hk), g, got):
        want = fb.quantize_heads(x.reshape(T, H * 128), H, fmt, gl)
        assert torch.equal(codes, want[0]) and torch.equal(sf, want[1])
    alone = fb.qk_norm_rope_quantize_heads(q, fmt=fmt, g_q=g[0], norm=norm, q_weight=qw, table=table, layout=layout)
    assert torch.equal(alone[0], got[0][0]) and torch.equal(alone[1], got[0][1])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,H", [(1, 1), (129, 3), (1000, 40)])
def test_dequantized_heads_match_the_oracle(fb, orc, fmt, T, H):
    """Every code's value times its scale: exact for MXFP4, one fp32 product and one bf16 rounding for NVFP4."""
    import numpy as np
    import torch

    x = make(T, H, 128, 31) * torch.logspace(-8, 8, T, device="cuda").bfloat16()[:, None, None]
    x[0, 0, :32] = 0
    g = torch.tensor([0.7], device="cuda") if fmt == "nvfp4" else None
    codes, sf = fb.quantize_heads(x.reshape(T, H * 128), H, fmt, g)
    rows = torch.full((T, H + 1, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    fb.dequantize_heads((codes, sf), T, fmt, g, x=rows[:, :H])
    got = rows[:, :H].float().cpu().numpy()
    assert bool((rows[:, H] == 5.0).all())
    for h in range(H):
        c = codes[h, :T].contiguous().cpu().numpy()
        s = sf[h].cpu().numpy()
        grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], np.float32)
        v = np.stack([grid[c & 15], grid[c >> 4]], 2).reshape(T, 128)
        G = 32 if fmt == "mxfp4" else 16
        apr, r, j = 128 // G // 4, np.arange(T)[:, None], np.arange(128 // G)[None]
        b = s[((r // 128) * apr + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4]
        if fmt == "mxfp4":
            d = np.ldexp(np.float32(1), b.astype(np.int32) - 127)
        else:
            d = torch.from_numpy(b.copy()).view(torch.float8_e4m3fn).float().numpy() * np.float32(0.7)
        want = torch.from_numpy(v * np.repeat(d.astype(np.float32), G, 1)).bfloat16().float().numpy()
        assert np.array_equal(got[:, h], want)


def test_quantize_dequantize_round_trip_in_the_attention(fb):
    """The FP4 attention's scores from the fused operands equal the products of the decoded heads."""
    import torch

    T, H = 200, 3
    q, k, table = make(T, H, 128, 41), make(T, H, 128, 42), make_table(T, 128)
    qh, kh = fb.qk_norm_rope_quantize_heads(q, k, norm="head", table=table)
    s = fb.attn_scores(qh, kh, T, T, 1)[:, :T]
    qd, kd = (fb.dequantize_heads(h, T)[:, 1].double() for h in (qh, kh))
    ref, mag = qd @ kd.t(), qd.abs() @ kd.abs().t()
    assert bool(((s.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 1e-5 * mag).all())


# ------------------------------------------------------------------------------- tables
@pytest.mark.parametrize("T,dims,theta,far,factor,window,amplitude", [
    (1, (2,), 10000.0, 0, 1.0, 0, 1.0), (75, (44, 42, 42), 10000.0, 0, 1.0, 0, 1.0),
    (1000, (128,), 500000.0, 1 << 22, 8.0, 8192, 1.2), (333, (64,), 10000.0, 12345, 2.5, 0, 1.0),
    (64, (256,), 1e6, (1 << 31) - 65, 1.0, 0, 1.0), (50, (0, 6), 100.0, -7, 4.0, 64, 0.5)])
def test_rope_table_matches_formula(fb, T, dims, theta, far, factor, window, amplitude):
    """Within 2^-22 of the amplitude (2^-20 beyond position 2^24)."""
    import torch

    pos = torch.stack([torch.arange(T, device="cuda") * (a + 1 if far < 1 << 24 else 1) + far for a in range(len(dims))], 1)
    got = fb.rope_table(pos.int(), dims, theta, factor, window, amplitude)
    cols = []
    for a, d in enumerate(dims):
        for j in range(d // 2):
            f = theta ** (-2.0 * j / d)
            if factor != 1.0 and window:
                border = lambda turns: d * math.log(window / (2 * math.pi * turns)) / (2 * math.log(theta))
                lo, hi = max(math.floor(border(32.0)), 0.0), min(math.ceil(border(1.0)), d - 1)
                ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                f = f * (1 - ramp) + f / factor * ramp
            elif factor != 1.0:
                f = f / factor
            angle = torch.remainder(pos[:, a].double() * f, 2 * math.pi)
            cols += [angle.cos(), angle.sin()]
    ref = torch.stack(cols, 1) * amplitude
    # the reference's own angle carries half an ulp of 2^31 f in 64 bits: 2^-22 at most
    tol = amplitude * (2.0 ** -20 + 2.0 ** -21 if far + T > 1 << 24 else 2.0 ** -22)
    assert float((got.double() - ref).abs().max()) <= tol


# ------------------------------------------------------------------------------- use
def test_capture_other_stream_and_repeat(fb):
    """Captured in a graph and replayed on new inputs; on a side stream; the same bits each time."""
    import torch

    T, H = 300, 4
    q, k, table = make(T, H, 128, 51), make(T, H, 128, 52), make_table(T, 128)
    kwargs = dict(norm="token", table=table)
    want = fb.qk_norm_rope(q, k, **kwargs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fb.qk_norm_rope(q, k, **kwargs)
    side.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.qk_norm_rope(q, k, q_out=qo, k_out=ko, **kwargs)
        heads = fb.qk_norm_rope_quantize_heads(q, k, **kwargs)
        back = fb.dequantize_heads(heads[1], T)
    q.copy_(make(T, H, 128, 53))
    graph.replay()
    torch.cuda.synchronize()
    fresh = fb.qk_norm_rope(q, k, **kwargs)
    assert torch.equal(qo, fresh[0]) and torch.equal(ko, want[1])
    assert torch.equal(heads[0][0], fb.quantize_heads(fresh[0].reshape(T, -1), H)[0])
    assert torch.equal(back, fb.dequantize_heads(fb.quantize_heads(ko.reshape(T, -1), H), T))


def test_infinities_of_unrotated_values_stay_alone(fb):
    """Without a norm, an infinity in the unrotated part changes no other value."""
    import torch

    x, table = make(40, 2, 128, 61), make_table(40, 64)
    for layout in ("interleaved", "half"):
        y = x.clone()
        y[3, 1, 70], y[3, 1, 101] = float("inf"), float("-inf")
        got, clean = (fb.qk_norm_rope(z, norm="none", table=table, layout=layout) for z in (y, x))
        clean[3, 1, 70], clean[3, 1, 101] = float("inf"), float("-inf")
        assert torch.equal(got, clean)
