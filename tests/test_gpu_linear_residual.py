"""The FP4 linear with activation, gate and residual in its epilogue against the 64-bit formula
over the oracle's quantized operands.

Tolerance: the accumulator is within 1e-5 sum|a w| of the exact sum (the GEMM's own criterion).
act has a slope of at most 1.13 and is evaluated within (2 |a| + 16) 2^-23 of its value (GELU; SiLU
within 8 2^-24 of its value plus z's own rounding 2^-24 |z|); the fma and its inputs add 2 2^-24 of
|gate act|; the result is rounded once to bf16: half a step is 2^-8 of it."""
import numpy as np
import pytest

import synth
from tests.gpu_helpers import dev_bf16, dev_f16, host_bf16_as_f64, sample_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def inputs(M, K, N, seed=0):
    s = synth.seeds_for(seed)
    return (synth.activation(s["x"], M, K, "outlier", gain_seed=s["gain"]), synth.weight(s["w"], N, K),
            synth.bias(s["bias"], N))


def f64(bits):
    return synth.bf16_bits_to_f32(bits).astype(np.float64)


def acts(z, act):
    """The activation and a bound on its evaluation's error."""
    if act == "gelu_tanh":
        a = -2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
        g = 0.5 * z * (1 + np.tanh(-a / 2))
        return g, (2 * np.abs(a) + 16) * 2.0 ** -23 * np.abs(g) + 2.0 ** -126 + 2.0 ** -23 * np.abs(z)
    if act == "silu":
        g = z / (1 + np.exp(-z))
        return g, (np.abs(z) + 8) * 2.0 ** -23 * np.abs(g) + 2.0 ** -23 * np.abs(z)
    return z, 2.0 ** -23 * np.abs(z)


def check(orc, fb, fmt, M, K, N, act, gate_rows, residual, bias, in_place=False, seed=0):
    import torch

    x, w, b = inputs(M, K, N, seed)
    pw = fb.pack_weight(dev_bf16(w), fmt)
    xd = dev_bf16(x)
    a_global = fb.calibrate_act_global(xd)[0] if fmt == "nvfp4" else None
    gen = torch.Generator(device="cuda").manual_seed(seed)
    res = (torch.randn(M, N, generator=gen, device="cuda") * 3).bfloat16() if residual else None
    gate = torch.randn(-(-M // gate_rows), N, generator=gen, device="cuda") if gate_rows else None
    before = res.clone() if residual else None
    y = fb.linear_residual(xd, pw, residual=res, bias=dev_f16(b) if bias else None, act=act, gate=gate,
                           gate_rows=gate_rows, a_global=a_global, y=res if in_place else None)
    assert fb.fp4_sync_status() == 0
    rows = sample_rows(M, seed=seed)
    f = orc.MX if fmt == "mxfp4" else orc.NV
    kw = {} if fmt == "mxfp4" else dict(g_a=np.float32(a_global.item()))
    Y, S = orc.fp4_linear_rows(f, x, w, b if bias else None, rows, **kw)
    g, off = acts(Y, act)
    gt = np.ones((len(rows), N)) if gate is None else gate.double().cpu().numpy()[rows // gate_rows]
    r = np.zeros((len(rows), N)) if before is None else before.double().cpu().numpy()[rows]
    ref = r + gt * g
    tol = np.abs(ref) * 2.0 ** -8 + (1 + 2.0 ** -8) * np.abs(gt) * (1.13e-5 * S + off + 2.0 ** -22 * np.abs(g))
    err = np.abs(host_bf16_as_f64(y)[rows] - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,K,N,act,gate_rows,residual,bias", [
    (1, 128, 128, "none", 0, True, True), (3, 256, 384, "silu", 1, True, False), (127, 512, 128, "gelu_tanh", 50, True, True),
    (256, 640, 512, "none", 256, False, True), (509, 1024, 640, "silu", 0, True, True),
    (700, 512, 2560, "gelu_tanh", 0, False, False), (1025, 384, 1280, "none", 300, True, True),
    (2049, 5120, 256, "none", 1 << 40, True, True)])
def test_matches_formula(orc, fb, fmt, M, K, N, act, gate_rows, residual, bias):
    check(orc, fb, fmt, M, K, N, act, gate_rows, residual, bias)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_in_place_over_many_tiles(orc, fb, fmt):
    """y = residual, more tiles than CTA pairs, ragged rows."""
    check(orc, fb, fmt, 5000, 512, 2560, "silu", 1250, True, True, in_place=True, seed=3)


def test_plain_epilogue_equals_the_linear(fb):
    """Without activation, gate and residual: the linear's result bit for bit."""
    import torch

    for fmt in ("mxfp4", "nvfp4"):
        x, w, b = inputs(900, 1024, 768, 5)
        pw, xd, bd = fb.pack_weight(dev_bf16(w), fmt), dev_bf16(x), dev_f16(b)
        g = fb.calibrate_act_global(xd)[0] if fmt == "nvfp4" else None
        assert torch.equal(fb.linear_residual(xd, pw, bias=bd, a_global=g), fb.linear(xd, pw, bd, g))


def test_pieces_equal_the_whole_and_replay(fb):
    """quantize_act and fp4_gemm_residual in sequence, and a replayed graph on new inputs, give the same bits."""
    import torch

    M, K, N = 333, 512, 640
    x, w, b = inputs(M, K, N, 7)
    pw, xd, bd = fb.pack_weight(dev_bf16(w)), dev_bf16(x), dev_f16(b)
    res = torch.randn(M, N, device="cuda").bfloat16()
    gate = torch.randn(1, N, device="cuda")
    want = fb.linear_residual(xd, pw, res, bd, "silu", gate, M)
    codes, sf = fb.quantize_act(xd)
    y = torch.empty_like(want)
    fb.fp4_gemm_residual("mxfp4", codes, sf, M, K, N, pw.codes, pw.sf, None, None, bd, "silu", gate, M, res, y)
    assert torch.equal(y, want)
    ws = torch.empty(fb.fp4_linear_workspace_bytes("mxfp4", M, K, N), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.linear_residual(xd, pw, res, bd, "silu", gate, M, y=y, workspace=ws)
    xd.copy_(xd.flip(0))
    res.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, fb.linear_residual(xd, pw, res, bd, "silu", gate, M))


def test_non_finite_residual_stays_where_it_is(fb):
    import torch

    x, w, _ = inputs(260, 256, 256, 9)
    pw, xd = fb.pack_weight(dev_bf16(w)), dev_bf16(x)
    res = torch.randn(260, 256, device="cuda").bfloat16()
    clean = fb.linear_residual(xd, pw, res)
    res[5, 7], res[259, 255] = float("nan"), float("-inf")
    got = fb.linear_residual(xd, pw, res)
    clean[5, 7], clean[259, 255] = float("nan"), float("-inf")
    assert torch.equal(got.nan_to_num(7.0), clean.nan_to_num(7.0))


def test_helper_refusals(fb):
    import torch

    x, w, _ = inputs(16, 256, 256, 11)
    pw, xd = fb.pack_weight(dev_bf16(w)), dev_bf16(x)
    for bad in (dict(residual=torch.zeros(16, 128, device="cuda", dtype=torch.bfloat16)),
                dict(residual=torch.zeros(16, 256, device="cuda")), dict(gate=torch.zeros(1, 256, device="cuda")),
                dict(gate=torch.zeros(2, 256, device="cuda"), gate_rows=16),
                dict(bias=torch.zeros(256, device="cuda")), dict(y=torch.zeros(16, 256).bfloat16())):
        with pytest.raises(ValueError):
            fb.linear_residual(xd, pw, **bad)
