"""Activations far out: z / (1 + 2^t) is within (2 |t| + 8) 2^-23 of its value, or within |z| 2^-126 where the
reciprocal of 1 + 2^t is below the smallest normal number (it is zero there).  z is the bias alone (x = 0), and
a large gate lifts the tail into bf16's normal range; the result is rounded once, 2^-8 of it at most."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_tails(fb, act):
    import torch

    N = 1024
    z = torch.linspace(-100, 30, N).half()
    if act == "gelu_tanh":
        z = (z / 8).half()
    pw = fb.PackedWeight(fb.MXFP4, N, 128, torch.full((N, 64), 0x22, dtype=torch.uint8, device="cuda"),
                         torch.full((N * 4,), 127, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    gate = torch.full((1, N), 2.0 ** 80, device="cuda")
    y = fb.linear_residual(x, pw, bias=z.cuda(), act=act, gate=gate, gate_rows=3).double().cpu().numpy() / 2.0 ** 80
    zd = z.double().numpy()
    w = zd if act == "silu" else 2 * np.sqrt(2 / np.pi) * (zd + 0.044715 * zd ** 3)
    ref = zd / (1 + np.exp(-w))
    t = np.abs(w) / np.log(2)
    tol = np.abs(ref) * (2.0 ** -8 + (2 * t + 8) * 2.0 ** -23) + np.abs(zd) * 2.0 ** -126
    err = np.abs(y - ref)
    assert (err <= tol).all(), (zd[(err > tol).any(0)][:8], float((err / np.maximum(tol, 1e-300)).max()))
    assert (np.abs(ref) > 2.0 ** -126).sum() > N // 2
