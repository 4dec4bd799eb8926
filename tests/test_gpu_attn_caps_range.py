"""Caps from far below the scale to far above it: the argument of the cap's tanh is formed in fp32 before its
powers are taken, so that no coefficient overflows or underflows.  Tolerance as in test_gpu_attn_capped."""
import pytest

from tests.test_gpu_attn_capped import check, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


@pytest.mark.parametrize("cap", [1e-44, 1e-30, 1e-12, 1e-6, 1e-3, 1.0, 1e6, 1e12])
@pytest.mark.parametrize("zero", [False, True])
def test_any_cap(fb, cap, zero):
    """Zero queries give the mean of the values, others the formula."""
    import torch

    q, k, v = randn(1, 100, 2, 128), randn(2, 300, 2, 128), randn(3, 300, 2, 128)
    if zero:
        q.zero_()
    q[50:] *= 1e-6
    o, lse = fb.attn_bf16(q, k, v, 128 ** -0.5, softcap=cap, return_lse=True)
    check(o, lse, q, k, v, 128 ** -0.5, cap)
    if zero:
        assert bool(((o.double() - v.double().mean(0)).abs() <= 2.0 ** -8 * v.double().abs().mean(0) * 2).all())


@pytest.mark.parametrize("scale,cap", [(0.01, 50.0), (1 / 128, 30.0), (0.1, 3e5), (1e-3, 1e3), (10.0, 0.01)])
def test_scores_near_the_cap(fb, scale, cap):
    """One key, scores from a hundredth of the cap to twice the cap: lse is the capped score (test_the_capped_score_itself)."""
    import torch

    T, D = 2000, 64
    q, k = torch.zeros(T, 1, D, device="cuda"), torch.zeros(1, 1, D, device="cuda")
    q[:, 0, 0] = torch.logspace(-2, 0.3, T, device="cuda") * (cap / scale)
    k[0, 0, 0] = 1.0
    q, k = q.bfloat16(), k.bfloat16()
    _, lse = fb.attn_bf16(q, k, k, scale, softcap=cap, return_lse=True)
    ref = cap * torch.tanh(q[:, 0, 0].double() * scale / cap)
    assert float(((lse[:, 0].double() - ref) / ref).abs().max()) <= 2.0 ** -20 + 2.0 ** -22
