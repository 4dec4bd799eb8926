"""Distance bias where the query stands far from the keys: distances are taken as whole numbers, and a part of
the bias that all of a row's keys share goes to its log-sum-exp alone.

Tolerance: relative to the row's largest bias (slope times its nearest key's distance, its farthest key's for
a negative slope) each bias b is off by 2^-22 |b|: the slope in log2 units, the distance and the product in fp32.
The rest is as in the tests of the attention: weights rounded to bf16 and scores in fp32."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def randn(seed, *shape):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def check(fb, q, k, v, scale, slopes, q_pos, start=None, end=None, softcap=0.0):
    import torch

    T_q, H, D = q.shape
    T_kv, H_kv, _ = k.shape
    o, lse = fb.attn_bf16(q, k, v, scale, softcap=softcap, slopes=slopes, q_pos=q_pos, key_start=start, key_end=end,
                          return_lse=True)
    key, row = torch.arange(T_kv, device="cuda"), torch.arange(T_q, device="cuda")
    seen = torch.ones(T_q, T_kv, dtype=torch.bool, device="cuda")
    if start is not None:
        seen &= key >= start[:, None]
    if end is not None:
        seen &= key < end[:, None]
    some = seen.any(1)
    dist = (row[:, None] + q_pos - key).abs()
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h * H_kv // H].double(), v[:, h * H_kv // H].double()
        slope = float(slopes[h])
        # whole numbers: the distance beyond the one whose bias is largest
        best = (torch.where(seen, dist, 1 << 60).amin(1) if slope >= 0 else torch.where(seen, dist, -1).amax(1))
        b = -slope * (dist - best[:, None]).double()
        s = qh @ kh.t() * scale
        off = (qh.abs() @ kh.abs().t()) * scale * 2.0 ** -23 * (math.log2(D) + 3)
        if softcap:
            s, off = softcap * torch.tanh(s / softcap), off + softcap * 2.0 ** -20
        s, off = s + b, off + b.abs() * 2.0 ** -22
        s, off = torch.where(seen, s, -math.inf), torch.where(seen, off, 0.0)
        rl = torch.logsumexp(s, 1)
        p = torch.where(seen & some[:, None], torch.exp(s - rl[:, None]), 0.0)
        ref, mag = p @ vh, p @ vh.abs()
        weighted = p * off
        extra = 2 * weighted @ vh.abs() + 2 * weighted.sum(1, keepdim=True) * mag
        tol = 2.0 ** -8 * (1 + 2.0 ** -7) * (mag + ref.abs()) + extra + 2.0 ** -130
        err = (o[:, h].double() - ref).abs()
        assert bool((err <= tol).all()), (h, float((err / tol).max()))
        assert bool((o[~some, h] == 0).all()) and bool((lse[~some, h] == -math.inf).all())
        want = rl - slope * best.double()
        tl = 2 * weighted.sum(1) + 2.0 ** -20 + 2.0 ** -22 * (want.abs() + rl.abs() + (slope * best.double()).abs())
        errl = (lse[:, h].double() - want).abs()[some]
        assert bool((errl <= tl[some]).all()), (h, float((errl / tl[some]).max()))


FAR = [1000, (1 << 24) + 1, (1 << 30) - 7, (1 << 39) + 12345, -(1 << 33) + 3, -100]


@pytest.mark.parametrize("q_pos", FAR)
@pytest.mark.parametrize("T_q,T_kv,H,H_kv,D", [(1, 5000, 8, 2, 128), (2, 129, 6, 2, 64), (300, 900, 4, 4, 128)])
def test_far_queries(fb, q_pos, T_q, T_kv, H, H_kv, D):
    import torch

    slopes = 2.0 ** -torch.arange(1, H + 1, device="cuda").float()
    check(fb, randn(1, T_q, H, D), randn(2, T_kv, H_kv, D), randn(3, T_kv, H_kv, D), D ** -0.5, slopes, q_pos)


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("q_pos", [2000, (1 << 26) + 5])
@pytest.mark.parametrize("T_q,T_kv", [(1, 70000), (200, 3000)])
def test_ranges_away_from_the_query(fb, T_q, T_kv, q_pos, softcap):
    """Rows whose keys end long before their own place, empty rows, slopes of both signs and of zero."""
    import torch

    H, D = 4, 128
    i = torch.arange(T_q, device="cuda")
    start, end = (i * 3 % 50).int(), (i * 5 % 40 + 45).int()  # (some empty)
    slopes = torch.tensor([0.7, 0.0, -0.3, 2.0], device="cuda")
    check(fb, randn(4, T_q, H, D), randn(5, T_kv, 2, D), randn(6, T_kv, 2, D), 0.1, slopes, q_pos, start, end, softcap)


def test_rising_bias(fb):
    """Negative slopes with the query in the midst of a long axis."""
    import torch

    slopes = torch.tensor([-0.5, -0.01], device="cuda")
    check(fb, randn(7, 3, 2, 64), randn(8, 200000, 2, 64), randn(9, 200000, 2, 64), 0.125, slopes, 90000)
