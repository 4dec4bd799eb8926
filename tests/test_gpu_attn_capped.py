"""Capped scores of the bf16 attention: a row's bits depend on its own visible keys alone, whatever masked
keys, other rows and rows that were never loaded hold; and the cap's error is relative to the capped score.

Tolerance of a capped score s' = cap tanh(s / cap): the score itself, s = scale q.k from exact products
summed in fp32, is off by at most 2^-23 (log2 D + 3) scale sum |q k| (and tanh has a slope of at most 1); the
polynomial is within 2^-20.6 of its value and the form for |s| > cap, 1 - 2 / (1 + 2^y), within 2^-21 absolute
where its value is 0.76 and more; products and roundings after that add 3 2^-24: 2^-20 of |s'| in all."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def randn(seed, *shape, scale=1.0):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def check(o, lse, q, k, v, scale, cap, end=None):
    """Against 64 bits, head by head, with the tolerance above."""
    import torch

    T_q, H, D = q.shape
    T_kv, H_kv, _ = k.shape
    seen = torch.ones(T_q, T_kv, dtype=torch.bool, device="cuda")
    if end is not None:
        seen &= torch.arange(T_kv, device="cuda") < end[:, None]
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h * H_kv // H].double(), v[:, h * H_kv // H].double()
        s = cap * torch.tanh(qh @ kh.t() * scale / cap)
        off = (qh.abs() @ kh.abs().t()) * scale * 2.0 ** -23 * (math.log2(D) + 3)
        off = torch.minimum(off, torch.full_like(off, 2 * cap)) + s.abs() * 2.0 ** -20
        s, off = torch.where(seen, s, -math.inf), torch.where(seen, off, 0.0)
        rl = torch.logsumexp(s, 1)
        p = torch.exp(s - rl[:, None])
        ref, mag = p @ vh, p @ vh.abs()
        extra = 2 * (p * off) @ vh.abs() + 2 * (p * off).sum(1, keepdim=True) * mag
        tol = 2.0 ** -8 * (1 + 2.0 ** -7) * (mag + ref.abs()) + extra + 2.0 ** -130
        err = (o[:, h].double() - ref).abs()
        assert bool((err <= tol).all()), (h, float((err / tol).max()))
        tl = (p * off).sum(1) * 2 + 2.0 ** -20 + 2.0 ** -22 * rl.abs()
        errl = (lse[:, h].double() - rl).abs()
        assert bool((errl <= tl).all()), (h, float((errl / tl).max()))


@pytest.mark.parametrize("T_q,T_kv,H", [(1, 900, 2), (300, 300, 2), (64, 700, 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e4, -3.3e38])
def test_masked_keys_hold_anything(fb, T_q, T_kv, H, bad):
    import torch

    D, cap = 128, 30.0
    q, k, v = randn(1, T_q, H, D), randn(2, T_kv, H, D), randn(3, T_kv, H, D)
    edge = T_kv // 2 + 5
    end = torch.full((T_q,), edge, dtype=torch.int32, device="cuda")
    clean, lse = fb.attn_bf16(q, k, v, 0.1, softcap=cap, key_end=end, return_lse=True)
    k[edge:], v[edge:] = bad, bad
    o, l2 = fb.attn_bf16(q, k, v, 0.1, softcap=cap, key_end=end, return_lse=True)
    assert torch.equal(o, clean) and torch.equal(lse, l2)


def test_other_rows_keys(fb):
    """A key of a large score that one row in three sees changes the others' bits no more than its absence."""
    import torch

    T, H, D, cap = 300, 2, 128, 30.0
    q, k, v = randn(4, T, H, D), randn(5, T, H, D), randn(6, T, H, D)
    i = torch.arange(T, device="cuda")
    end = torch.where(i % 3 == 0, 200, 190).int()
    clean, lse = fb.attn_bf16(q, k, v, 0.1, softcap=cap, key_end=end, return_lse=True)
    k[195] = 500.0
    o, l2 = fb.attn_bf16(q, k, v, 0.1, softcap=cap, key_end=end, return_lse=True)
    rest = i % 3 != 0
    assert torch.equal(o[rest], clean[rest]) and torch.equal(lse[rest], l2[rest])
    assert not torch.equal(o[~rest], clean[~rest])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [3, 5, 7])
def test_rows_that_are_not_there(fb, g, D):
    """Where g does not divide 128 the last rows of a tile are never loaded: what an earlier call left in their
    place changes no bit."""
    import torch

    T_q, T_kv = 148 * 2 * (128 // g), 256
    q, k, v = randn(7, T_q, g, D), randn(8, T_kv, 1, D), randn(9, T_kv, 1, D)
    rows = 148 * 256
    kb = torch.ones(128, 1, D, dtype=torch.bfloat16, device="cuda")
    got = []
    for fill in (0.0, 3e4, 0.0):
        fb.attn_bf16(torch.full((rows, 1, D), fill, dtype=torch.bfloat16, device="cuda"), kb, kb, 0.1)
        got.append(fb.attn_bf16(q, k, v, 0.1, softcap=30.0, return_lse=True))
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("cap", [0.5, 30.0, 1e3, 1e5, 1e7])
@pytest.mark.parametrize("T_q,T_kv,H,H_kv,D", [(1, 3000, 6, 2, 128), (130, 700, 3, 1, 64)])
def test_small_scores_beside_large_ones(fb, cap, T_q, T_kv, H, H_kv, D):
    """Every seventh key scores far below -cap (and has no weight): the others keep their accuracy."""
    import torch

    q, k, v = randn(10, T_q, H, D), randn(11, T_kv, H_kv, D), randn(12, T_kv, H_kv, D)
    q[:, :, 0] = 1.0
    k[:, :, 0] = 0.0
    k[::7, :, 0] = -200.0 * cap
    o, lse = fb.attn_bf16(q, k, v, 0.1, softcap=cap, return_lse=True)
    check(o, lse, q, k, v, 0.1, cap)


@pytest.mark.parametrize("cap", [1e-3, 1.0, 30.0, 1e6])
def test_the_capped_score_itself(fb, cap):
    """One key: lse is the capped score.  2^-20 of it, and 2^-22 for the two factors between log2 and log units
    and the roundings around them (four of 2^-24)."""
    import torch

    T, D = 4000, 64
    q, k = torch.zeros(T, 1, D, device="cuda"), torch.zeros(1, 1, D, device="cuda")
    q[:, 0, 0] = torch.logspace(-6, 2, T, device="cuda") * cap * 8
    q[::2] *= -1
    k[0, 0, 0] = 1.0
    q, k = q.bfloat16(), k.bfloat16()
    _, lse = fb.attn_bf16(q, k, k, 0.125, softcap=cap, return_lse=True)
    ref = cap * torch.tanh(q[:, 0, 0].double() * 0.125 / cap)
    err = ((lse[:, 0].double() - ref) / ref).abs()
    assert float(err.max()) <= 2.0 ** -20 + 2.0 ** -22
