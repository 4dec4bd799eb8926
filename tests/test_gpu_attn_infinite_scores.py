"""Rows whose visible keys all score minus infinity: the softmax is undefined, o is NaN and lse -infinity, in
one part or joined from several; keys that score so beside finite ones have no weight."""
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


@pytest.mark.parametrize("T_q,T_kv", [(1, 100), (1, 5000), (3, 129), (400, 300)])
def test_all_minus_infinity(fb, T_q, T_kv):
    import torch

    q, k, v = randn(1, T_q, 2, 128), randn(2, T_kv, 2, 128), randn(3, T_kv, 2, 128)
    q[:, :, 0] = 1.0
    k[:, 0, 0] = -math.inf  # the first head's keys
    o, lse = fb.attn_bf16(q, k, v, 0.1, return_lse=True)
    assert bool(o[:, 0].isnan().all()) and bool((lse[:, 0] == -math.inf).all())
    assert bool(o[:, 1].isfinite().all()) and bool(lse[:, 1].isfinite().all())


@pytest.mark.parametrize("T_q,T_kv", [(1, 5000), (400, 900)])
def test_some_minus_infinity(fb, T_q, T_kv):
    """The same bits as with keys that score very low; rows without any key give zeros."""
    import torch

    q, k, v = randn(4, T_q, 2, 128), randn(5, T_kv, 2, 128), randn(6, T_kv, 2, 128)
    q[:, :, 0] = 1.0
    end = torch.full((T_q,), T_kv, dtype=torch.int32, device="cuda")
    end[T_q // 2:] = 0 if T_q > 1 else T_kv
    k[: T_kv - 50, :, 0] = -1e30
    want, wl = fb.attn_bf16(q, k, v, 0.1, key_end=end, return_lse=True)
    k[: T_kv - 50, :, 0] = -math.inf
    o, lse = fb.attn_bf16(q, k, v, 0.1, key_end=end, return_lse=True)
    assert torch.equal(o, want) and torch.equal(lse, wl) and bool(o.isfinite().all())
