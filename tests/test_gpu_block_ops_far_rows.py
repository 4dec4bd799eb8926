"""Rows that lie further apart than 32 bits of elements reach (slots of a large cache): the same bits as
from contiguous tensors, through the attention's tensor maps, its repair of masked infinities, the norm
and the decoder, and nothing between the rows is written."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROWS, STRIDE = 70, 1 << 25  # 2.3e9 elements


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


@pytest.fixture(scope="module")
def buffer():
    import torch

    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 5 GB of device memory")
    return torch.full((ROWS * STRIDE,), 7.0, dtype=torch.bfloat16, device="cuda")


def randn(seed, *shape):
    import torch

    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)).cuda().bfloat16()


def rows(buffer, at, H, D):
    return buffer.as_strided((ROWS, H, D), (STRIDE, D, 1), at)


def test_far_rows(fb, buffer):
    import torch

    H, D = 2, 128
    k, v, q = randn(1, ROWS, H, D), randn(2, ROWS, H, D), randn(3, ROWS, H, D)
    v[68, 1, 5] = float("inf")  # seen by the last row alone
    end = torch.full((ROWS,), 68, dtype=torch.int32, device="cuda")
    end[-1] = 69
    far = {n: rows(buffer, 1024 * i, H, D) for i, n in enumerate(("k", "v", "q", "o", "n"))}
    for n, t in (("k", k), ("v", v), ("q", q)):
        far[n].copy_(t)
    want = fb.attn_bf16(q, k, v, 0.1, key_end=end)
    assert torch.isinf(want[-1, 1, 5]) and torch.isfinite(want[:-1]).all()
    fb.attn_bf16(far["q"], far["k"], far["v"], 0.1, key_end=end, o=far["o"])
    assert torch.equal(far["o"], want)

    w = torch.ones(D, device="cuda")
    assert torch.equal(fb.qk_norm_rope(far["q"], q_weight=w, q_out=far["n"]), fb.qk_norm_rope(q, q_weight=w))
    codes = fb.qk_norm_rope_quantize_heads(q, q_weight=w)
    for a, b in zip(fb.qk_norm_rope_quantize_heads(far["q"], q_weight=w), codes):
        assert torch.equal(a, b)
    assert torch.equal(fb.dequantize_heads(codes, ROWS, x=far["n"]), fb.dequantize_heads(codes, ROWS))

    # the five rows of a slot hold 5 * 1024 elements at most; what lies behind them is as it was
    for r in (0, 33, ROWS - 1):
        behind = buffer[r * STRIDE + 5 * 1024:r * STRIDE + 5 * 1024 + 65536]
        assert (behind == 7.0).all()
        for i in range(5):
            assert (buffer[r * STRIDE + 1024 * i + H * D:r * STRIDE + 1024 * (i + 1)] == 7.0).all()
