"""Numbers beyond 64 bits are refused by the helpers around the attention instead of being cut on their way into the
C calls, and a gate for more rows than there are is one row."""
import pytest


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


@pytest.mark.parametrize("value", [1 << 63, (1 << 64) + 5, -(1 << 63) - 1])
def test_numbers_that_do_not_fit(fb, value):
    with pytest.raises(ValueError):
        fb._int64(value, "n")
    assert fb._int64((1 << 63) - 1, "n") == (1 << 63) - 1 and fb._int64(-(1 << 63), "n") == -(1 << 63)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [1 << 64, (1 << 64) + 5, -(1 << 64)])
def test_helpers(fb, value):
    import torch

    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: fb.attn_bf16(q, q, q, 0.1, slopes=torch.ones(2, device="cuda"), q_pos=value),
                 lambda: fb.rope_table(off[:, None].contiguous(), (64,), factor=2.0, window=value),
                 lambda: fb.attn_ranges(off, off, 4, value)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fb.FP4Error):
        fb.attn_bf16(q, q, q, 0.1, slopes=torch.ones(2, device="cuda"), q_pos=1 << 41)


@pytest.mark.gpu
@pytest.mark.parametrize("gate_rows", [300, 301, 1 << 40, (1 << 64) + 5])
def test_one_gate_row_for_all(fb, gate_rows):
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(300, 256, generator=g, device="cuda").bfloat16()
    pw = fb.pack_weight(torch.randn(128, 256, generator=g, device="cuda").bfloat16())
    gate = torch.randn(1, 128, generator=g, device="cuda")
    want = fb.linear_residual(x, pw, gate=gate.expand(300, 128).contiguous(), gate_rows=1)
    assert torch.equal(fb.linear_residual(x, pw, gate=gate, gate_rows=gate_rows), want)


@pytest.mark.gpu
def test_no_rows_at_all(fb):
    import torch

    pw = fb.pack_weight(torch.randn(128, 256, device="cuda").bfloat16())
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((ValueError, fb.FP4Error)):
        fb.linear_residual(x, pw, gate=torch.ones(1, 128, device="cuda"), gate_rows=5)
    with pytest.raises((ValueError, fb.FP4Error)):
        fb.linear_residual(x, pw)
