"""The helpers around the attention refuse tensors in host memory before any call (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def test_host_tensors_are_refused(fb):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(4, dtype=torch.int32)
    heads = (torch.zeros(2, 128, 64, dtype=torch.uint8), torch.zeros(2, 512, dtype=torch.uint8))
    pw = fb.PackedWeight(fb.MXFP4, 128, 128, heads[0], heads[1])
    for call in (lambda: fb.rope_table(i32[:, None].contiguous(), [128]), lambda: fb.qk_norm_rope(x, x),
                 lambda: fb.qk_norm_rope_quantize_heads(x), lambda: fb.dequantize_heads(heads, 4),
                 lambda: fb.attn_ranges(i32, i32, 4, 4), lambda: fb.attn_bf16(x, x, x, 0.1),
                 lambda: fb.linear_residual(torch.zeros(4, 128, dtype=torch.bfloat16), pw)):
        with pytest.raises(ValueError):
            call()
