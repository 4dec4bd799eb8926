"""The operators around the attention on a stream that the caller names: what a helper allocates
belongs to that stream, so that memory freed on return is not another tensor's while the work waits;
and weights that do not fit the call are refused before anything is launched."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


def randn(seed, *shape):
    import torch

    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)).cuda().bfloat16()


def calls(fb):
    """Name -> a call with a `stream`, from inputs that are there already; some take a workspace of their own."""
    import torch

    q, k, v = randn(1, 2, 8, 128), randn(2, 5000, 2, 128), randn(3, 5000, 2, 128)  # (split over the keys)
    x, w, res = randn(4, 300, 512), fb.pack_weight(randn(5, 256, 512), "mxfp4"), randn(6, 300, 256)
    heads = randn(7, 140, 4, 128)
    pos = torch.arange(140, dtype=torch.int32, device="cuda")[:, None]
    off = torch.tensor([0, 100, 140], dtype=torch.int32, device="cuda")
    coded = fb.qk_norm_rope_quantize_heads(heads)
    return {
        "attn_bf16": lambda s: fb.attn_bf16(q, k, v, 0.1, return_lse=True, stream=s),
        "linear_residual": lambda s: (fb.linear_residual(x, w, res, stream=s),),
        "qk_norm_rope": lambda s: fb.qk_norm_rope(heads, heads, stream=s),
        "qk_norm_rope_quantize_heads": lambda s: fb.qk_norm_rope_quantize_heads(heads, stream=s),
        "dequantize_heads": lambda s: (fb.dequantize_heads(coded, 140, stream=s),),
        "rope_table": lambda s: (fb.rope_table(pos, (128,), stream=s),),
        "attn_ranges": lambda s: fb.attn_ranges(off, off, 140, 140, causal=True, stream=s),
    }


@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("name", ["attn_bf16", "linear_residual", "qk_norm_rope", "qk_norm_rope_quantize_heads",
                                  "dequantize_heads", "rope_table", "attn_ranges"])
def test_named_stream(fb, name, as_int):
    """While the named stream is held up, the current one takes and overwrites all memory that is free."""
    import torch

    call = calls(fb)[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    got = call(side.cuda_stream if as_int else side)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 12, 1 << 16, 1 << 20, 1 << 22)
            for _ in range(12)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        # (codes and scales of padding tokens are written too)
        assert a.shape == b.shape and torch.equal(a, b)
    del junk


def test_default_stream_by_number(fb):
    import torch

    heads = randn(8, 5, 2, 64)
    assert torch.equal(fb.qk_norm_rope(heads, stream=0), fb.qk_norm_rope(heads))


def test_weights_that_do_not_fit(fb):
    import torch

    x, w = randn(9, 130, 256), fb.pack_weight(randn(10, 128, 256), "mxfp4")
    for codes, sf in ((w.codes.cpu(), w.sf), (w.codes, w.sf.cpu()), (w.codes[:64], w.sf), (w.codes, w.sf[:-16]),
                      (w.codes.view(torch.int8), w.sf)):
        with pytest.raises(ValueError):
            fb.linear_residual(x, fb.PackedWeight(w.fmt, w.N, w.K, codes, sf))
