"""The gated residual GEMM when its bounded waits run out: a stage that is never filled (test hook), in the first
output tile of a CTA pair or in a later one, with residual copies in flight.  The kernel returns, the status word
reads FP4_ERR_TIMEOUT, and the next call is right."""
import numpy as np
import pytest

import synth
from tests.gpu_helpers import dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fb():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("stage", [0, 1, 5, 9])
def test_timeout_and_recovery(fb, fmt, stage):
    import torch

    M, K, N = 9000, 512, 2560  # two k-stages, several output tiles a CTA pair
    s = synth.seeds_for(17)
    x, w = dev_bf16(synth.activation(s["x"], M, K, "outlier", gain_seed=s["gain"])), dev_bf16(synth.weight(s["w"], N, K))
    pw = fb.pack_weight(w, fmt)
    g = fb.calibrate_act_global(x)[0] if fmt == "nvfp4" else None
    res = torch.from_numpy(np.random.default_rng(3).standard_normal((M, N), dtype=np.float32)).cuda().bfloat16()
    want = fb.linear_residual(x, pw, res, a_global=g)
    assert fb.fp4_sync_status() == 0
    L = fb.lib()
    try:
        fb.fp4_set_wait_timeout_ns(2_000_000)  # 2 ms
        L.fp4bsa_test_skip_iteration(stage)
        fb.linear_residual(x, pw, res, a_global=g)
        st = fb.fp4_sync_status()
    finally:
        L.fp4bsa_test_skip_iteration(-1)
        fb.fp4_set_wait_timeout_ns(0)
    assert fb.fp4_status_string(st) == "FP4_ERR_TIMEOUT"
    assert torch.equal(fb.linear_residual(x, pw, res, a_global=g), want) and fb.fp4_sync_status() == 0
