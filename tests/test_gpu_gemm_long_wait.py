"""The pair GEMM when a stage early in a long tile is never filled (test hook): more stages are left in the tile than
the hand-off ring has barriers (tests/test_stage_release_model.py).  The kernel returns, the status word reads
FP4_ERR_TIMEOUT, and the next call is right."""
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
@pytest.mark.parametrize("stage", [0, 1, 7, 21])
@pytest.mark.parametrize("residual", [False, True])
def test_timeout_and_recovery(fb, fmt, stage, residual):
    import torch

    M, K, N = 512, 5120, 512
    s = synth.seeds_for(23)
    x, w = dev_bf16(synth.activation(s["x"], M, K, "outlier", gain_seed=s["gain"])), dev_bf16(synth.weight(s["w"], N, K))
    pw = fb.pack_weight(w, fmt)
    g = fb.calibrate_act_global(x)[0] if fmt == "nvfp4" else None
    res = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    call = (lambda: fb.linear_residual(x, pw, res, a_global=g)) if residual else (lambda: fb.linear(x, pw, a_global=g))
    want = call()
    assert fb.fp4_sync_status() == 0
    L = fb.lib()
    try:
        fb.fp4_set_wait_timeout_ns(2_000_000)  # 2 ms
        L.fp4bsa_test_skip_iteration(stage)
        call()
        st = fb.fp4_sync_status()
    finally:
        L.fp4bsa_test_skip_iteration(-1)
        fb.fp4_set_wait_timeout_ns(0)
    # (a pair has one tile of 20 or, beyond stage 19, no such stage)
    assert fb.fp4_status_string(st) == ("FP4_ERR_TIMEOUT" if stage < 20 else "FP4_OK")
    assert torch.equal(call(), want) and fb.fp4_sync_status() == 0
