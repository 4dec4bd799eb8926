"""Refusals of the operators around the attention, on the host: every invalid call returns its
status before anything is launched (the addresses are fake and never read)."""
import ctypes

import pytest

A = 1 << 20          # 16-byte aligned fake address
BAD = A + 8
ST = ctypes.c_void_p(0)
OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    import fp4_block_scaled_act_b200 as fb

    fb.build()
    return fb.lib()


def call(fn, args, **change):
    args = dict(args)
    assert set(change) <= set(args)
    args.update(change)
    return fn(*args.values(), ST)


TABLE = dict(positions=A, T=16, axes=2, dims=(ctypes.c_int64 * 4)(64, 32, 0, 0), theta=1e4, factor=1.0, window=0,
             amplitude=1.0, table=A)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(positions=None)), (INVALID, dict(table=None)), (INVALID, dict(dims=None)), (INVALID, dict(T=0)),
    (INVALID, dict(axes=0)), (INVALID, dict(axes=5)), (INVALID, dict(theta=1.0)), (INVALID, dict(theta=float("nan"))),
    (INVALID, dict(factor=0.5)), (INVALID, dict(factor=float("inf"))), (INVALID, dict(window=-1)),
    (INVALID, dict(amplitude=0.0)), (INVALID, dict(amplitude=float("nan"))), (SHAPE, dict(T=1 << 30)),
    (SHAPE, dict(dims=(ctypes.c_int64 * 4)(63, 32, 0, 0))), (SHAPE, dict(dims=(ctypes.c_int64 * 4)(-2, 32, 0, 0))),
    (SHAPE, dict(dims=(ctypes.c_int64 * 4)(256, 2, 0, 0))), (SHAPE, dict(dims=(ctypes.c_int64 * 4)(0, 0, 0, 0))),
    (SHAPE, dict(dims=(ctypes.c_int64 * 4)(1 << 62, 1 << 62, 0, 0))),
    (MISALIGNED, dict(positions=A + 2)), (MISALIGNED, dict(table=BAD))])
def test_rope_table_refuses(L, want, change):
    assert call(L.fp4_rope_table, TABLE, **change) == want


ROPE = dict(q=A, q_stride=1024, H_q=8, k=A, k_stride=256, H_k=2, T=16, D=128, norm=1, q_weight=A, k_weight=A, eps=1e-6,
            table=A, rot=128, layout=0, q_out=A, q_out_stride=1024, k_out=A, k_out_stride=256)
COMMON = [
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(T=0)), (INVALID, dict(H_q=0)),
    (INVALID, dict(H_k=-1)), (INVALID, dict(norm=3)), (INVALID, dict(norm=0)), (INVALID, dict(layout=2)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(table=None)), (INVALID, dict(rot=0)),
    (INVALID, dict(q_stride=1016)), (INVALID, dict(k_stride=0)), (SHAPE, dict(D=96)), (SHAPE, dict(rot=144)),
    (SHAPE, dict(rot=24)), (SHAPE, dict(rot=-16)), (SHAPE, dict(T=1 << 30)),
    (SHAPE, dict(H_q=129, q_stride=1 << 20, q_out_stride=1 << 20)), (SHAPE, dict(H_q=1 << 40)),
    (MISALIGNED, dict(q=BAD)), (MISALIGNED, dict(k=BAD)), (MISALIGNED, dict(q_stride=1028)),
    (MISALIGNED, dict(k_weight=A + 4)), (MISALIGNED, dict(table=A + 4))]


@pytest.mark.parametrize("want,change", COMMON + [
    (INVALID, dict(q_out=None)), (INVALID, dict(k_out=None)), (INVALID, dict(q_out_stride=512)),
    (MISALIGNED, dict(q_out=BAD)), (MISALIGNED, dict(k_out_stride=260))])
def test_norm_rope_refuses(L, want, change):
    assert call(L.fp4_qk_norm_rope, ROPE, **change) == want


QUANT = {**{"fmt": 0}, **{k: v for k, v in ROPE.items() if "_out" not in k}, **dict(
    g_q=None, g_k=None, q_codes=A, q_sf=A, k_codes=A, k_sf=A)}


@pytest.mark.parametrize("want,change", [c for c in COMMON if "q_out_stride" not in c[1]] + [
    (INVALID, dict(fmt=2)), (INVALID, dict(g_q=A)), (INVALID, dict(fmt=1)), (INVALID, dict(fmt=1, g_q=A)),
    (INVALID, dict(q_codes=None)), (INVALID, dict(k_sf=None)), (SHAPE, dict(D=64)), (SHAPE, dict(layout=1, rot=32)),
    (MISALIGNED, dict(q_sf=BAD)), (MISALIGNED, dict(fmt=1, g_q=A, g_k=A + 2))])
def test_norm_rope_quantize_heads_refuses(L, want, change):
    assert call(L.fp4_qk_norm_rope_quantize_heads, QUANT, **change) == want


DEQUANT = dict(fmt=0, codes=A, sf=A, T=16, H=8, D=128, g=None, x=A, x_stride=1024)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(fmt=3)), (INVALID, dict(codes=None)), (INVALID, dict(sf=None)), (INVALID, dict(x=None)),
    (INVALID, dict(T=0)), (INVALID, dict(H=0)), (INVALID, dict(fmt=1)), (INVALID, dict(g=A)),
    (INVALID, dict(x_stride=1016)), (SHAPE, dict(D=64)), (SHAPE, dict(T=1 << 30)),
    (SHAPE, dict(H=1 << 16, x_stride=1 << 23)), (MISALIGNED, dict(codes=BAD)),
    (MISALIGNED, dict(x=BAD)), (MISALIGNED, dict(x_stride=1028)), (MISALIGNED, dict(fmt=1, g=A + 1))])
def test_dequantize_heads_refuses(L, want, change):
    assert call(L.fp4_dequantize_heads, DEQUANT, **change) == want


GEMM = dict(fmt=0, a_codes=A, a_sf=A, M=16, K=256, N=256, w_codes=A, w_sf=A, w_global=None, a_global=None, bias=A, act=0,
            gate=A, gate_rows=16, residual=A, y=A)
RESIDUAL = [
    (INVALID, dict(fmt=2)), (INVALID, dict(w_codes=None)), (INVALID, dict(w_sf=None)), (INVALID, dict(y=None)),
    (INVALID, dict(w_global=A)), (INVALID, dict(fmt=1)), (INVALID, dict(fmt=1, w_global=A)), (INVALID, dict(act=3)),
    (INVALID, dict(gate_rows=0)), (INVALID, dict(gate=None)), (INVALID, dict(M=0)), (SHAPE, dict(K=200)),
    (SHAPE, dict(N=192)), (SHAPE, dict(M=1 << 30)), (MISALIGNED, dict(residual=BAD)), (MISALIGNED, dict(y=BAD)),
    (MISALIGNED, dict(gate=A + 4)), (MISALIGNED, dict(bias=A + 2)), (MISALIGNED, dict(w_sf=BAD))]


@pytest.mark.parametrize("want,change", RESIDUAL + [(INVALID, dict(a_codes=None)), (INVALID, dict(a_sf=None)),
                                                    (MISALIGNED, dict(a_sf=BAD))])
def test_gemm_residual_refuses(L, want, change):
    assert call(L.fp4_gemm_residual, GEMM, **change) == want


LINEAR = {("x" if k == "a_codes" else k): v for k, v in GEMM.items() if k != "a_sf"} | dict(workspace=A, ws_bytes=1 << 30)


@pytest.mark.parametrize("want,change", RESIDUAL + [(INVALID, dict(x=None)), (INVALID, dict(workspace=None)),
                                                    (WORKSPACE, dict(ws_bytes=100)), (MISALIGNED, dict(x=BAD)),
                                                    (MISALIGNED, dict(workspace=BAD))])
def test_linear_residual_refuses(L, want, change):
    assert call(L.fp4_linear_residual, LINEAR, **change) == want


ATTN = dict(q=A, q_stride=1024, T_q=16, k=A, k_stride=256, v=A, v_stride=256, T_kv=16, H=8, H_kv=2, D=128, scale=0.1,
            softcap=0.0, slopes=None, q_pos=0, key_start=None, key_end=None, o=A, o_stride=1024, lse=None, workspace=None,
            ws_bytes=0)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(o=None)),
    (INVALID, dict(T_q=0)), (INVALID, dict(T_kv=0)), (INVALID, dict(H=0)), (INVALID, dict(H_kv=0)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(softcap=-1.0)),
    (INVALID, dict(softcap=float("inf"))), (INVALID, dict(q_stride=1016)), (INVALID, dict(k_stride=128)),
    (INVALID, dict(v_stride=0)), (INVALID, dict(o_stride=8)), (INVALID, dict(q_pos=1 << 41)), (SHAPE, dict(D=96)),
    (SHAPE, dict(H=9, q_stride=4096, o_stride=4096)), (SHAPE, dict(H=258, q_stride=1 << 20, o_stride=1 << 20)),
    (SHAPE, dict(T_q=1 << 30)), (SHAPE, dict(T_kv=1 << 30)), (SHAPE, dict(k_stride=1 << 38)), (MISALIGNED, dict(q=BAD)),
    (MISALIGNED, dict(o=BAD)), (MISALIGNED, dict(v_stride=260)), (MISALIGNED, dict(lse=A + 2)),
    (MISALIGNED, dict(key_end=A + 2)), (INVALID, dict(T_kv=100000)), (WORKSPACE, dict(T_kv=100000, workspace=A)),
    (MISALIGNED, dict(T_kv=100000, workspace=BAD, ws_bytes=1 << 30))])
def test_attn_bf16_refuses(L, want, change):
    assert call(L.fp4_attn_bf16, ATTN, **change) == want


def test_attn_bf16_workspace_sizes(L):
    f = L.fp4_attn_bf16_workspace_bytes
    assert f(75600, 75600, 40, 40, 128) == 0            # the row tiles fill the device
    assert f(1, 128, 8, 8, 128) == 0                     # one key tile: one part
    # 8 key heads on 148 SMs: 18 items each, two parts an item; O parts, then (maximum, sum) pairs
    assert f(1, 100001, 40, 8, 128) == 36 * 40 * 128 * 4 + (36 * 40 * 8 + 255) // 256 * 256
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 32), (1 << 30, 1, 1, 1, 64)):
        assert f(*bad) == 0


RANGES = dict(q_offsets=A, k_offsets=A, docs=2, T_q=16, T_kv=16, causal=1, prefix=None, key_start=A, key_end=A)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(q_offsets=None)), (INVALID, dict(k_offsets=None)), (INVALID, dict(key_start=None)),
    (INVALID, dict(key_end=None)), (INVALID, dict(docs=0)), (INVALID, dict(T_q=0)), (INVALID, dict(T_kv=0)),
    (SHAPE, dict(docs=1 << 30)), (SHAPE, dict(T_q=1 << 30)), (MISALIGNED, dict(prefix=A + 1)),
    (MISALIGNED, dict(key_end=A + 2))])
def test_attn_ranges_refuses(L, want, change):
    assert call(L.fp4_attn_ranges, RANGES, **change) == want
