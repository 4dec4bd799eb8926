"""bf16 attention with key ranges, capped scores, distance bias and shared key heads against the
formula in 64 bits.

Tolerance of an output, from the arithmetic: the weights p are rounded to bf16 (2^-8 of each, one
half step 2^-9 of the value's binade: at most 2^-8 relative), their sum is not, and the output is
rounded once more (2^-8 of it): |o - ref| <= 2^-8 (sum_j p_j |v_j| / sum_j p_j + |ref|) plus the fp32
part: scores within 2^-23 (log2 D + 3) sum |q k| scale + 2^-20 cap (exp2 and the sums add less than
2^-16 of the first term), as a relative error of each weight.  lse: the scores' error and 2^-20."""
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


def reference(q, k, v, scale, softcap=0.0, slopes=None, q_pos=0, start=None, end=None):
    """Per head in 64 bits: (o, lse, tolerance of o, tolerance of lse)."""
    import torch

    T_q, H, D = q.shape
    T_kv, H_kv, _ = k.shape
    key, row = torch.arange(T_kv, device="cuda"), torch.arange(T_q, device="cuda")
    seen = torch.ones(T_q, T_kv, dtype=torch.bool, device="cuda")
    if start is not None:
        seen &= key >= start[:, None].clamp(min=0)
    if end is not None:
        seen &= key < end[:, None]
    outs = []
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h * H_kv // H].double(), v[:, h * H_kv // H].double()
        s = qh @ kh.t() * scale
        off = (qh.abs() @ kh.abs().t()) * scale * 2.0 ** -23 * (math.log2(D) + 3)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            off = off + softcap * 2.0 ** -20
        if slopes is not None:
            b = slopes[h].double() * (row[:, None] + q_pos - key).abs()
            s, off = s - b, off + b.abs() * 2.0 ** -22
        s = torch.where(seen, s, -math.inf)
        off = torch.where(seen, off, 0.0)
        lse = torch.logsumexp(s, 1)
        p = torch.where(seen, torch.exp(s - lse[:, None]), 0.0)
        some = seen.any(1)[:, None]
        p = torch.where(some, p, 0.0)
        o, mag = p @ vh, p @ vh.abs()
        extra = 2 * (p * off) @ vh.abs() + 2 * (p * off).sum(1, keepdim=True) * mag
        outs.append((o, lse, 2.0 ** -8 * (1 + 2.0 ** -7) * (mag + o.abs()) + extra + 2.0 ** -130,
                     off.amax(1) + 2.0 ** -20 + 2.0 ** -22 * torch.where(some[:, 0], lse, 0.0).abs()))
    return [torch.stack(x, 1) for x in zip(*outs)]


def check(fb, q, k, v, scale=None, **kw):
    import torch

    scale = scale or q.shape[2] ** -0.5
    o, lse = fb.attn_bf16(q, k, v, scale, return_lse=True, **kw)
    assert fb.fp4_sync_status() == 0
    ref_kw = {n: kw.get(m) for n, m in (("slopes", "slopes"), ("start", "key_start"), ("end", "key_end"))}
    ref, rl, tol, tl = reference(q, k, v, scale, kw.get("softcap", 0.0), q_pos=kw.get("q_pos", 0), **ref_kw)
    err = (o.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    errl = torch.where(empty, 0.0, lse.double() - rl).abs()
    assert bool((errl <= tl).all()), float((errl / tl).max())
    return o, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T_q,T_kv,H,H_kv", [
    (1, 1, 1, 1), (1, 127, 4, 2), (128, 128, 1, 1), (129, 130, 2, 2), (256, 384, 3, 1), (300, 1000, 5, 1), (40, 77, 24, 24),
    (7, 5000, 14, 2), (1030, 515, 2, 2), (2, 129, 128, 1)])
def test_dense(fb, T_q, T_kv, H, H_kv, D):
    check(fb, randn(1, T_q, H, D, scale=1.5), randn(2, T_kv, H_kv, D), randn(3, T_kv, H_kv, D))


@pytest.mark.parametrize("cap,bias", [(0.0, True), (30.0, False), (2.0, True)])
@pytest.mark.parametrize("T_q,T_kv,H,H_kv,D", [(1, 3000, 8, 2, 128), (260, 400, 4, 2, 64), (513, 513, 3, 3, 128)])
def test_capped_and_biased(fb, T_q, T_kv, H, H_kv, D, cap, bias):
    import torch

    slopes = 2.0 ** -torch.arange(1, H + 1, device="cuda").float() if bias else None
    check(fb, randn(4, T_q, H, D, scale=4), randn(5, T_kv, H_kv, D), randn(6, T_kv, H_kv, D), softcap=cap, slopes=slopes,
          q_pos=T_kv - T_q)


def ranges(T_q, T_kv, kind, seed=0):
    import torch

    i = torch.arange(T_q, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "causal":
        return None, (i + 1 + T_kv - T_q).int()
    if kind == "window":
        return (i + T_kv - T_q - 99).int(), (i + 1 + T_kv - T_q).int()
    if kind == "random":  # among them empty, reversed and outlying ones
        a, b = (torch.randint(-50, T_kv + 50, (T_q,), generator=g, device="cuda") for _ in "ab")
        return a.int(), b.int()
    if kind == "suffix":
        return torch.full((T_q,), T_kv // 2 + 3, device="cuda").int(), None
    if kind == "one":
        a = torch.randint(0, T_kv, (T_q,), generator=g, device="cuda").int()
        return a, a + 1
    return torch.zeros(T_q, device="cuda").int(), torch.zeros(T_q, device="cuda").int()  # empty


@pytest.mark.parametrize("kind", ["causal", "window", "random", "suffix", "one", "empty"])
@pytest.mark.parametrize("T_q,T_kv,H,H_kv,D", [(1, 2000, 4, 2, 128), (130, 130, 2, 1, 64), (700, 500, 6, 2, 128),
                                               (1000, 1500, 5, 5, 64)])
def test_ranges(fb, T_q, T_kv, H, H_kv, D, kind):
    start, end = ranges(T_q, T_kv, kind)
    check(fb, randn(7, T_q, H, D), randn(8, T_kv, H_kv, D), randn(9, T_kv, H_kv, D), key_start=start, key_end=end)


@pytest.mark.parametrize("T_q,T_kv,H", [(1, 900, 2), (300, 300, 2), (64, 700, 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3e38])
def test_masked_keys_hold_anything(fb, T_q, T_kv, H, bad):
    """Keys and values outside a row's range do not change its bits, whatever they hold; a row that
    does see an infinite value gets it."""
    import torch

    D = 128
    q, k, v = randn(10, T_q, H, D), randn(11, T_kv, H, D), randn(12, T_kv, H, D)
    edge = T_kv // 2 + 5
    i = torch.arange(T_q, device="cuda")
    end = torch.where(i % 3 == 0, edge + 20, edge).int()
    clean, lse = fb.attn_bf16(q, k, v, 0.1, key_end=end, return_lse=True)
    k2, v2 = k.clone(), v.clone()
    k2[edge + 20:], v2[edge + 20:] = bad, bad
    o, l2 = fb.attn_bf16(q, k2, v2, 0.1, key_end=end, return_lse=True)
    assert torch.equal(o, clean) and torch.equal(lse, l2)
    v2[edge + 10, H - 1, 17] = bad  # rows i % 3 == 0 see it
    o = fb.attn_bf16(q, k, torch.where(torch.arange(T_kv, device="cuda")[:, None, None] == edge + 10, v2, v), 0.1, key_end=end)
    sees = i % 3 == 0
    assert torch.equal(o[~sees], clean[~sees])
    other = torch.ones(H, D, dtype=torch.bool, device="cuda")
    other[H - 1, 17] = False
    if math.isfinite(bad):
        return
    assert torch.equal(o[sees][:, other], clean[sees][:, other])
    got = o[sees][:, H - 1, 17]
    assert bool(got.isnan().all()) if math.isnan(bad) else bool((got == bad).all())


def test_scores_of_extreme_size(fb):
    """Scores that rise by hundreds from tile to tile, and a row of equal ones."""
    import torch

    T, D = 640, 128
    q, k, v = randn(13, 200, 2, D), randn(14, T, 2, D), randn(15, T, 2, D)
    q[:, :, 0], k[:, :, 0] = 8.0, (torch.arange(T, device="cuda") * 0.5).bfloat16()[:, None]
    q[5] = 0
    check(fb, q, k, v, scale=1.0)
    check(fb, q, k.flip(0).contiguous(), v, scale=1.0)


def test_slices_strides_and_neighbours(fb):
    """Q, K, V as slices of one projection, O as rows of a wider buffer whose other values stay."""
    import torch

    T, H, Hk, D = 333, 6, 2, 64
    qkv = randn(16, T, H + 2 * Hk, D)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    wide = torch.full((T, H + 1, D), 3.0, device="cuda", dtype=torch.bfloat16)
    fb.attn_bf16(q, k, v, 0.125, o=wide[:, :H])
    want = fb.attn_bf16(q.contiguous(), k.contiguous(), v.contiguous(), 0.125)
    assert torch.equal(wide[:, :H], want) and bool((wide[:, H] == 3.0).all())


def test_split_equals_itself_and_replay(fb):
    """The split form is deterministic, its workspace need not be cleared, and it replays from a graph."""
    import torch

    q, k, v = randn(17, 1, 8, 128), randn(18, 20000, 2, 128), randn(19, 20000, 2, 128)
    ws = fb.fp4_attn_bf16_workspace_bytes(1, 20000, 8, 2, 128)
    assert ws > 0 and fb.fp4_attn_bf16_workspace_bytes(20000, 20000, 8, 2, 128) == 0
    want = fb.attn_bf16(q, k, v, 0.1)
    for fill in (0, 255):
        w = torch.full((ws,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(fb.attn_bf16(q, k, v, 0.1, workspace=w), want)
    o, graph = torch.empty_like(q), torch.cuda.CUDAGraph()
    w = torch.empty(ws, dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        fb.attn_bf16(q, k, v, 0.1, workspace=w, o=o)
    q.copy_(randn(20, 1, 8, 128))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, fb.attn_bf16(q, k, v, 0.1)) and not torch.equal(o, want)


# ------------------------------------------------------------------------------- ranges
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_off,k_off,prefix", [
    ([0, 5, 5, 12], [0, 7, 9, 9], None), ([2, 300], [3, 200], [50]), ([0, 1], [0, 1000], [0]),
    ([0, 100, 230, 300], [0, 100, 230, 300], [0, 200, 7])])
def test_attn_ranges(fb, causal, q_off, k_off, prefix):
    """Against the definition, row by row."""
    import torch

    T_q, T_kv = q_off[-1] + 3, k_off[-1] + 2
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    start, end = fb.attn_ranges(dev(q_off), dev(k_off), T_q, T_kv, causal, dev(prefix))
    for i in range(T_q):
        d = [j for j in range(len(q_off) - 1) if q_off[j] <= i < q_off[j + 1]]
        want = set()
        if d:
            j = d[0]
            place = k_off[j + 1] - (q_off[j + 1] - i)  # the row's own key
            want = {x for x in range(k_off[j], k_off[j + 1])
                    if not causal or x <= place or x < k_off[j] + (prefix[j] if prefix else 0)}
        assert set(range(int(start[i]), int(end[i]))) == want, i


def test_documents_are_apart_and_rows_behind_the_last_are_empty(fb):
    """Packed documents give what each gives by itself; rows of no document give zeros."""
    import torch

    H, D = 4, 128
    off = [0, 70, 333, 600]
    T = 650
    q, k, v = randn(21, T, H, D), randn(22, T, 2, D), randn(23, T, 2, D)
    o32 = torch.tensor(off, dtype=torch.int32, device="cuda")
    start, end = fb.attn_ranges(o32, o32, T, T, causal=True)
    v[600:], k[600:] = float("nan"), float("inf")
    o, lse = check(fb, q, k, v.nan_to_num(0.0), key_start=start, key_end=end)
    o2 = fb.attn_bf16(q, k, v, D ** -0.5, key_start=start, key_end=end)
    assert torch.equal(o, o2) and bool((o[600:] == 0).all()) and bool((lse[600:] == -math.inf).all())
    for a, b in zip(off, off[1:]):
        n = b - a
        e = torch.arange(1, n + 1, device="cuda").int()
        check(fb, q[a:b], k[a:b], v[a:b], key_end=e)


# ------------------------------------------------------------------------------- together
def test_attention_block_in_one_graph(fb):
    """Norm and rotation, FP4 and bf16 attention's operands, masked attention, gated residual projection:
    captured together, replayed on new inputs, equal to the eager calls."""
    import torch

    T, H, Hk, D = 300, 4, 2, 128
    C = H * D
    pw = fb.pack_weight(randn(30, C, C, scale=0.05))
    x, qkv = randn(31, T, C), randn(32, T, H + 2 * Hk, D)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)[:, None].contiguous()
    off = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    gate = torch.randn(1, C, device="cuda")

    def block():
        table = fb.rope_table(pos, [D])
        q, k = fb.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hk], norm="head", table=table, layout="half")
        k4 = fb.qk_norm_rope_quantize_heads(k, norm="none")
        start, end = fb.attn_ranges(off, off, T, T, causal=True)
        o = fb.attn_bf16(q, fb.dequantize_heads(k4, T), qkv[:, H + Hk:], D ** -0.5, softcap=30.0, key_start=start, key_end=end)
        return fb.linear_residual(o.view(T, C), pw, x, gate=gate, gate_rows=T)

    block()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block()
    qkv.copy_(randn(33, T, H + 2 * Hk, D))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, block())


def test_two_streams_at_once(fb):
    """Calls on two streams with their own workspaces do not disturb one another."""
    import torch

    q, k, v = randn(40, 3, 8, 128), randn(41, 9000, 2, 128), randn(42, 9000, 2, 128)
    want = [fb.attn_bf16(q, k, v, s) for s in (0.05, 0.2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(fb.attn_bf16(q, k, v, (0.05, 0.2)[n]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[n]) for n in range(2) for x in got[n])


@pytest.mark.parametrize("T_q,T_kv,H,H_kv", [(700, 300, 8, 2), (3, 5000, 8, 2), (130, 1, 3, 3)])
def test_output_over_the_queries(fb, T_q, T_kv, H, H_kv):
    import torch

    q, k, v = randn(44, T_q, H, 128), randn(45, T_kv, H_kv, 128), randn(46, T_kv, H_kv, 128)
    want = fb.attn_bf16(q, k, v, 0.1)
    assert fb.attn_bf16(q, k, v, 0.1, o=q) is q
    assert torch.equal(q, want)


def test_helper_refusals(fb):
    import torch

    q, k = randn(50, 4, 2, 64), randn(51, 5, 2, 64)
    end = torch.ones(4, dtype=torch.int32, device="cuda")
    for args, kw in (((q, k, randn(52, 6, 2, 64)), {}), ((q, k[..., :32], k), {}), ((q.float(), k, k), {}),
                     ((q, k, k), dict(key_end=end.long())), ((q, k, k), dict(key_end=end[:3])),
                     ((q, k, k), dict(slopes=torch.ones(3, device="cuda"))), ((q, k, k), dict(o=q[:3])),
                     ((q.transpose(0, 1), k, k), {}), ((q.cpu(), k, k), {}), ((q, k, k), dict(key_end=end.cpu()))):
        with pytest.raises(ValueError):
            fb.attn_bf16(*args, 0.1, **kw)
    with pytest.raises(fb.FP4Error):
        fb.attn_bf16(randn(53, 4, 3, 64), k, k, 0.1)
