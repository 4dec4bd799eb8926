"""Cases of the attention-side operators of the framework, with their plain forms.

Six operators around the FP4 linears and the FP4 attention of a transformer block:

  rope_table   cos / sin of every position and frequency pair, one or several position axes,
               optionally scaled for long contexts;
  norm_rope    queries and keys: RMS norm over the head or the whole token, and the rotation;
  norm_quant   the same, written as head-major FP4 codes and scales, and these decoded to bf16, as for
               keys that are held in FP4 and read by attention in bf16;
  attn         bf16 attention with shared key heads, capped scores, a distance bias and one
               range of keys per query row (documents, prefixes, causal order);
  linear       the FP4 linear with bias, activation, gate and residual in its epilogue.

`run` computes them from elementary torch operations, or through the package where `own` is set.
"""
import math

import numpy as np
import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a 21 x 45 x 80 latent grid: one table for every layer and step of a video
        dict(name="rope table, video grid", op="rope_table", T=75600, grid="45x80", dims="44,42,42", theta=10000.0,
             far=0, factor=1.0, window=0),
        # a text stream continued far behind the trained length, odd length
        dict(name="rope table, far positions", op="rope_table", T=1021, grid="", dims="128", theta=500000.0,
             far=1000000, factor=8.0, window=8192),
        # Q and K of one self attention of a 40-head video transformer, norm over the token
        dict(name="norm+rope, 75600 tokens", op="norm_rope", T=75600, Hq=40, Hk=40, D=128, norm="token", rot=128,
             layout="interleaved", packed=False),
        # per-head norm, half layout, half of the head rotated, slices of one fused projection
        dict(name="norm+rope, 515 tokens", op="norm_rope", T=515, Hq=24, Hk=8, D=128, norm="head", rot=64,
             layout="half", packed=True),
        # Q and K of a 720p video (NVFP4) and of a small clip (MXFP4) as FP4 attention operands
        dict(name="norm+rope+fp4, 75600 tokens", op="norm_quant", T=75600, Hq=40, Hk=40, D=128, norm="token", rot=128,
             layout="interleaved", fmt="nvfp4"),
        dict(name="norm+rope+fp4, 4290 tokens", op="norm_quant", T=4290, Hq=24, Hk=24, D=128, norm="head", rot=128,
             layout="half", fmt="mxfp4"),
        # three clips packed on one token axis, each seeing itself
        dict(name="attn, three clips", op="attn", Tq=4290, Tk=4290, Hq=24, Hk=24, D=128, docs=3, causal=False,
             prefix=0, cap=0.0, bias=False),
        # a prefix language model: the prefix sees itself whole, the rest is causal; capped scores
        dict(name="attn, prefix, capped", op="attn", Tq=8192, Tk=8192, Hq=16, Hk=4, D=128, docs=1, causal=True,
             prefix=1000, cap=30.0, bias=False),
        # video tokens reading two prompts of text
        dict(name="attn, video to text", op="attn", Tq=32760, Tk=512, Hq=40, Hk=40, D=128, docs=2, causal=False,
             prefix=0, cap=0.0, bias=False),
        # one new token over a long cache, distance bias
        dict(name="attn, one token", op="attn", Tq=1, Tk=100001, Hq=40, Hk=8, D=128, docs=1, causal=True, prefix=0,
             cap=0.0, bias=True),
        # the attention output projection of a video transformer with its gated residual
        dict(name="linear+residual, video", op="linear", M=75600, K=5120, N=5120, fmt="mxfp4", act="none", gate=75600),
        # a short text stream through an activated projection with a plain residual
        dict(name="linear+residual, text", op="linear", M=509, K=2048, N=2560, fmt="nvfp4", act="silu", gate=0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_table", "norm_rope", "norm_quant", "attn", "attn", "linear"])
    if op == "rope_table":
        if rng.random() < 0.5:
            h, w = rng.randint(3, 60), rng.randint(3, 80)
            return dict(op=op, T=min(75600, h * w * rng.randint(1, 21)), grid="%dx%d" % (h, w),
                        dims=rng.choice(["44,42,42", "16,24,24", "32,48,48"]), theta=10000.0, far=0, factor=1.0,
                        window=0)
        return dict(op=op, T=_logint(rng, 1, 75600), grid="", dims=rng.choice(["64", "96", "128"]),
                    theta=rng.choice([10000.0, 500000.0]), far=_logint(rng, 1, 4000000),
                    factor=rng.choice([1.0, 2.0, 8.0]), window=rng.choice([0, 4096, 8192]))
    if op in ("norm_rope", "norm_quant"):
        Hk = rng.choice([4, 8, 10])
        case = dict(op=op, T=_logint(rng, 1, 32760), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, D=128,
                    norm=rng.choice(["token", "head"]), rot=rng.choice([64, 128]),
                    layout=rng.choice(["interleaved", "half"]))
        if op == "norm_quant":
            case["fmt"] = rng.choice(["mxfp4", "nvfp4"])
        else:
            case["D"], case["packed"] = rng.choice([64, 128]), rng.random() < 0.5
            case["rot"] = min(case["rot"], case["D"]) if rng.random() < 0.7 else 32
        return case
    if op == "attn":
        Hk = rng.choice([2, 4, 8])
        case = dict(op=op, Tq=_logint(rng, 1, 16384), Tk=_logint(rng, 1, 65536), Hq=Hk * rng.choice([1, 2, 3, 4, 5]),
                    Hk=Hk, D=rng.choice([64, 128]), docs=rng.randint(1, 4), causal=rng.random() < 0.6,
                    prefix=rng.choice([0, 100]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.3)
        while case["Hq"] * case["Tq"] * case["Tk"] > 16 * 8192 * 8192:
            case["Tk"] = max(1, case["Tk"] // 2)
        return case
    return dict(op=op, M=_logint(rng, 1, 32760), K=128 * rng.randint(4, 40), N=128 * rng.randint(4, 40),
                fmt=rng.choice(["mxfp4", "nvfp4"]), act=rng.choice(["none", "gelu_tanh", "silu"]),
                gate=rng.choice([0, 1, 4096]))


# ------------------------------------------------------------------------------ sizes
def _axis_dims(case):
    return [int(d) for d in case["dims"].split(",")]


def _offsets(T, docs):
    """Where documents packed on an axis of T tokens begin and end: uneven, some tokens behind the last."""
    cuts = [round(T * 0.97 * (i / docs) ** 1.2) for i in range(1, docs)]
    return [0, *cuts, T if docs == 1 else max(cuts[-1], T - T // 50)]


def _ranges(case):
    """Each query row's keys start .. end - 1: its document's, and of those in causal order the ones up to its own
    place counted from the document's end, or the document's prefix where that is longer."""
    q, k = _offsets(case["Tq"], case["docs"]), _offsets(case["Tk"], case["docs"])
    start, end = np.zeros(case["Tq"], np.int64), np.zeros(case["Tq"], np.int64)
    for d in range(case["docs"]):
        rows = np.arange(q[d], q[d + 1])
        n = np.full(rows.size, k[d + 1] - k[d])
        if case["causal"]:
            own_place = rows - q[d] + 1 + (k[d + 1] - k[d]) - (q[d + 1] - q[d])
            n = np.clip(np.maximum(own_place, min(case["prefix"], k[d + 1] - k[d])), 0, k[d + 1] - k[d])
        start[rows], end[rows] = k[d], k[d] + n
    return start, end


def work(case):
    op = case["op"]
    if op == "rope_table":
        dims = _axis_dims(case)
        return {"bytes": case["T"] * 4 * (len(dims) + sum(dims)), "flops": case["T"] * sum(dims) * 4}
    if op in ("norm_rope", "norm_quant"):
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        out = 2 * n
        if op == "norm_quant":  # codes and scales written, then read again
            out += 2 * (n // 2 + n // (32 if case["fmt"] == "mxfp4" else 16))
        return {"bytes": 2 * n + out + 4 * case["T"] * case["rot"] + 8 * case["Hk"] * case["D"], "flops": 8 * n}
    if op == "attn":
        start, end = _ranges(case)
        pairs = int(np.sum(end - start))
        seen = int(np.max(end) - np.min(start[end > start], initial=case["Tk"])) if pairs else 0
        return {"bytes": 2 * case["D"] * (2 * case["Tq"] * case["Hq"] + 2 * max(0, seen) * case["Hk"]),
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    M, K, N = case["M"], case["K"], case["N"]
    g = 32 if case["fmt"] == "mxfp4" else 16
    gates = 4 * N * -(-M // case["gate"]) if case["gate"] else 0
    return {"bytes": 2 * M * K + N * K // 2 + N * K // g + 4 * M * N + 2 * N + gates, "flops": 2 * M * N * K}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    op, s = case["op"], {"case": case}
    if op == "rope_table":
        t = torch.arange(case["T"], device="cuda", dtype=torch.int64)
        shift = torch.randint(0, 4096, (1,), generator=gen, device="cuda") + case["far"]
        if case["grid"]:
            h, w = (int(n) for n in case["grid"].split("x"))
            pos = torch.stack([t // (h * w) + shift, t // w % h, t % w], 1)
        else:
            pos = (t + shift)[:, None]
        s["positions"] = pos.to(torch.int32).contiguous()
    elif op in ("norm_rope", "norm_quant"):
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        if case.get("packed"):
            qkv = randn(T, Hq + 2 * Hk, D, scale=1.5)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = randn(T, Hq, D, scale=1.5), randn(T, Hk, D, scale=0.7)
        shape = (lambda H: (D,)) if case["norm"] == "head" else (lambda H: (H * D,))
        s["q_weight"] = 1 + randn(*shape(Hq), scale=0.2, dtype=F32)
        s["k_weight"] = 1 + randn(*shape(Hk), scale=0.2, dtype=F32)
        angle = torch.arange(T, device="cuda", dtype=F64)[:, None] * 10000.0 ** (
            -torch.arange(case["rot"] // 2, device="cuda", dtype=F64) / (case["rot"] // 2))
        angle += torch.rand(1, generator=gen, device="cuda", dtype=F64)
        s["table"] = torch.stack([angle.cos(), angle.sin()], 2).to(F32).reshape(T, case["rot"]).contiguous()
        if case.get("fmt") == "nvfp4":  # calibrated globals: amax / (6 * 448) of normed, rotated values
            s["q_global"] = torch.full((1,), 9.0 / 2688.0, device="cuda") * (1 + 0.1 * torch.rand(1, generator=gen, device="cuda"))
            s["k_global"] = s["q_global"] * 0.9
    elif op == "attn":
        Tq, Tk, Hq, Hk, D = (case[n] for n in ("Tq", "Tk", "Hq", "Hk", "D"))
        # sharper scores where they are capped, so that the cap is felt
        s["q"] = randn(Tq, Hq, D, scale=4.0 if case["cap"] else 1.5)
        kv = randn(Tk, 2 * Hk, D)
        s["k"], s["v"] = kv[:, :Hk], kv[:, Hk:]
        s["q_offsets"] = torch.tensor(_offsets(Tq, case["docs"]), dtype=torch.int32, device="cuda")
        s["k_offsets"] = torch.tensor(_offsets(Tk, case["docs"]), dtype=torch.int32, device="cuda")
        s["prefix"] = torch.full((case["docs"],), case["prefix"], dtype=torch.int32, device="cuda")
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=F32) / Hq) if case["bias"] else None
    else:
        M, K, N, g = case["M"], case["K"], case["N"], 32 if case["fmt"] == "mxfp4" else 16
        s["x"] = randn(M, K) * torch.exp(randn(K, scale=0.5, dtype=F32)).to(BF16)
        # a packed weight as it is stored: two codes a byte, scales in 128 x 4 atoms of 512 bytes
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        lo, hi = (117, 121) if g == 32 else (40, 120)
        s["scales"] = torch.randint(lo, hi, (N * K // g,), generator=gen, device="cuda", dtype=torch.uint8)
        s["w_global"] = torch.full((1,), 1.0 / 4096.0, device="cuda") if g == 16 else None
        s["a_global"] = torch.full((1,), 24.0 / 2688.0, device="cuda") if g == 16 else None
        s["bias"] = randn(N, scale=0.1, dtype=torch.float16)
        s["residual"] = randn(M, N, scale=2.0)
        rows = case["gate"]
        s["gate"] = randn((M + rows - 1) // rows, N, scale=0.5, dtype=F32) if rows else None
    return s


# ------------------------------------------------------------------------------ plain forms
def _frequencies(dims, theta, factor, window):
    """The pairs' frequencies of one axis; by parts where a trained window is given: pairs that turn often within
    it keep theirs, pairs that turn seldom are slowed by the factor, those between are blended."""
    j = torch.arange(dims // 2, device="cuda", dtype=F64)
    f = theta ** (-2.0 * j / dims)
    if factor == 1.0:
        return f
    if not window:
        return f / factor
    lo, hi = (dims * math.log(window / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (32.0, 1.0))
    lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), dims - 1)
    ramp = ((j - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp


def _amplitude(case):
    return 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0


def _plain_table(s):
    case = s["case"]
    dims = _axis_dims(case)
    f = torch.cat([_frequencies(d, case["theta"], case["factor"], case["window"]) for d in dims])
    axis = torch.repeat_interleave(torch.arange(len(dims), device="cuda"), torch.tensor([d // 2 for d in dims], device="cuda"))
    angle = s["positions"][:, axis].to(F64) * f
    return (torch.stack([angle.cos(), angle.sin()], 2) * _amplitude(case)).reshape(case["T"], -1).to(F32)


def _plain_norm_rope(x, weight, table, case, dtype):
    T, H, D = x.shape
    y = x.to(dtype)
    if case["norm"] == "head":
        y = y * (y.square().mean(2, keepdim=True) + 1e-6).rsqrt() * weight.to(dtype)
    else:
        y = y * (y.square().mean((1, 2), keepdim=True) + 1e-6).rsqrt() * weight.to(dtype).view(H, D)
    R = case["rot"]
    cos, sin = table.to(dtype).view(T, 1, R // 2, 2).unbind(3)
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["layout"] == "interleaved" else (y[..., :R // 2], y[..., R // 2:R])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], 3).flatten(2) if case["layout"] == "interleaved" else torch.cat([u, v], 2)
    return torch.cat([turned, y[..., R:]], 2)


def _to_bf16(x):
    """64-bit values rounded once to the nearest bf16 (the conversion by way of 32 bits would round twice)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8)


def _to_e2m1(x):
    """The nearest FP4 value, ties to the even code, saturating; x within a block's scale."""
    m = x.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign((torch.round(m / step) * step).clamp(max=6.0), x)


def _to_e4m3(x):
    return x.clamp(max=448.0).to(torch.float8_e4m3fn).to(F32)


def _plain_fp4(x, fmt, g):
    """bf16-valued x [..., n] (32 bits) quantized in blocks along its last axis: the values that codes and scales
    stand for, in 32 bits."""
    b = x.reshape(*x.shape[:-1], -1, 32 if fmt == "mxfp4" else 16)
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        scale = torch.ldexp(torch.ones_like(amax), torch.frexp(amax)[1] - 3)
        out = _to_e2m1(b / scale) * scale
    else:
        d = _to_e4m3(amax / (6.0 * g)) * g
        out = _to_e2m1(b * (1.0 / d)) * d
    return torch.where(amax > 0, out, 0.0).reshape(x.shape)


def _plain_ranges(s):
    case = s["case"]
    row = torch.arange(case["Tq"], device="cuda")[:, None]
    q0, q1, k0, k1 = s["q_offsets"][:-1].long(), s["q_offsets"][1:].long(), s["k_offsets"][:-1].long(), s["k_offsets"][1:].long()
    n = (k1 - k0).expand(case["Tq"], -1)
    if case["causal"]:
        n = torch.minimum(n, torch.maximum(row - q0 + 1 + n - (q1 - q0), s["prefix"].long())).clamp(min=0)
    inside = (row >= q0) & (row < q1)
    return torch.where(inside, k0, 0).sum(1), torch.where(inside, k0 + n, 0).sum(1)


def _plain_attn(s):
    case = s["case"]
    Tq, Tk, Hq, Hk, D = (case[n] for n in ("Tq", "Tk", "Hq", "Hk", "D"))
    q = s["q"].to(F32).view(Tq, Hk, Hq // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)
    scores = (q @ s["k"].to(F32).permute(1, 2, 0)).view(Hq, Tq, Tk) * D ** -0.5
    if case["cap"]:
        scores = torch.tanh(scores / case["cap"]) * case["cap"]
    key = torch.arange(Tk, device="cuda")
    if case["bias"]:
        place = torch.arange(Tq, device="cuda") + (Tk - Tq)
        scores = scores - s["slopes"][:, None, None] * (place[:, None] - key).abs()
    start, end = _plain_ranges(s)
    scores = torch.where((key >= start[:, None]) & (key < end[:, None]), scores, -math.inf)
    top = scores.amax(2, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(2, keepdim=True)
    o = (p.view(Hk, -1, Tk) @ s["v"].to(F32).transpose(0, 1)).view(Hq, Tq, D) / torch.where(total == 0, 1.0, total)
    return o.transpose(0, 1).to(BF16), (top + torch.log(total)).squeeze(2).t()


def _weight(s, dtype):
    """The packed weight's values: codes times scales (times the NVFP4 global)."""
    case = s["case"]
    N, K, g = case["N"], case["K"], 32 if case["fmt"] == "mxfp4" else 16
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda", dtype=dtype)
    w = grid[torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).long()].view(N, K // g, g)
    sf = s["scales"].view(N // 128, K // g // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(N, K // g)
    scale = torch.ldexp(torch.ones_like(sf, dtype=dtype), sf.int() - 127) if g == 32 else sf.view(torch.float8_e4m3fn).to(dtype)
    return (w * scale[:, :, None]).view(N, K)


def _plain_linear(s):
    case = s["case"]
    x = _plain_fp4(s["x"].to(F32), case["fmt"], s["a_global"])
    z = x @ _weight(s, F32).t()
    if s["w_global"] is not None:
        z = z * s["w_global"]
    z = z + s["bias"].to(F32)
    if case["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    elif case["act"] == "gelu_tanh":
        z = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if s["gate"] is not None:
        z = z * s["gate"][torch.arange(case["M"], device="cuda") // case["gate"]]
    return (s["residual"].to(F32) + z).to(BF16)


# ------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s)
    if op == "rope_table":
        return _plain_table(s)
    if op == "norm_rope":
        return tuple(_plain_norm_rope(s[n], s[n + "_weight"], s["table"], case, F32).to(BF16) for n in ("q", "k"))
    if op == "norm_quant":  # 64 bits: which bf16, and then which code, is a matter of borders
        return tuple(_plain_fp4(_to_bf16(_plain_norm_rope(s[n], s[n + "_weight"], s["table"], case, F64)).to(F32),
                                case["fmt"], s.get(n + "_global")).to(BF16) for n in ("q", "k"))
    return _plain_attn(s) if op == "attn" else _plain_linear(s)


def _own(s):
    import fp4_block_scaled_act_b200 as fb

    case = s["case"]
    op = case["op"]
    if op == "rope_table":
        return fb.rope_table(s["positions"], _axis_dims(case), case["theta"], factor=case["factor"],
                             window=case["window"], amplitude=_amplitude(case))
    if op == "norm_rope":
        return fb.qk_norm_rope(s["q"], s["k"], norm=case["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                               eps=1e-6, table=s["table"], layout=case["layout"])
    if op == "norm_quant":
        heads = fb.qk_norm_rope_quantize_heads(s["q"], s["k"], fmt=case["fmt"], norm=case["norm"],
                                               q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                               table=s["table"], layout=case["layout"], g_q=s.get("q_global"),
                                               g_k=s.get("k_global"))
        return tuple(fb.dequantize_heads(h, case["T"], fmt=case["fmt"], g=s.get(n + "_global"))
                     for n, h in zip("qk", heads))
    if op == "attn":
        start, end = fb.attn_ranges(s["q_offsets"], s["k_offsets"], case["Tq"], case["Tk"], causal=case["causal"],
                                    prefix=s["prefix"])
        return fb.attn_bf16(s["q"], s["k"], s["v"], scale=case["D"] ** -0.5, softcap=case["cap"], slopes=s["slopes"],
                            q_pos=case["Tk"] - case["Tq"], key_start=start, key_end=end, return_lse=True)
    pw = fb.PackedWeight(fb.MXFP4 if case["fmt"] == "mxfp4" else fb.NVFP4, case["N"], case["K"], s["codes"],
                         s["scales"], s["w_global"])
    return fb.linear_residual(s["x"], pw, s["residual"], bias=s["bias"], act=case["act"], gate=s["gate"],
                              gate_rows=case["gate"], a_global=s["a_global"])


# ------------------------------------------------------------------------------ 64 bits
def _exact_rotate(x, weight, table, case):
    """Norm and rotation as a product of complex numbers."""
    T, H, D = x.shape
    R = case["rot"]
    z = x.double()
    over = z.reshape(T, H, D) if case["norm"] == "head" else z.reshape(T, 1, H * D)
    rms = torch.sqrt(torch.sum(over * over, 2) / over.shape[2] + 1e-6)
    z = z / rms[:, :, None] * (weight.double() if case["norm"] == "head" else weight.double().reshape(1, H, D))
    turn = torch.view_as_complex(table.double().reshape(T, 1, R // 2, 2).contiguous())
    if case["layout"] == "interleaved":
        out = torch.view_as_real(torch.view_as_complex(z[:, :, :R].reshape(T, H, R // 2, 2).contiguous()) * turn).reshape(T, H, R)
    else:
        w = torch.complex(z[:, :, :R // 2].contiguous(), z[:, :, R // 2:R].contiguous()) * turn
        out = torch.cat((w.real, w.imag), 2)
    return torch.cat((out, z[:, :, R:]), 2)


def _exact_fp4(x, fmt, g):
    """Blocks quantized by the format's rule: each step of the scale's own rule in 32 bits where the format says so,
    the codes by counting the borders that a magnitude has passed."""
    size = 32 if fmt == "mxfp4" else 16
    b = x.reshape(*x.shape[:-1], x.shape[-1] // size, size)
    top = b.abs().max(-1, keepdim=True).values
    if fmt == "mxfp4":
        scale = 2.0 ** (torch.floor(torch.log2(top.clamp(min=2.0 ** -120))) - 2)
        scale = torch.where(scale * 8 <= top, scale * 2, torch.where(scale * 4 > top, scale / 2, scale))
        ratio = b / scale
    else:
        step = (top.float() / (g.float() * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float() * g.float()
        scale = step.double()
        ratio = (b.float() * step.reciprocal()).double()
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device, dtype=torch.float64)
    m = ratio.abs()
    code = torch.bucketize(m, borders, right=False)  # borders strictly below m
    tie_up = (m == 0.75) | (m == 1.75) | (m == 3.5)  # ties go to the even code
    code = (code + tie_up).clamp(max=7)
    values = torch.tensor(E2M1, device=x.device, dtype=torch.float64)[code]
    return torch.where(top > 0, torch.sign(b) * values * scale, 0.0).reshape(x.shape)


def _exact_attn(s):
    case = s["case"]
    Tq, Tk, Hq, Hk, D = (case[n] for n in ("Tq", "Tk", "Hq", "Hk", "D"))
    start, end = (torch.from_numpy(a).cuda() for a in _ranges(case))
    q, k, v = (s[n].double() for n in "qkv")
    key = torch.arange(Tk, device="cuda")[None, :]
    open_ = (start[:, None] <= key) & (key < end[:, None])
    o, lse = torch.zeros(Tq, Hq, D, device="cuda", dtype=F64), torch.empty(Tq, Hq, device="cuda", dtype=F64)
    for h in range(Hq):
        a = torch.mm(q[:, h], k[:, h // (Hq // Hk)].t()) / math.sqrt(D)
        if case["cap"]:
            a = case["cap"] * torch.tanh(a / case["cap"])
        if s["slopes"] is not None:
            place = torch.arange(Tk - Tq, Tk, device="cuda")[:, None]
            a = a - s["slopes"][h].double() * torch.abs(key - place).double()
        a = a.masked_fill(~open_, -math.inf)
        lse[:, h] = torch.logsumexp(a, 1)
        some = torch.isfinite(lse[:, h])
        o[some, h] = torch.mm(torch.exp(a[some] - lse[some, h, None]), v[:, h // (Hq // Hk)])
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope_table":
        parts = []
        for axis, d in enumerate(_axis_dims(case)):
            freq = []
            for j in range(d // 2):
                f = case["theta"] ** (-2.0 * j / d)
                if case["factor"] != 1.0 and case["window"]:
                    place = [d * math.log(case["window"] / (2 * math.pi * t)) / (2 * math.log(case["theta"])) for t in (32.0, 1.0)]
                    first, last = max(math.floor(place[0]), 0), min(math.ceil(place[1]), d - 1)
                    slow = min(max((j - first) / max(last - first, 1e-3), 0.0), 1.0)
                    f = slow * f / case["factor"] + (1.0 - slow) * f
                elif case["factor"] != 1.0:
                    f /= case["factor"]
                freq.append(f)
            parts.append(torch.outer(s["positions"][:, axis].double(), torch.tensor(freq, device="cuda", dtype=F64)))
        z = torch.polar(torch.full((), _amplitude(case), device="cuda", dtype=F64), torch.cat(parts, 1))
        return torch.view_as_real(z).reshape(case["T"], -1)
    if op == "norm_rope":
        return tuple(_exact_rotate(s[n], s[n + "_weight"], s["table"], case) for n in ("q", "k"))
    if op == "norm_quant":
        return tuple(_exact_fp4(_to_bf16(_exact_rotate(s[n], s[n + "_weight"], s["table"], case)), case["fmt"],
                                s.get(n + "_global")) for n in ("q", "k"))
    if op == "attn":
        return _exact_attn(s)
    x = _exact_fp4(s["x"].double(), case["fmt"], s["a_global"])
    z = torch.addmm(s["bias"].double(), x, _weight(s, F64).t(), alpha=1.0 if s["w_global"] is None else float(s["w_global"]))
    if case["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif case["act"] == "gelu_tanh":
        z = torch.nn.functional.gelu(z, approximate="tanh")
    if s["gate"] is not None:
        z = z * torch.repeat_interleave(s["gate"].double(), case["gate"], 0)[:case["M"]]
    return s["residual"].double() + z
