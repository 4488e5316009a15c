"""The INT8 (W8A8, one scale per token and per channel) operators and the several-axis rotary: what is
measured, with each operator's plain form in elementary torch operations and its definition in 64 bits.

Sizes are the vision tower's own (hidden 1152, QKV 3456, MLP 4304, merger 4608 -> 2048, 16 heads of 72,
the 46x136, 36x27 and 16x16 images and packed batches of them) and a grouped-query language layer's
rotary (32 + 8 heads of 128).
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one merged token through the merger's first linear: latency, every weight read once
        dict(name="gemm_1x4608x4608", op="gemm", M=1, N=4608, K=4608, out="bf16", bias=True, residual=False),
        # the merged tokens of one 36x27 image through the merger's second linear: few tiles, ragged M
        dict(name="gemm_243x2048x4608", op="gemm", M=243, N=2048, K=4608, out="fp32", bias=True, residual=False),
        # fc2 of one 46x136 image with its residual
        dict(name="gemm_6256x1152x4304", op="gemm", M=6256, N=1152, K=4304, out="bf16", bias=True, residual=True),
        # QKV of four packed 46x136 images, fp16 out
        dict(name="gemm_25024x3456x1152", op="gemm", M=25024, N=3456, K=1152, out="fp16", bias=True, residual=False),
        # the attention output of a packed batch before the output projection
        dict(name="quant_9164x1152", op="quant", M=9164, K=1152, dtype="bf16", pad=0),
        # fp32 master weights of the merger's linear, one scale per output channel
        dict(name="quant_4608x4608_fp32", op="quant", M=4608, K=4608, dtype="fp32", pad=0),
        # the first LayerNorm of a small image: latency
        dict(name="ln_256x1152", op="ln", M=256, K=1152, pad=0),
        # the same over four packed 46x136 images
        dict(name="ln_25024x1152", op="ln", M=25024, K=1152, pad=0),
        # the MLP of one 36x27 image
        dict(name="gelu_972x4304", op="gelu", M=972, K=4304, pad=0),
        # the MLP of four packed 46x136 images
        dict(name="gelu_25024x4304", op="gelu", M=25024, K=4304, pad=0),
        # q and k inside packed qkv rows of a video of 8 x 32 x 32 patches, 12 frequencies per axis
        dict(name="rope_video_8192", op="rope", n=8192, hq=16, hk=16, d=72, st=12, sh=12, sw=12, dtype="bf16",
             packed=True, interleaved=False, axis_freq=True, adjacent=False, inverse=False, far=0),
        # the gradient through a language layer's rotary over a long prompt with images
        dict(name="rope_grad_16384", op="rope", n=16384, hq=32, hk=8, d=128, st=24, sh=20, sw=20, dtype="bf16",
             packed=False, interleaved=True, axis_freq=False, adjacent=False, inverse=True, far=100000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:   # a case that costs no more than the largest listed ones
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= 3.3e8 and w["flops"] <= 1.99e11:
            return case


def _draw(rng):
    op = rng.choice(["gemm", "gemm", "quant", "ln", "gelu", "rope"])
    if op == "gemm":
        residual = rng.random() < 0.3
        return dict(op=op, M=_log(rng, 1, 25024), N=_log(rng, 64, 4608), K=_log(rng, 64, 4608),
                    out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), bias=rng.random() < 0.7, residual=residual)
    if op == "quant":
        return dict(op=op, M=_log(rng, 1, 25024), K=_log(rng, 32, 8192), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    pad=rng.choice([0, 0, 8, 24, 5]))
    if op in ("ln", "gelu"):
        return dict(op=op, M=_log(rng, 1, 25024), K=_log(rng, 64, 4608), pad=rng.choice([0, 0, 8, 40, 3]))
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([1, 1, 2, 4]) if hk < 16 else hk
    st, sh, sw = rng.choice([(12, 12, 12), (24, 20, 20), (16, 24, 24), (0, 18, 18), (8, 12, 12), (9, 10, 11), (11, 11, 10)])
    interleaved = st >= max(sh, sw) and rng.random() < 0.5
    d = 2 * (st + sh + sw)
    return dict(op=op, n=_log(rng, 1, 16384), hq=hq, hk=hk, d=rng.choice([d, d, d + 16, 2 * d]), st=st, sh=sh, sw=sw,
                dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), packed=rng.random() < 0.5, interleaved=interleaved,
                axis_freq=rng.random() < 0.4, adjacent=rng.random() < 0.3, inverse=rng.random() < 0.4,
                far=rng.choice([0, 0, 1000, 100000, 1000000]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(x, pad):
    """x with `pad` unused elements behind each row."""
    if not pad:
        return x.contiguous()
    wide = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _codes(x):
    """int8 codes with a row stride of a multiple of 16 bytes, and a scale per row."""
    s = x.abs().amax(dim=1) / 127
    q = torch.zeros((x.shape[0], (x.shape[1] + 15) // 16 * 16), dtype=torch.int8, device=x.device)
    q[:, :x.shape[1]] = torch.round(x / s.clamp_min(1e-30)[:, None]).clamp(-127, 127).to(torch.int8)
    return q[:, :x.shape[1]], s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "gemm":
        M, N, K, t = case["M"], case["N"], case["K"], _T[case["out"]]
        # a LayerNorm's output: unit variance with a few channels of large activations
        chan = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 8.0, 1.0)
        qa, sa = _codes(_rand(g, M, K) * chan)
        qw, sw = _codes(_rand(g, N, K) * 0.02)
        bias = (_rand(g, N) * 0.01).to(t) if case["bias"] else None
        residual = _rand(g, M, N).to(t) if case["residual"] else None
        return dict(case, qa=qa, sa=sa, qw=qw, sw=sw, bias_t=bias, residual_t=residual)
    if op == "quant":
        x = _rand(g, case["M"], case["K"]) * torch.exp(_rand(g, case["M"], 1))
        return dict(case, x=_rows(x.to(_T[case["dtype"]]), case["pad"]))
    if op == "ln":
        x = _rand(g, case["M"], case["K"]) * torch.exp(_rand(g, case["M"], 1)) + _rand(g, case["M"], 1)
        gamma, beta = 1 + 0.02 * _rand(g, case["K"]), 0.01 * _rand(g, case["K"])
        return dict(case, x=_rows(x.bfloat16(), case["pad"]), gamma=gamma.bfloat16(), beta=beta.bfloat16())
    if op == "gelu":
        return dict(case, x=_rows((_rand(g, case["M"], case["K"]) * 1.3).bfloat16(), case["pad"]))
    n, hq, hk, d, t = case["n"], case["hq"], case["hk"], case["d"], _T[case["dtype"]]
    if case["packed"]:   # q, k and v of a token side by side
        qkv = _rand(g, n, (hq + 2 * hk) * d).to(t)
        q, k = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
    else:
        q, k = _rand(g, n, hq, d).to(t), _rand(g, n, hk, d).to(t)
    # (time, row, column) of the patches of a video, behind `far` earlier positions
    i = torch.arange(n, device="cuda")
    side = 32 if n >= 1024 else 4
    at = torch.stack([i // (side * side), i // side % side, i % side], 1)
    pos = (at + torch.randint(0, case["far"] + 64, (1, 3), generator=g, device="cuda")).int().contiguous()
    return dict(case, q=q, k=k, pos=pos)


# ---------------------------------------------------------------- plain forms

def _axis_and_frequency(case, theta=10000.0):
    """Axis of each rotary pair, and its frequency, in 64 bits."""
    sec = [case["st"], case["sh"], case["sw"]]
    total = sum(sec)
    j = torch.arange(total, dtype=torch.int64, device="cuda")
    if case["interleaved"]:   # pair j belongs to axis j mod 3 while that axis has pairs left, else to axis 0
        axis = torch.zeros_like(j)
        axis = torch.where((j % 3 == 1) & (j < 3 * sec[1]), 1, axis)
        axis = torch.where((j % 3 == 2) & (j < 3 * sec[2]), 2, axis)
    else:
        axis = (j >= sec[0]).long() + (j >= sec[0] + sec[1]).long()
    if case["axis_freq"]:     # the frequencies start over on each axis
        same = (axis[None, :] == axis[:, None])
        rank = (same & (j[None, :] < j[:, None])).sum(1)
        power = rank.double() / same.sum(1).double()
    else:
        power = j.double() / total
    return axis, theta ** -power


def _round_bf16(y):
    """64-bit values rounded once to bf16 (a cast by way of fp32 would round twice)."""
    b = y.contiguous().view(torch.int64)
    b = (b + (((b >> 45) & 1) + ((1 << 44) - 1))) >> 45 << 45
    return torch.where(torch.isfinite(y), b.view(torch.float64), y).to(torch.bfloat16)


def _quant(y):
    """One scale per row, and the nearest codes (the quotient in 64 bits: values lie next to a border)."""
    amax = y.abs().amax(dim=1).float()
    s = torch.where(torch.isfinite(amax), amax / torch.full_like(amax, 127), math.nan)   # a division: by the
    # number 127 torch multiplies with its rounded reciprocal
    q = torch.round(y.double() / s.double()[:, None])
    q = torch.where((s > 0)[:, None], q, 0.0).clamp(-127, 127).to(torch.int8)
    return q, s


def _rotate(x, cos, sin, pairs, adjacent):
    r = 2 * pairs
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if adjacent else (x[..., :pairs], x[..., pairs:r])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if adjacent:
        y[..., 0:r:2], y[..., 1:r:2] = ya, yb
    else:
        y[..., :pairs], y[..., pairs:r] = ya, yb
    return y


def run(s):
    op = s["op"]
    if own:
        from quantized_vit_encoder_b200 import vitq
        if op == "gemm":
            return vitq.int8_gemm(s["qa"], s["sa"], s["qw"], s["sw"], bias=s["bias_t"], residual=s["residual_t"],
                                  out_dtype=_T[s["out"]])
        if op == "quant":
            return vitq.quant_int8(s["x"])
        if op == "ln":
            return vitq.ln_quant_int8(s["x"], s["gamma"], s["beta"], eps=1e-6)
        if op == "gelu":
            return vitq.gelu_quant_int8(s["x"])
        return vitq.rope_axes(s["q"], s["k"], s["pos"], (s["st"], s["sh"], s["sw"]), theta=10000.0,
                              interleaved=s["interleaved"], axis_freq=s["axis_freq"], adjacent=s["adjacent"],
                              inverse=s["inverse"])
    if op == "gemm":
        y = s["qa"].float() @ s["qw"].float().t()
        y = y * s["sa"][:, None] * s["sw"][None, :]
        if s["bias_t"] is not None:
            y = y + s["bias_t"].float()
        if s["residual_t"] is not None:
            y = y + s["residual_t"].float()
        return y.to(_T[s["out"]])
    if op == "quant":
        return _quant(s["x"])
    if op == "ln":
        x = s["x"].double()
        c = x - x.mean(dim=1, keepdim=True)
        y = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + 1e-6) * s["gamma"].double() + s["beta"].double()
        return _quant(_round_bf16(y))
    if op == "gelu":
        x = s["x"].double()
        u = math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
        return _quant(_round_bf16(x / (1 + torch.exp(-2 * u))))
    axis, freq = _axis_and_frequency(s)
    angle = s["pos"][:, axis].double() * freq
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    sin = -sin if s["inverse"] else sin
    pairs = s["st"] + s["sh"] + s["sw"]
    return [_rotate(x.float(), cos, sin, pairs, s["adjacent"]).to(x.dtype) for x in (s["q"], s["k"])]


# ---------------------------------------------------------------- work and the definitions in 64 bits

def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K, e = case["M"], case["N"], case["K"], _ES[case["out"]]
        mn = M * N * e * (2 if case["residual"] else 1)
        return {"bytes": M * K + N * K + 4 * M + 4 * N + (N * e if case["bias"] else 0) + mn, "flops": 2 * M * N * K}
    if op == "rope":
        n, d = case["n"], case["d"]
        moved = 2 * n * (case["hq"] + case["hk"]) * d * _ES[case["dtype"]]
        return {"bytes": moved + 12 * n, "flops": 6 * n * (case["hq"] + case["hk"]) * (case["st"] + case["sh"] + case["sw"])}
    M, K = case["M"], case["K"]
    moved = M * K * (_ES[case.get("dtype", "bf16")] + 1) + 4 * M
    if op == "ln":
        return {"bytes": moved + 4 * K, "flops": 9 * M * K}
    return {"bytes": moved, "flops": (12 if op == "gelu" else 2) * M * K}


def _exact_codes(y):
    """Scale and codes of rows that hold bf16, fp16 or fp32 values, from the definition."""
    top = y.abs().max(dim=1, keepdim=True).values
    scale = torch.div(top, torch.full_like(top, 127))
    held = scale.float().double()      # the scale is a 32-bit number, the codes go by that number
    return torch.round(y / held).to(torch.int8), scale[:, 0]


def _nearest_bf16(y):
    """bf16 neighbours of 64-bit values: eight significant bits, ties to even."""
    m, e = torch.frexp(y)
    return torch.ldexp(torch.round(m * 256), e - 8)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gemm":
        acc = torch.matmul(s["qa"].double(), s["qw"].double().transpose(0, 1))   # whole numbers below 2^53
        acc *= s["sa"].double().unsqueeze(1) * s["sw"].double().unsqueeze(0)
        for extra in (s["bias_t"], s["residual_t"]):
            if extra is not None:
                acc += extra.double()
        return acc
    if op == "quant":
        return _exact_codes(s["x"].double())
    if op == "ln":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        return _exact_codes(_nearest_bf16((x - mean) / torch.sqrt(var + 1e-6) * s["gamma"].double() + s["beta"].double()))
    if op == "gelu":
        x = s["x"].double()
        return _exact_codes(_nearest_bf16(x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))))
    # each pair as a complex number, turned by its angle
    sec, out = (case["st"], case["sh"], case["sw"]), []
    total, taken, owner, power = sum(sec), [0, 0, 0], [], []
    for j in range(total):
        if case["interleaved"]:
            a = j % 3 if j % 3 and j < 3 * sec[j % 3] else 0
        else:
            a = 0 if j < sec[0] else 1 if j < sec[0] + sec[1] else 2
        power.append(taken[a] / sec[a] if case["axis_freq"] else j / total)
        taken[a] += 1
        owner.append(a)
    turn = s["pos"].double()[:, owner] * torch.tensor([10000.0 ** -p for p in power], dtype=torch.float64, device="cuda")
    spin = torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn).unsqueeze(1)
    for x in (s["q"].double(), s["k"].double()):
        head, rest = x[..., :2 * total], x[..., 2 * total:]
        if case["adjacent"]:
            z = torch.view_as_complex(head.unflatten(-1, (total, 2)).contiguous()) * spin
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :total].contiguous(), head[..., total:].contiguous()) * spin
            head = torch.cat([z.real, z.imag], dim=-1)
        out.append(torch.cat([head, rest], dim=-1))
    return out
