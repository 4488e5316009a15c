"""Rotary over several axes against its definition in 64 bits, forward and inverse.

Tolerance: the angle's turn is exact to 2^-45 or better, its fp32 reduction is off by
2^-26 of a turn (2^-23.3 rad), sine and cosine by 2 units of 2^-24, so each of the two
products is off by at most 2^-22 |x|, plus two fp32 roundings; with |x_a| + |x_b| <= m
that is 2^-21 m, then one rounding to the type.
"""
import math

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _pos(seed, n, axes, far):
    return torch.randint(-min(far, 50), far + 1, (n, axes), generator=torch.Generator(device="cuda").manual_seed(seed),
                         device="cuda", dtype=torch.int32)


def _layout(sections, theta, interleaved, axis_freq):
    """(axis, frequency) of every pair, one by one."""
    total, n = sum(sections), len(sections)
    axis = []
    for j in range(total):
        if interleaved:
            a = j % n
            axis.append(a if a and j < n * sections[a] else 0)
        else:
            a, left = 0, j
            while left >= sections[a]:
                left -= sections[a]
                a += 1
            axis.append(a)
    seen, freq = [0] * n, []
    for j, a in enumerate(axis):
        freq.append(theta ** (-seen[a] / sections[a] if axis_freq else -j / total))
        seen[a] += 1
    assert seen == list(sections)
    return axis, freq


def _ref(x, pos, sections, theta=10000.0, interleaved=False, axis_freq=False, adjacent=False, inverse=False):
    axis, freq = _layout(sections, theta, interleaved, axis_freq)
    ang = pos.double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None] * (-1 if inverse else 1)
    x, y, r, h = x.double(), x.double().clone(), 2 * len(axis), len(axis)
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if adjacent else (slice(0, h), slice(h, r))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag = torch.zeros_like(x)
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def _close(got, x, pos, sections, **kw):
    want, mag = _ref(x, pos, sections, **kw)
    t = got.dtype
    tol = 2.0 ** -21 * mag + torch.finfo(t).eps / 2 * (want.abs() + 2.0 ** -21 * mag)
    tol = torch.where(mag > 0, tol + (2.0 ** -25 if t == HF else 0.0), 0.0)      # what passes through is equal
    off = (got.double() - want).abs() - tol
    assert (off <= 0).all(), f"{int((off > 0).sum())} of {off.numel()} off, worst {off.max().item():.3e}"


CASES = [  # sections, head_dim, heads q, heads k
    ((12, 12, 12), 72, 16, 16), ((0, 18, 18), 72, 4, 2), ((24, 20, 20), 128, 8, 2), ((16, 24, 24), 128, 3, 1),
    ((9, 10, 11), 60, 2, 2), ((11, 11, 10), 64, 5, 1), ((1,), 2, 1, 1), ((3, 2), 16, 2, 1), ((7, 5, 4, 1), 40, 2, 3),
    ((64, 0, 0), 256, 2, 2), ((128, 64, 64), 512, 1, 1), ((5,), 11, 3, 2),
    ((1,), 511, 1, 2), ((64, 64, 127), 512, 2, 1), ((30, 30, 4), 200, 20, 7)]


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("sections,d,hq,hk", CASES)
@pytest.mark.parametrize("adjacent", [False, True])
def test_forward_and_inverse(sections, d, hq, hk, adjacent, t):
    for n in (1, 7, 130):
        q, k, pos = _randn(n, n, hq, d).to(t), _randn(n + 1, n, hk, d).to(t), _pos(n, n, len(sections), 300)
        for kw in (dict(), dict(axis_freq=True), dict(inverse=True, theta=1e6)):
            kw = dict(kw, adjacent=adjacent)
            yq, yk = vitq.rope_axes(q, k, pos, sections, **kw)
            _close(yq, q, pos, sections, **kw)
            _close(yk, k, pos, sections, **kw)


@pytest.mark.parametrize("sections,d", [((24, 20, 20), 128), ((12, 12, 12), 72), ((11, 11, 10), 64), ((6, 6), 24),
                                        ((5, 4, 4, 3), 32), ((20, 0, 8), 64)])
@pytest.mark.parametrize("axis_freq", [False, True])
def test_interleaved(sections, d, axis_freq):
    q, k, pos = _randn(1, 50, 4, d).to(BF), _randn(2, 50, 2, d).to(BF), _pos(3, 50, len(sections), 1000)
    yq, yk = vitq.rope_axes(q, k, pos, sections, interleaved=True, axis_freq=axis_freq)
    _close(yq, q, pos, sections, interleaved=True, axis_freq=axis_freq)
    _close(yk, k, pos, sections, interleaved=True, axis_freq=axis_freq)


@pytest.mark.parametrize("far", [10 ** 5, 10 ** 7, 2 ** 31 - 1])
def test_far_positions(far):
    q, pos = _randn(1, 40, 2, 128), _pos(2, 40, 3, far)
    pos[0] = far
    pos[1] = -far
    y, none = vitq.rope_axes(q, None, pos, (24, 20, 20))
    assert none is None
    if far <= 10 ** 7:
        _close(y, q, pos, (24, 20, 20))
    else:   # 2^31 positions times a frequency known to 2^-47: 2^-13 rad, of both sides' angles
        want, mag = _ref(q, pos, (24, 20, 20))
        assert ((y.double() - want).abs() <= 2.0 ** -12 * mag).all()


def test_matches_the_two_axis_rotary():
    """Sections (18, 18) with per-axis frequencies are vit_rope2d's rotary of 72-wide heads."""
    n = 300
    qkv = _randn(4, n, 3456).to(BF)
    pos = _pos(5, n, 2, 130).clamp_min(0)
    want = vitq.rope2d_(qkv.clone(), vitq.rope_table(pos))
    q, k = qkv[:, :1152].view(n, 16, 72), qkv[:, 1152:2304].view(n, 16, 72)
    v = qkv[:, 2304:].clone()
    yq, yk = vitq.rope_axes(q, k, pos, (18, 18), axis_freq=True)
    for got, ref in ((yq, want[:, :1152]), (yk, want[:, 1152:2304])):
        # both round the same value to bf16, from fp32 results at most 2^-20 of |a| + |b| apart
        d = (got.reshape(n, 1152).double() - ref.double()).abs()
        assert (d <= 2.0 ** -20 * 20 + torch.finfo(BF).eps * ref.double().abs()).all()
    vitq.rope_axes_(q, k, pos, (18, 18), axis_freq=True)
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, 2304:], v)


@pytest.mark.parametrize("t", [BF, F32])
def test_strides_orders_and_alignments(t):
    n, h, d, sec = 33, 6, 80, (10, 12, 10)
    pos = _pos(1, n, 3, 200)
    base = _randn(2, n, h, d).to(t)
    views = [base.transpose(0, 1).contiguous().transpose(0, 1),                          # heads outermost
             torch.nn.functional.pad(base, (1, 2))[..., 1:d + 1],                        # odd start and row pitch
             base[:, :1].expand(n, h, d), base[:1].expand(n, h, d)]                      # broadcast inputs
    for x in views:
        y, _ = vitq.rope_axes(x, None, pos, sec)
        _close(y, x, pos, sec)
        out = torch.full((h, n, d + 3), 9.0, dtype=t, device="cuda")
        o = out[:, :, 1:d + 1].transpose(0, 1)
        vitq.rope_axes(x, None, pos, sec, out=(o, None))
        assert torch.equal(o, y) and (out[:, :, 0] == 9).all() and (out[:, :, d + 1:] == 9).all()
    by_axis = pos.t().contiguous()                                                       # positions as [axes, n]
    assert torch.equal(vitq.rope_axes(base, None, by_axis.t(), sec)[0], vitq.rope_axes(base, None, pos, sec)[0])
    one = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].expand(n, 3)        # text: the same on every axis
    _close(vitq.rope_axes(base, None, one, sec)[0], base, one, sec)


def test_in_place_equals_out_of_place():
    q, k, pos = _randn(1, 65, 4, 96).to(HF), _randn(2, 65, 2, 96).to(HF), _pos(3, 65, 3, 99)
    want = vitq.rope_axes(q, k, pos, (16, 8, 8), interleaved=True)
    vitq.rope_axes_(q, k, pos, (16, 8, 8), interleaved=True)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_inverse_is_the_gradient():
    """Against the definition differentiated by torch in fp64, and against differences."""
    n, sec = 9, (6, 5, 5)
    pos = _pos(1, n, 3, 40)
    x = _randn(2, n, 2, 40).double().requires_grad_()
    dy = _randn(3, n, 2, 40)
    y, _ = _ref_grad(x, pos, sec)
    (grad,) = torch.autograd.grad(y, x, dy.double())
    got, _ = vitq.rope_axes(dy, None, pos, sec, inverse=True)
    mag = dy.abs().amax().double() * 2
    assert ((got.double() - grad).abs() <= 2.0 ** -21 * mag + 2.0 ** -24 * grad.abs()).all()
    # directional difference of the library's own forward (linear, so any step is exact up to rounding)
    x32, v = x.detach().float(), _randn(5, n, 2, 40)
    fwd = lambda z: vitq.rope_axes(z, None, pos, sec)[0].double()          # noqa: E731
    lhs = ((fwd(x32 + v) - fwd(x32)) * dy.double()).sum()
    rhs = (v.double() * got.double()).sum()
    # 720 products, each term off by 2^-20 of values of a few units at most (|x|, |v|, |dy| < 5)
    assert (lhs - rhs).abs() <= 720 * 2.0 ** -20 * 5 * 20


def _ref_grad(x, pos, sec):
    axis, freq = _layout(sec, 10000.0, False, False)
    ang = pos.double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    c, s, h = torch.cos(ang)[:, None], torch.sin(ang)[:, None], len(axis)
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1), None


def test_no_tokens_and_non_finite_values():
    e = torch.empty((0, 4, 72), dtype=BF, device="cuda")
    y, _ = vitq.rope_axes(e, e, torch.empty((0, 3), dtype=torch.int32, device="cuda"), (12, 12, 12))
    assert y.shape == (0, 4, 72)
    q, pos = _randn(1, 4, 2, 72), _pos(2, 4, 3, 9)
    clean, _ = vitq.rope_axes(q, None, pos, (12, 12, 12))
    q[1, 0, 5] = math.nan
    q[2, 1, 40] = math.inf
    y, _ = vitq.rope_axes(q, None, pos, (12, 12, 12))
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, 0, [5, 41]] = True
    hit[2, 1, [4, 40]] = True
    assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], clean[~hit])


def test_captured_and_replayed_on_another_stream():
    q, k, pos = _randn(1, 100, 4, 72).to(BF), _randn(2, 100, 4, 72).to(BF), _pos(3, 100, 3, 60)
    want = vitq.rope_axes(q, k, pos, (12, 12, 12))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = vitq.rope_axes(q, k, pos, (12, 12, 12))
    q2 = _randn(9, 100, 4, 72).to(BF)
    q.copy_(q2)
    g.replay()
    torch.cuda.synchronize()
    ref = vitq.rope_axes(q2, k, pos, (12, 12, 12))
    assert torch.equal(y[0], ref[0]) and torch.equal(y[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vitq.rope_axes(q2, k, pos, (12, 12, 12), stream=side)
    side.synchronize()
    assert torch.equal(got[0], ref[0])


def test_offsets_past_32_bits():
    """More than 2^31 elements between the first and the last token (an 8.6 GB buffer)."""
    n, stride = 9, 2 ** 29 + 8
    buf = torch.empty(n * stride, dtype=BF, device="cuda")
    q = buf.as_strided((n, 2, 72), (stride, 72, 1))
    q.copy_(_randn(1, n, 2, 72))
    pos = _pos(2, n, 3, 50)
    x = q.clone()
    vitq.rope_axes_(q, None, pos, (12, 12, 12))
    _close(q, x, pos, (12, 12, 12))


def test_int8_projection_rotary_and_attention():
    """The pieces as they are used: INT8 QKV, rotary in place on its packed rows, attention, INT8 projection."""
    n, H = 256, 1152
    x = _randn(1, n, H).to(BF)
    g, b = (1 + 0.02 * _randn(2, H)).to(BF), (0.01 * _randn(3, H)).to(BF)
    w, wo = 0.02 * _randn(4, 3 * H, H), 0.02 * _randn(5, H, H)
    qw, qo = vitq.quant_int8(w), vitq.quant_int8(wo)
    qkv = vitq.int8_gemm(*vitq.ln_quant_int8(x, g, b), *qw)
    plain = qkv.double()
    i = torch.arange(n, device="cuda")
    pos = torch.stack([i // 64, i // 8 % 8, i % 8], 1).int()
    q, k = qkv[:, :H].view(n, 16, 72), qkv[:, H:2 * H].view(n, 16, 72)
    vitq.rope_axes_(q, k, pos, (12, 12, 12), axis_freq=True)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    att = vitq.attention_varlen(qkv, cu, n)
    y = vitq.int8_gemm(*vitq.quant_int8(att), *qo, residual=x)
    assert vitq.device_error() == 0
    kw = dict(sections=(12, 12, 12), axis_freq=True)
    rq = _ref(plain[:, :H].view(n, 16, 72), pos, **kw)[0]
    rk = _ref(plain[:, H:2 * H].view(n, 16, 72), pos, **kw)[0]
    v = plain[:, 2 * H:].view(n, 16, 72)
    p = torch.softmax(torch.einsum("ihd,jhd->hij", rq, rk) / math.sqrt(72), -1)
    o = torch.einsum("hij,jhd->ihd", p, v).reshape(n, H)
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()         # noqa: E731
    # q and k carry one bf16 rounding (2^-8 at most, 2^-9.8 rms), P another, the output a third
    assert rel(att, o) <= 1e-2
    # one int8 rounding of the attention (half a step of amax / 127 ~ 4 rms / 127) on top; y itself is rounded to
    # bf16 after the residual's add, by at most 2^-8 |y| an element and so 2^-8 ||y|| in the norm
    out = o @ (qo[0].double() * qo[1].double()[:, None]).t()
    assert (y.double() - x.double() - out).norm() <= 3e-2 * out.norm() + 2.0 ** -8 * y.double().norm()
