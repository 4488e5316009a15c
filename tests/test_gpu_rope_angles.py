"""The several-axis rotary: angles of fp32 tensors, the most tokens, and what lies around the heads.

Tolerance of the angles' test: cos and sin are fp32 roundings of the exact angle's, off by 2^-24 of themselves;
vb sin and the last FMA round once each, so |y - want| <= 2^-24 (|va cos| + 2 |vb sin| + |want|), want itself
being at most |va cos| + |vb sin|.  The angle is pos times a frequency made by up to 128 products in fp64: off by
2^-45 of the angle.
"""
import pytest
import torch

from quantized_vit_encoder_b200 import vitq

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("far", [0, 300, 10 ** 5])
@pytest.mark.parametrize("sections", [(24, 20, 20), (12, 12, 12), (18, 17), (9, 10, 11, 3)])
def test_fp32_angles(sections, far, inverse, adjacent):
    n, pairs = 300, sum(sections)
    g = torch.Generator(device="cuda").manual_seed(far + pairs)
    pos = torch.randint(-far, far + 1, (n, len(sections)), generator=g, device="cuda", dtype=torch.int32)
    x = _randn(far, n, 3, 2 * pairs)
    x[:, 1, :pairs] = 0                                # where one product is 0, the other's angle shows
    x[:, 2, pairs:] = 0
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    freq = torch.tensor([10000.0 ** (-j / pairs) for j in range(pairs)], dtype=torch.float64, device="cuda")
    ang = (pos.double()[:, axis] * freq)[:, None]
    c, s = torch.cos(ang), torch.sin(ang) * (-1 if inverse else 1)
    ia, ib = (slice(0, None, 2), slice(1, None, 2)) if adjacent else (slice(0, pairs), slice(pairs, None))
    a, b = x[..., ia].double(), x[..., ib].double()
    y, _ = vitq.rope_axes(x, None, pos, sections, inverse=inverse, adjacent=adjacent)
    for got, u, v in ((y[..., ia], a * c, -b * s), (y[..., ib], b * c, a * s)):
        tol = 2.0 ** -24 * (2 * u.abs() + 3 * v.abs()) + 2.0 ** -45 * ang.abs() * (a.abs() + b.abs())
        off = (got.double() - (u + v)).abs() - tol
        assert (off <= 0).all(), f"{int((off > 0).sum())} of {off.numel()} off, worst {off.max().item():.3e}"


def test_most_tokens():
    """2^24 tokens, the entry point's limit, of one narrow head; every token is one of 1000."""
    n, few = 1 << 24, _randn(1, 1000, 1, 8).bfloat16()
    pos = torch.arange(1000, device="cuda", dtype=torch.int32)[:, None]
    want, _ = vitq.rope_axes(few, None, pos, (3,))
    times = -(-n // 1000)
    y, _ = vitq.rope_axes(few.repeat(times, 1, 1)[:n], None, pos.repeat(times, 1)[:n], (3,))
    assert torch.equal(y, want.repeat(times, 1, 1)[:n])


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("sections,d,gap", [((24, 20, 20), 128, 8), ((24, 20, 20), 144, 16), ((12, 12, 12), 72, 4),
                                            ((12, 12, 12), 84, 4), ((9, 9), 40, 2), ((5,), 11, 1), ((5,), 10, 3)])
def test_nothing_around_the_heads_is_written(sections, d, gap, adjacent, t):
    """Heads of q and k between sentinels, at each width of access, out of place and in place."""
    n, hq, hk = 37, 3, 2
    row = (hq + hk) * (d + gap) + gap
    x = torch.full((n, row), 7.0, device="cuda").to(t)
    q = x.as_strided((n, hq, d), (row, d + gap, 1), gap)
    k = x.as_strided((n, hk, d), (row, d + gap, 1), gap + hq * (d + gap))
    q.copy_(_randn(1, n, hq, d))
    k.copy_(_randn(2, n, hk, d))
    pos = torch.arange(n * len(sections), device="cuda", dtype=torch.int32).view(n, len(sections))
    want = vitq.rope_axes(q.contiguous(), k.contiguous(), pos, sections, adjacent=adjacent)
    before, inside = x.clone(), torch.zeros(n, row, dtype=torch.bool, device="cuda")
    for v in (q, k):
        inside.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(True)
    out = torch.full_like(x, 5.0)
    oq, ok = (out.as_strided(v.shape, v.stride(), v.storage_offset()) for v in (q, k))
    vitq.rope_axes(q, k, pos, sections, adjacent=adjacent, out=(oq, ok))
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and (out[~inside] == 5.0).all() and torch.equal(x, before)
    vitq.rope_axes_(q, k, pos, sections, adjacent=adjacent)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[~inside], before[~inside])
