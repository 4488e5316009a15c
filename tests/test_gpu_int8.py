"""The INT8 row kernels and the INT8 GEMM against their definitions in 64 bits.

Codes and scales are compared bit for bit: s = fl32(amax / 127) is one IEEE division,
and the codes are the exact quotient's roundings.  GEMM outputs: the integer sum is exact,
and acc, sa * acc, the FMA with sw and bias, and the residual's add each round once in
fp32 (four roundings of at most 2^-24 of the largest magnitude met on the way), then one
rounding to the output type (half a step, finfo.eps / 2 of the value).
"""
import math

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _g(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(seed, *shape):
    return torch.randn(shape, generator=_g(seed), device="cuda")


def _rows(x, pad, shift=0):
    """x as a view into a wider buffer: `shift` elements in, `pad` unused elements a row."""
    buf = torch.full((x.shape[0], x.shape[1] + pad + shift), 3.0, dtype=x.dtype, device="cuda")
    buf[:, shift:shift + x.shape[1]] = x
    return buf[:, shift:shift + x.shape[1]]


def _codes_ref(y):
    """(codes, scales) of rows of y (any type), from the definition."""
    amax = y.abs().amax(1).float()
    # by a tensor: torch multiplies with the reciprocal of a number
    s = torch.where(torch.isfinite(amax), amax / torch.full_like(amax, 127), math.nan)
    q = torch.round(y.double() / s.double()[:, None])
    return torch.where((s > 0)[:, None], q, 0.0).clamp(-127, 127).to(torch.int8), s


def _bf16_of(y):
    """fp64 -> bf16 with one rounding (normal range)."""
    m, e = torch.frexp(y)
    return torch.ldexp(torch.round(m * 256), e - 8).to(BF)


def _same(got, want, what=""):
    q, s = got
    torch.cuda.synchronize()
    wq, ws = want
    assert torch.equal(s.nan_to_num(-1.0), ws.nan_to_num(-1.0)), f"{what}: scales differ"
    bad = (q != wq).nonzero()
    assert not len(bad), f"{what}: {len(bad)} codes differ, first at {bad[:3].tolist()}"
    assert vitq.device_error() == 0


# widths around every variant of the row kernel (chunks of 8 or 4 elements; 160, 256, 640,
# 1024, 2048 and 8192 chunks) and ragged ones
WIDTHS = [1, 7, 8, 9, 31, 255, 640, 1000, 1152, 1279, 2048, 2056, 4304, 4608, 5121, 8192, 8200, 16383, 65536]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("K", WIDTHS)
def test_quant_rows(dtype, K):
    M = 37 if K < 9000 else 3
    x = (_randn(K, M, K) * torch.exp(_randn(K + 1, M, 1))).to(dtype)
    _same(vitq.quant_int8(x), _codes_ref(x), f"{dtype} {K}")


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (24, 8), (5, 4)])
def test_quant_strided_and_unaligned_rows(dtype, pad, shift):
    x = _rows(_randn(5, 19, 333).to(dtype), pad, shift)
    _same(vitq.quant_int8(x), _codes_ref(x))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_quant_special_rows(dtype):
    """Zero rows, one element, infinities, NaN, the type's smallest and largest values."""
    top, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = _randn(11, 12, 200).to(dtype)
    x[0] = 0
    x[1] = -0.0
    x[2, 7] = math.inf
    x[3, 199] = -math.inf
    x[4, 100] = math.nan
    x[5] = 0
    x[5, 3] = -2.5
    x[6] = top
    x[7] = (x[7].float() * top / 8).to(dtype)
    x[8] = (x[8].double() * tiny / 64).to(dtype)       # subnormal values (and scales, in fp32 range)
    x[9] = torch.nextafter(torch.zeros((), device="cuda", dtype=F32), torch.ones((), device="cuda")).to(dtype)
    x[10] = (x[10].double() * tiny * 100).to(dtype)
    got, want = vitq.quant_int8(x), _codes_ref(x)
    _same(got, want)
    assert got[1][:2].tolist() == [0.0, 0.0] and got[1][2:5].isnan().all() and not got[0][:5].any()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_quant_values_on_and_next_to_ties(dtype):
    """Rows made of (k + 1/2) s and its neighbours, for scales with and without exact ties."""
    rows = []
    for amax in (127.0, 254.0, 1.0, 3.0, 96.5, 127 * 9.0, 127 * 13.0, 0.7, 1e-3):
        a = torch.tensor(amax, dtype=dtype).double()
        s = (a.float() / 127).double()
        t = (torch.arange(0, 127).double() + 0.5) * s
        v = t.to(dtype)
        near = [v, torch.nextafter(v, torch.tensor(math.inf, dtype=dtype)), torch.nextafter(v, torch.tensor(0.0, dtype=dtype))]
        row = torch.cat([torch.cat(near), -torch.cat(near), a.to(dtype).reshape(1)])
        rows.append(torch.where(row.abs().double() <= a, row, torch.zeros((), dtype=dtype)))
    x = torch.stack(rows).cuda()
    _same(vitq.quant_int8(x), _codes_ref(x))


def test_quant_every_bf16_pair_of_significands():
    """Every significand of amax against every bf16 magnitude down to 2^-9 of it."""
    sig = 1 + torch.arange(128, dtype=torch.float64) / 128
    vals = torch.cat([sig * 2.0 ** -e for e in range(10)])
    x = torch.where(vals[None, :] <= sig[:, None], vals[None, :], 0.0)
    x = torch.cat([sig[:, None], x], 1)
    for scale in (1.0, 2.0 ** 100, 2.0 ** -90, 2.0 ** -104):
        xs = (x * scale).to(BF).cuda()
        _same(vitq.quant_int8(xs), _codes_ref(xs), scale)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("start", [0, 1, 3, 7])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 5), (1, 17), (2, 9), (3, 1203), (2, 4303), (9, 40)])
def test_quant_rows_that_fill_their_storage(M, K, start, dtype):
    """Rows that start anywhere in a 16-byte unit, first and last row at the ends of the storage."""
    buf = torch.empty(start + M * K, dtype=dtype, device="cuda")
    x = buf[start:].view(M, K)
    x.copy_(_randn(K + start, M, K))
    _same(vitq.quant_int8(x), _codes_ref(x))
    if dtype == BF:
        g, b = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
        _same(vitq.ln_quant_int8(x, g, b), _codes_ref(_ln_ref(x, g, b, 1e-6)))
        _same(vitq.gelu_quant_int8(x), _codes_ref(_gelu_ref(x)))


@pytest.mark.parametrize("K", [65535, 65536, 20001, 16392, 16376, 2305, 1160])
def test_widest_rows(K):
    for dtype in (BF, HF, F32):
        x = _randn(K, 3, K).to(dtype)
        _same(vitq.quant_int8(x), _codes_ref(x), (K, dtype))
    x = (_randn(K, 3, K) + 0.5).to(BF)
    g, b = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    _same(vitq.ln_quant_int8(x, g, b), _codes_ref(_ln_ref(x, g, b, 1e-6)), K)
    _same(vitq.gelu_quant_int8(x), _codes_ref(_gelu_ref(x)), K)


@pytest.mark.parametrize("K", [40, 1152, 1153, 2056, 4608, 16392])
def test_ln_quant_not_finite_gamma_or_beta(K):
    """A NaN that only gamma or beta brings in (or 0 * infinity) marks every row it reaches."""
    x = _randn(3, 5, K).to(BF)
    x[3] = 1.25                                     # x - mean = 0
    one, zero = torch.ones(K, dtype=BF, device="cuda"), torch.zeros(K, dtype=BF, device="cuda")
    for col in (0, K // 2, K - 1):
        for v in (float("nan"), float("inf"), -float("inf")):
            for w in (one, zero):
                bad = w.clone()
                bad[col] = v
                q, s = vitq.ln_quant_int8(x, *((bad, zero) if w is one else (one, bad)))
                assert torch.isnan(s).all() and (q == 0).all(), (col, v, w is one)


def test_ln_quant_unaligned_gamma_and_beta():
    K = 1152
    x = _randn(1, 50, K).to(BF)
    gb = (1 + 0.1 * _randn(2, 2 * K + 3)).to(BF)
    gamma, beta = gb[1:K + 1], gb[K + 2:2 * K + 2]
    _same(vitq.ln_quant_int8(x, gamma, beta), _codes_ref(_ln_ref(x, gamma, beta, 1e-6)))


def test_quant_leaves_the_rest_of_its_outputs():
    x = _randn(3, 5, 100).to(BF)
    buf, s = torch.full((7, 128), 99, dtype=torch.int8, device="cuda"), torch.full((7,), -1.0, device="cuda")
    vitq.quant_int8(x, out=(buf[1:6, :100], s[1:6]))
    _same((buf[1:6, :100], s[1:6]), _codes_ref(x))
    assert (buf[0] == 99).all() and (buf[6] == 99).all() and (buf[:, 100:] == 99).all() and s[0] == s[6] == -1


@pytest.mark.parametrize("fn", ["quant", "ln", "gelu", "gemm"])
def test_no_rows(fn):
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    if fn == "gemm":
        q = torch.empty((0, 64), dtype=torch.int8, device="cuda")
        y = vitq.int8_gemm(q, torch.empty(0, device="cuda"), torch.zeros((8, 64), dtype=torch.int8, device="cuda"),
                           torch.zeros(8, device="cuda"))
        assert y.shape == (0, 8)
        return
    q, s = {"quant": lambda: vitq.quant_int8(x), "ln": lambda: vitq.ln_quant_int8(x, w, w),
            "gelu": lambda: vitq.gelu_quant_int8(x)}[fn]()
    assert q.shape == (0, 64) and s.shape == (0,)


# ------------------------------------------------------------------ LayerNorm, GELU
def _ln_ref(x, gamma, beta, eps):
    x = x.double()
    c = x - x.mean(1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * gamma.double() + beta.double()
    return _bf16_of(y)


@pytest.mark.parametrize("M,K,pad", [(1, 1152, 0), (2, 1, 0), (3, 2, 0), (300, 1152, 0), (41, 1152, 3), (64, 4608, 0),
                                     (1000, 264, 8), (17, 2049, 7), (5, 9000, 0), (2, 65536, 0), (2000, 72, 0)])
def test_ln_quant(M, K, pad):
    x = _rows((_randn(M + K, M, K) * torch.exp(_randn(K, M, 1)) + _randn(M, M, 1)).to(BF), pad)
    gamma, beta = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    _same(vitq.ln_quant_int8(x, gamma, beta), _codes_ref(_ln_ref(x, gamma, beta, 1e-6)), (M, K))


def test_ln_quant_far_means_constant_and_broken_rows():
    K = 1152
    x = _randn(7, 64, K)
    x[0] = 3.0                                     # variance 0: y = beta
    x[1] = 0.0
    x[2] = 1000 + 8 * torch.round(x[2])            # mean far above the spread
    x[3] = 1.0
    x[3, 5] = 1.0078125                            # one neighbour of an otherwise constant row
    x[4] *= 1e30
    x[5] *= 1e-30
    x[6, 9] = math.inf
    x[7, 9] = math.nan
    x[8, 0] = 3e38
    x[8, 1] = -3e38
    x[9] = -1.0
    x[9, 1151] = 16384.0                           # one massive channel
    x[10] = x[10] * 1e-4 + 100.0                   # rounds to few distinct values
    x = x.to(BF)
    gamma, beta = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    for b in (beta, torch.zeros_like(beta)):
        want = _codes_ref(_ln_ref(x, gamma, b, 1e-6))
        got = vitq.ln_quant_int8(x, gamma, b)
        _same(got, want)
        assert got[1][6:8].isnan().all() and not got[0][6:8].any()
    q, s = vitq.ln_quant_int8(x[4:6], gamma, beta, eps=0.0)
    _same((q, s), _codes_ref(_ln_ref(x[4:6], gamma, beta, 0.0)))


def _gelu_ref(f):
    x = f.double()
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return _bf16_of(x / (1 + torch.exp(-2 * u)))


@pytest.mark.parametrize("M,K,pad", [(1, 4304, 0), (3, 1, 0), (200, 4304, 0), (33, 4304, 5), (40, 4608, 0), (2, 65536, 0),
                                     (500, 96, 8), (7, 9001, 0)])
def test_gelu_quant(M, K, pad):
    f = _rows((_randn(M * K, M, K) * 2).to(BF), pad)
    _same(vitq.gelu_quant_int8(f), _codes_ref(_gelu_ref(f)), (M, K))


def test_gelu_quant_every_finite_bf16():
    """Every finite value, in rows of neighbours (so that each is near its row's largest)."""
    bits = torch.arange(65536, dtype=torch.int32)
    v = (bits << 16).view(F32)
    v = v[torch.isfinite(v)].to(BF).cuda()
    v = v[torch.argsort(v.float())].reshape(-1, 128)
    y = _gelu_ref(v)
    keep = (y.abs().amax(1).float() >= 2.0 ** -120)      # the reference's rounding is for normal bf16 values
    got = vitq.gelu_quant_int8(v)
    _same((got[0][keep], got[1][keep]), _codes_ref(y[keep]))
    # one row a binade: about 247 of positive values, and 122 of negative ones before GELU underflows at -10
    assert keep.sum() > 360


def test_gelu_quant_infinity_and_nan():
    f = _randn(1, 4, 64).to(BF)
    f[0, 3], f[1, 5], f[2, 63] = math.inf, -math.inf, math.nan
    q, s = vitq.gelu_quant_int8(f)
    assert s[:3].isnan().all() and not q[:3].any() and s[3] > 0


# ------------------------------------------------------------------ GEMM
def _i8(seed, m, k, full=True):
    q = torch.full((m, (k + 15) // 16 * 16), 77, dtype=torch.int8, device="cuda")   # what lies behind K must not count
    q[:, :k] = torch.randint(-127, 128, (m, k), generator=_g(seed), device="cuda", dtype=torch.int8)
    return q[:, :k]


def _gemm_check(M, N, K, t, bias=False, residual=False, out=None, res=None):
    qa, qw = _i8(M + K, M, K), _i8(N + K + 1, N, K)
    sa = torch.exp(_randn(1, M)) * 1e-2
    sw = torch.exp(_randn(2, N)) * 1e-3
    b = _randn(3, N).to(t) if bias else None
    r = res if res is not None else (_randn(4, M, N).to(t) if residual else None)
    want = (qa.double() @ qw.double().t()) * sa.double()[:, None] * sw.double()[None, :]
    mag = want.abs()
    for e in (b, r):
        if e is not None:
            want = want + e.double()
            mag = mag + e.double().abs()
    y = vitq.int8_gemm(qa, sa, qw, sw, bias=b, residual=r, out=out, out_dtype=t)
    assert vitq.device_error() == 0
    tol = 4 * 2.0 ** -24 * mag + torch.finfo(t).eps / 2 * (want.abs() + 4 * 2.0 ** -24 * mag)
    if t == HF:   # spacing of subnormal fp16 values
        tol = tol + 2.0 ** -25
    off = (y.double() - want).abs() - tol
    assert (off <= 0).all(), f"{(M, N, K, t)}: {int((off > 0).sum())} outputs off, worst {off.max().item():.3e}"
    return y


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 1, 1), (1, 4608, 4608), (2, 129, 65), (3, 257, 1152), (5, 1152, 4304),
                                   (8, 64, 200), (9, 100, 100), (16, 2048, 1000), (17, 300, 31), (31, 1152, 1152),
                                   (64, 3456, 1152), (100, 37, 4304), (128, 256, 128), (129, 257, 129), (243, 2048, 4608),
                                   (300, 4304, 1152), (1000, 72, 640)])
def test_gemm(M, N, K, t):
    _gemm_check(M, N, K, t)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 1152, 1152), (4, 33, 80), (40, 130, 320), (200, 384, 640), (333, 1152, 1152)])
def test_gemm_bias_and_residual(M, N, K, t):
    _gemm_check(M, N, K, t, bias=True)
    _gemm_check(M, N, K, t, bias=True, residual=True)
    _gemm_check(M, N, K, t, residual=True)


# shapes for each kernel behind int8_gemm: few rows (by 8, 16, 16 x 32 channels, 32), a tile split over
# 2, 4 and 8 CTAs at both widths, single tiles, pairs with short and long sums; whole and odd N and K
VARIANTS = [(8, 64, 200), (7, 4607, 4603), (16, 2048, 1000), (33, 1152, 1152), (40, 4200, 1152), (24, 4608, 4608),
            (100, 100, 700), (128, 512, 512), (127, 515, 509), (64, 4608, 4608), (129, 900, 4304), (512, 2048, 4608),
            (500, 2049, 4607), (243, 2048, 4608), (250, 2043, 4601), (128, 1152, 4304), (121, 1101, 5001),
            (300, 4304, 1152), (301, 4303, 1151), (2000, 300, 300), (5000, 2688, 200), (5001, 2689, 203),
            (2100, 1156, 1100), (3001, 2690, 900), (70000, 8, 16)]


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("M,N,K", VARIANTS)
def test_gemm_every_kernel(M, N, K, t):
    _gemm_check(M, N, K, t, bias=True, residual=True)


@pytest.mark.parametrize("M,N,K", [(5, 40, 50), (20, 40, 50), (130, 40, 50), (300, 264, 205)])
def test_gemm_operands_that_end_with_their_last_row(M, N, K):
    """Row pitch 64 (208), but storage that ends right behind the last row's last code."""
    ld = (K + 15) // 16 * 16
    qa, qw = _i8(1, M, K), _i8(2, N, K)
    def tight(q):
        buf = torch.zeros((q.shape[0] - 1) * ld + K, dtype=torch.int8, device="cuda")
        v = buf.as_strided(q.shape, (ld, 1))
        v.copy_(q)
        return v
    sa, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    assert torch.equal(vitq.int8_gemm(tight(qa), sa, tight(qw), sw), vitq.int8_gemm(qa, sa, qw, sw))


@pytest.mark.parametrize("M", [2, 40, 150, 700])
def test_gemm_largest_width(M):
    """N and K at the entry point's limit (65536), rows of weights of one shared value."""
    N, K = 65536, 64
    qa = _i8(1, M, K)
    qw = _i8(2, N, K)
    sa, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    y = vitq.int8_gemm(qa, sa, qw, sw, out_dtype=F32)
    want = (qa.double() @ qw.double().t()) * sa.double()[:, None] * sw.double()
    assert ((y.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("M,N,K", [(6256, 1152, 1152), (2500, 3456, 1152), (1564, 4608, 4608)])
def test_gemm_many_tiles(M, N, K):
    _gemm_check(M, N, K, BF, bias=True, residual=True)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("M", [3, 20, 150])
@pytest.mark.parametrize("pad,shift", [(0, 0), (16, 8), (3, 1), (1, 0)])
def test_gemm_strided_output_and_residual(M, t, pad, shift):
    N, K = 133, 192
    buf = torch.full((M + 2, N + pad + shift), 5.0, dtype=t, device="cuda")
    out = buf[1:M + 1, shift:shift + N]
    _gemm_check(M, N, K, t, bias=True, res=_rows(_randn(9, M, N).to(t), pad, shift), out=out)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:M + 1, shift:shift + N] = False
    assert (buf[keep] == 5.0).all(), "wrote outside C"


@pytest.mark.parametrize("M", [2, 70, 300])
def test_gemm_residual_may_be_the_output(M):
    N, K = 1152, 640
    qa, qw, sa, sw = _i8(1, M, K), _i8(2, N, K), torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    x = _randn(3, M, N).to(BF)
    want = vitq.int8_gemm(qa, sa, qw, sw, residual=x)
    vitq.int8_gemm(qa, sa, qw, sw, residual=x, out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("M", [1, 7, 40, 140])
def test_gemm_sums_are_exact_integers(M):
    """Largest codes over the widest K: the sum passes 2^29 and odd sums above 2^24 stay exact until
    the conversion to fp32 (one rounding)."""
    N, K = 24, 65536
    qa = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    qw = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    qa[:, ::3] = 127
    qw[:, 0] = torch.arange(N, device="cuda", dtype=torch.int8)
    y = vitq.int8_gemm(qa, torch.ones(M, device="cuda"), qw, torch.ones(N, device="cuda"), out_dtype=F32)
    assert torch.equal(y, (qa.double() @ qw.double().t()).to(F32))


@pytest.mark.parametrize("M", [2, 50, 200])
def test_gemm_row_does_not_depend_on_its_batch(M):
    """A packed batch equals its images run alone, bit for bit, at every size (integer sums)."""
    N, K = 700, 1152
    qa, qw, sw = _i8(1, M, K), _i8(2, N, K), torch.rand(N, device="cuda")
    sa = torch.rand(M, device="cuda")
    whole = vitq.int8_gemm(qa, sa, qw, sw, out_dtype=F32)
    big = vitq.int8_gemm(qa.repeat(40, 1), sa.repeat(40), qw, sw, out_dtype=F32)
    assert torch.equal(big.view(40, M, N), whole.expand(40, M, N))
    assert torch.equal(vitq.int8_gemm(qa[:1], sa[:1], qw, sw, out_dtype=F32), whole[:1])


def test_gemm_nan_rows_and_infinite_scales_stay_in_their_rows():
    for M in (4, 90, 200):
        qa, qw, sa, sw = _i8(1, M, 96), _i8(2, 50, 96), torch.rand(M, device="cuda"), torch.rand(50, device="cuda")
        sa[1], qa[1] = math.nan, 0
        y = vitq.int8_gemm(qa, sa, qw, sw)
        assert y[1].isnan().all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def _chain(x, p, n_heads=16):
    """The INT8 linears of a block as they are used, with the library's own quantisers."""
    q, s = vitq.ln_quant_int8(x, p["g"], p["b"])
    f = vitq.int8_gemm(q, s, p["w1"][0], p["w1"][1], bias=p["b1"])
    q, s = vitq.gelu_quant_int8(f)
    return vitq.int8_gemm(q, s, p["w2"][0], p["w2"][1], bias=p["b2"], residual=x)


def _mlp(seed=0):
    H, F = 1152, 4304
    return dict(g=(1 + 0.02 * _randn(seed, H)).to(BF), b=(0.01 * _randn(seed + 1, H)).to(BF),
                w1=vitq.quant_int8(0.02 * _randn(seed + 2, F, H)), b1=(0.01 * _randn(seed + 3, F)).to(BF),
                w2=vitq.quant_int8(0.02 * _randn(seed + 4, H, F)), b2=(0.01 * _randn(seed + 5, H)).to(BF))


@pytest.mark.parametrize("M", [1, 30, 256, 972])
def test_mlp_chain(M):
    """LayerNorm -> fc1 -> GELU -> fc2 + residual, stage by stage on the GPU's own inputs, then as one run."""
    p, x = _mlp(), _randn(50, M, 1152).to(BF)
    q, s = vitq.ln_quant_int8(x, p["g"], p["b"])
    _same((q, s), _codes_ref(_ln_ref(x, p["g"], p["b"], 1e-6)))
    f = vitq.int8_gemm(q, s, p["w1"][0], p["w1"][1], bias=p["b1"])
    q2, s2 = vitq.gelu_quant_int8(f)
    _same((q2, s2), _codes_ref(_gelu_ref(f)))
    want = (q2.double() @ p["w2"][0].double().t()) * s2.double()[:, None] * p["w2"][1].double() + p["b2"].double() + x.double()
    y = _chain(x, p)
    mag = want.abs() + x.double().abs() + p["b2"].double().abs()
    assert ((y.double() - want).abs() <= 4 * 2.0 ** -24 * mag * 4 + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("M", [4, 256])
def test_chain_captured_replayed_and_on_another_stream(M):
    p, x = _mlp(7), _randn(51, M, 1152).to(BF)
    want = _chain(x, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _chain(x, p)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    given = vitq.int8_gemm(*vitq.quant_int8(x, stream=side), *p["w1"], stream=side)   # stream as an argument
    side.synchronize()
    assert torch.equal(given, vitq.int8_gemm(*vitq.quant_int8(x), *p["w1"]))
    static = x.clone()
    graphs = []
    for _ in range(2):                                   # two graphs of the same call, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = _chain(static, p)
        graphs.append((g, y))
    for k in range(3):
        new = _randn(60 + k, M, 1152).to(BF)
        static.copy_(new)
        for g, y in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref = _chain(new, p)
        assert all(torch.equal(y, ref) for _, y in graphs)


def test_two_streams_at_once():
    p, xs = _mlp(9), [_randn(70 + i, 200, 1152).to(BF) for i in range(2)]
    want = [_chain(x, p) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _chain(xs[i], p)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ more rows than run at once, far offsets
@pytest.mark.parametrize("M,K", [(5000, 1152), (5001, 1001), (5003, 2304), (3000, 4304), (2501, 4303), (1300, 9000), (1301, 9001),
                                 (700, 18000), (701, 17999), (400, 24000), (401, 24001)])
def test_gelu_quant_more_rows_than_run_at_once(M, K):
    f = (_randn(M, M, K) * torch.exp(_randn(K, M, 1))).to(BF)
    _same(vitq.gelu_quant_int8(f), _codes_ref(_gelu_ref(f)), (M, K))


@pytest.mark.parametrize("M,K", [(20001, 1152), (10001, 264), (10003, 1151), (5000, 2000), (5003, 2001), (1500, 4608),
                                 (1503, 4607), (450, 16000), (451, 15999)])
def test_ln_quant_more_rows_than_run_at_once(M, K):
    x = (_randn(M, M, K) * torch.exp(_randn(K, M, 1)) + _randn(M + 1, M, 1)).to(BF)
    gamma, beta = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    _same(vitq.ln_quant_int8(x, gamma, beta), _codes_ref(_ln_ref(x, gamma, beta, 1e-6)), (M, K))


FAR_ROWS, FAR_STRIDE = 33001, 65536 + 16        # 2.16e9 elements from the first row to the last


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("fn", ["quant", "ln", "gelu"])
def test_rows_past_32_bit_offsets(fn, pad):
    """Rows of x and of the codes more than 2^31 elements apart (4.3 and 2.2 GB); pad: a stride of any alignment."""
    ld, K = FAR_STRIDE + pad, 72
    x = torch.empty(FAR_ROWS * ld, dtype=BF, device="cuda").as_strided((FAR_ROWS, K), (ld, 1))
    x.copy_(_randn(3, FAR_ROWS, K))
    out = (torch.empty(FAR_ROWS * FAR_STRIDE, dtype=torch.int8, device="cuda").as_strided((FAR_ROWS, K), (FAR_STRIDE, 1)),
           torch.empty(FAR_ROWS, device="cuda"))
    w = torch.ones(K, dtype=BF, device="cuda")
    call = {"quant": vitq.quant_int8, "gelu": vitq.gelu_quant_int8,
            "ln": lambda a, out=None: vitq.ln_quant_int8(a, w, w, out=out)}[fn]
    want = call(x.contiguous())
    got = call(x, out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("N,K", [(40, 200), (264, 640)])
def test_gemm_past_32_bit_offsets(N, K, pad):
    """A, the residual and C with rows more than 2^31 elements apart (2.2, 4.3 and 4.3 GB)."""
    M, ld = FAR_ROWS, FAR_STRIDE + pad
    far = torch.empty(M * FAR_STRIDE, dtype=torch.int8, device="cuda").as_strided((M, K), (FAR_STRIDE, 1))
    qa, qw = _i8(1, M, K), _i8(2, N, K)
    far.copy_(qa)
    sa, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    r, c = (torch.empty(M * ld, dtype=BF, device="cuda").as_strided((M, N), (ld, 1)) for _ in range(2))
    r.copy_(_randn(4, M, N))
    want = vitq.int8_gemm(qa, sa, qw, sw, residual=r.contiguous())
    assert torch.equal(vitq.int8_gemm(far, sa, qw, sw, residual=r, out=c), want)
    assert vitq.device_error() == 0
