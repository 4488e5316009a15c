"""Each kernel behind int8_gemm at what is hard on it: the residual in place, rows of C and of the residual
anywhere, scales that are not finite, sums past 2^24, operands that end with their last code, capture.

The shapes below take one kernel each by the library's own choice, which a CPU test checks, so that a change
of the choice cannot leave a kernel without its tests.  Tolerances: the integer sum is exact; fl(sum) * sa, the
FMA with sw and bias, and the residual's add each round once in fp32 (four roundings of at most 2^-24 of the
largest magnitude on the way), then one rounding to the type (finfo.eps / 2 of the value).
"""
import math
import os
import shutil
import subprocess

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# kernel -> (M, N, K), N a multiple of 8; one column fewer takes the same kernel, with rows of C off 16 bytes
SHAPES = {
    "kRows11": (7, 200, 303), "kRows21": (30, 1160, 1000), "kRows22": (40, 4208, 1152), "kRows41": (100, 104, 1100),
    "kSplit64x2": (60, 4608, 4600), "kSplit64x4": (129, 904, 4303), "kSplit128x2": (500, 2048, 4607),
    "kSplit128x4": (243, 2048, 4600), "kSplit128x8": (121, 1104, 5001), "kTile": (301, 4304, 1151),
    "kPairs": (2100, 1160, 1100), "kPairs, short sums": (5001, 2688, 203),
}
EDGES = {"kTile": [(1030, 1, 16), (2000, 3, 1), (1025, 129, 1), (1500, 24, 65536)], "kPairs": [(30000, 1000, 1)],
         "kSplit128x8": [(200, 200, 65536)]}


def test_shapes_take_their_kernels(tmp_path):
    """The library's choice on a B200 (148 SMs), from the header that it is compiled from."""
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    want = [(k.split(",")[0], (m, n - off, kk)) for k, (m, n, kk) in SHAPES.items() for off in (0, 1, 4)]
    want += [(k, s) for k, shapes in EDGES.items() for s in shapes]
    src = '#include <cstdio>\n#include "int8_choose.h"\nusing namespace vitq;\nint main() {\n' + "".join(
        f'  std::printf("%d\\n", i8_choose({m}, {n}, {k}, 148) == {kernel});\n' for kernel, (m, n, k) in want) + "}\n"
    (tmp_path / "c.cpp").write_text(src)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "quantized_vit_encoder_b200", "csrc"), str(tmp_path / "c.cpp"),
                    "-o", str(tmp_path / "c")], check=True)
    got = subprocess.run([str(tmp_path / "c")], capture_output=True, text=True, check=True).stdout.split()
    assert [w for w, ok in zip(want, got) if ok != "1"] == [] and len(got) == len(want)


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _i8(seed, m, k):
    q = torch.full((m, (k + 15) // 16 * 16), 77, dtype=torch.int8, device="cuda")   # what lies behind K must not count
    g = torch.Generator(device="cuda").manual_seed(seed)
    q[:, :k] = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    return q[:, :k]


def _operands(M, N, K):
    return _i8(M + K, M, K), torch.exp(_randn(1, M)) * 1e-2, _i8(N + K + 1, N, K), torch.exp(_randn(2, N)) * 1e-3


def _check(y, ops, bias=None, residual=None):
    """y against the definition in 64 bits."""
    qa, sa, qw, sw = ops
    want = (qa.double() @ qw.double().t()) * sa.double()[:, None] * sw.double()
    mag = want.abs()
    for e in (bias, residual):
        if e is not None:
            want = want + e.double()
            mag = mag + e.double().abs()
    tol = 4 * 2.0 ** -24 * mag + torch.finfo(y.dtype).eps / 2 * (want.abs() + 4 * 2.0 ** -24 * mag)
    tol = tol + (2.0 ** -25 if y.dtype == HF else 0.0)      # spacing of subnormal fp16 values
    off = (y.double() - want).abs() - tol
    assert (off <= 0).all(), f"{int((off > 0).sum())} outputs off, worst {off.max().item():.3e}"
    assert vitq.device_error() == 0


def _placed(M, N, t, pad, shift):
    """A buffer of sentinels, [M, N] inside it, and a mask of what lies around."""
    buf = torch.full((M + 2, N + pad + shift), 5.0, dtype=t, device="cuda")
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:M + 1, shift:shift + N] = False
    return buf, buf[1:M + 1, shift:shift + N], keep


# columns fewer, padding and start of the rows of C: whole 16-byte units, rows that start anywhere, and (1, 1, 0),
# (1, 9, 8), (4, 4, 0): rows that start on 16 bytes and end inside a unit that holds something else
PLACES = [(0, 0, 0), (0, 16, 8), (1, 0, 0), (0, 3, 1), (1, 1, 0), (1, 9, 8), (4, 4, 0), (1, 5, 4)]


@gpu
@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("less,pad,shift", PLACES)
@pytest.mark.parametrize("kernel", SHAPES)
def test_residual_in_place_and_nothing_around_it(kernel, less, pad, shift, t):
    """x += A W^T with x anywhere; the elements around x stay, and the result is that of a C of its own."""
    M, N, K = SHAPES[kernel]
    N -= less
    ops, bias = _operands(M, N, K), _randn(3, N).to(t)
    x = _randn(4, M, N).to(t)
    want = vitq.int8_gemm(*ops, bias=bias, residual=x, out_dtype=t)
    _check(want, ops, bias, x)
    buf, view, keep = _placed(M, N, t, pad, shift)
    view.copy_(x)
    vitq.int8_gemm(*ops, bias=bias, residual=view, out=view)
    assert torch.equal(view, want) and (buf[keep] == 5.0).all() and vitq.device_error() == 0


@gpu
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("c_place,r_place", [((0, 0), (3, 1)), ((3, 1), (0, 0)), ((2, 2), (5, 3)), ((7, 1), None)])
@pytest.mark.parametrize("kernel", SHAPES)
def test_output_and_residual_of_different_alignments(kernel, c_place, r_place, t):
    M, N, K = SHAPES[kernel]
    ops, res = _operands(M, N, K), None
    buf, out, keep = _placed(M, N, t, *c_place)
    if r_place is not None:
        rbuf, res, rkeep = _placed(M, N, t, *r_place)
        res.copy_(_randn(4, M, N))
        before = rbuf.clone()
    vitq.int8_gemm(*ops, residual=res, out=out)
    _check(out, ops, None, res)
    assert (buf[keep] == 5.0).all() and (r_place is None or torch.equal(rbuf, before))


@gpu
@pytest.mark.parametrize("kernel,shape", [(k, s) for k, shapes in EDGES.items() for s in shapes])
@pytest.mark.parametrize("t", [BF, F32])
def test_edges(kernel, shape, t):
    M, N, K = shape
    ops, res = _operands(M, N, K), _randn(4, M, N).to(t)
    _check(vitq.int8_gemm(*ops, residual=res, out_dtype=t), ops, None, res)


@gpu
@pytest.mark.parametrize("less", [0, 1])
@pytest.mark.parametrize("kernel", SHAPES)
def test_scales_that_are_not_finite_stay_in_their_row_or_column(kernel, less):
    M, N, K = SHAPES[kernel]
    N -= less
    qa, sa, qw, sw = _operands(M, N, K)
    clean = vitq.int8_gemm(qa, sa, qw, sw, out_dtype=F32)
    rows, cols = [0, M // 2, M - 1], [0, N // 2, N - 1]
    sa, sw = sa.clone(), sw.clone()
    sa[rows] = torch.tensor([math.nan, math.inf, math.inf], device="cuda")
    sw[cols] = torch.tensor([math.inf, math.nan, math.inf], device="cuda")
    qa[rows[0]] = 0                                   # a quantiser's row with a NaN
    qa[rows[2]] = 0                                   # 0 times infinity
    y = vitq.int8_gemm(qa, sa, qw, sw, out_dtype=F32)
    acc = (qa.double() @ qw.double().t()).float()
    want = acc * sa[:, None] * sw
    odd = torch.zeros_like(y, dtype=torch.bool)
    odd[rows], odd[:, cols] = True, True
    assert not torch.isfinite(y[odd]).any() and torch.equal(y[odd].nan_to_num(7.0), want[odd].nan_to_num(7.0))
    assert torch.equal(y[~odd], clean[~odd]) and vitq.device_error() == 0


@gpu
@pytest.mark.parametrize("kernel,shape", list(SHAPES.items()) + [("kTile", (1500, 24, 65536)), ("kSplit128x8", (200, 200, 65536))])
def test_sums_are_exact_integers(kernel, shape):
    """Largest codes, so that from K = 1041 on most sums are above 2^24, odd ones among them: exact until
    the one rounding to fp32."""
    M, N, K = shape
    qa, qw = _i8(1, M, K), _i8(2, N, K)
    qa.copy_(torch.where(qa < -100, 126, 127))
    qw.copy_(torch.where(qw < -100, -127, -128))
    qw[:, 0] = (torch.arange(N, device="cuda") % 120).to(torch.int8)
    one = torch.ones(max(M, N), device="cuda")
    acc = qa.double() @ qw.double().t()
    if K > 1040:
        big = acc.abs() > 2 ** 24
        assert big.any() and (acc[big] % 2 != 0).any()
    assert torch.equal(vitq.int8_gemm(qa, one[:M], qw, one[:N], out_dtype=F32), acc.to(F32))
    assert vitq.device_error() == 0


@gpu
@pytest.mark.parametrize("kernel", SHAPES)
def test_operands_that_end_with_their_last_code(kernel):
    M, N, K = SHAPES[kernel]
    K -= K % 16 == 0                                  # rows that end inside their last 16 bytes
    qa, sa, qw, sw = _operands(M, N, K)

    def tight(q):
        ld = (K + 15) // 16 * 16
        v = torch.zeros((q.shape[0] - 1) * ld + K, dtype=torch.int8, device="cuda").as_strided(q.shape, (ld, 1))
        return v.copy_(q)
    assert torch.equal(vitq.int8_gemm(tight(qa), sa, tight(qw), sw), vitq.int8_gemm(qa, sa, qw, sw))


@gpu
def test_row_does_not_depend_on_the_kernel():
    """The same tokens alone, in few rows, split along K, in tiles and in pairs: equal bits."""
    for kernel in ("kSplit64x4", "kSplit128x2", "kSplit128x4", "kSplit128x8", "kTile"):
        M, N, K = SHAPES[kernel]
        qa, sa, qw, sw = _operands(M, N, K)
        whole = vitq.int8_gemm(qa, sa, qw, sw, out_dtype=F32)
        times = -(-6000 // M)
        batch = _i8(1, times * M, K).copy_(qa.repeat(times, 1))
        many = vitq.int8_gemm(batch, sa.repeat(times), qw, sw, out_dtype=F32)
        assert torch.equal(many.view(times, M, N), whole.expand(times, M, N)), kernel
        for few in (1, 5, 40):
            assert torch.equal(vitq.int8_gemm(qa[:few], sa[:few], qw, sw, out_dtype=F32), whole[:few]), kernel


@gpu
@pytest.mark.parametrize("t", [BF, F32])
def test_products_that_underflow_have_the_same_sign_in_every_kernel(t):
    """Below 2^-150 a product becomes a zero of its sign."""
    for kernel in ("kSplit64x4", "kSplit128x4", "kTile", "kPairs", "kRows41"):
        M, N, K = SHAPES[kernel]
        qa, sa, qw, sw = _operands(M, N, K)
        y = vitq.int8_gemm(qa, sa * 1e-26, qw, sw * 1e-26, out_dtype=t)
        few = vitq.int8_gemm(qa[:5], sa[:5] * 1e-26, qw, sw * 1e-26, out_dtype=t)
        assert not y.any() and torch.signbit(y).any() and torch.equal(torch.signbit(y[:5]), torch.signbit(few)), kernel


@gpu
def test_every_kernel_in_one_graph_and_on_two_streams():
    ops = {k: _operands(*s) for k, s in SHAPES.items()}
    want = {k: vitq.int8_gemm(*o) for k, o in ops.items()}
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, {k: vitq.int8_gemm(*o) for k, o in ops.items()}))
    for g, y in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y[k], want[k]) for _, y in graphs for k in want)
    for o in ops.values():                           # new scales under the same addresses
        o[1].mul_(2.0)
    for g, y in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y[k], want[k] * 2) for _, y in graphs for k in want)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for k, o in ops.items():
        for st in streams:
            with torch.cuda.stream(st):
                got.append((k, vitq.int8_gemm(*o)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k] * 2) for k, y in got) and vitq.device_error() == 0


@gpu
@pytest.mark.parametrize("N", [3, 8])
def test_most_rows(N):
    """2^24 rows, the entry point's limit; every row is one of 1000."""
    M, (qa, sa, qw, sw) = 1 << 24, _operands(1000, N, 16)
    want = vitq.int8_gemm(qa, sa, qw, sw)
    times = -(-M // 1000)
    y = vitq.int8_gemm(qa.repeat(times, 1)[:M], sa.repeat(times)[:M], qw, sw)
    for a in range(0, M, 1000 << 10):
        n = min(M - a, 1000 << 10)
        assert torch.equal(y[a:a + n], want.repeat(1024, 1)[:n]), a
    assert vitq.device_error() == 0
