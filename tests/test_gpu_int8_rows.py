"""The INT8 row kernels where a call is hard on them: calls from two host threads, LayerNorm rows without
spread, statistics and results at the ends of the number range.

Codes and scales are compared bit for bit with the definition in 64 bits, stated directly where the
definition is plain (a constant row's LayerNorm is beta).
"""
import ctypes as C
import math
import os
import shutil
import subprocess

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _codes_ref(y):
    """(codes, scales) of rows of y, from the definition."""
    amax = y.abs().amax(1).float()
    s = torch.where(torch.isfinite(amax), amax / torch.full_like(amax, 127), math.nan)   # a division, not a product
    q = torch.round(y.double() / s.double()[:, None])
    return torch.where((s > 0)[:, None], q, 0.0).clamp(-127, 127).to(torch.int8), s


def _same(got, want, what=""):
    q, s = got
    torch.cuda.synchronize()
    wq, ws = want
    assert torch.equal(s.nan_to_num(-1.0), ws.nan_to_num(-1.0)), f"{what}: scales differ"
    bad = (q != wq).nonzero()
    assert not len(bad), f"{what}: {len(bad)} codes differ, first at {bad[:3].tolist()}"
    assert vitq.device_error() == 0


# ------------------------------------------------------------------ calls from two host threads
HAMMER = r"""
#include <pthread.h>
#include "vitq.h"
typedef struct {
  int kind, dtype, M, K, ldx, ldq, n, failed, status;
  const void *x, *gamma, *beta;   /* of a product: A, W and sA */
  int8_t* q;
  float* s;
  void* stream;
  int N, ldw;
  const float* sW;
  const vitq_rope_axes* rope;
  pthread_barrier_t* start;
} job;
static void* work(void* p) {
  job* j = (job*)p;
  pthread_barrier_wait(j->start);
  for (int i = 0; i < j->n; ++i) {
    int r = j->kind == 0   ? vit_quant_int8(j->x, j->dtype, j->M, j->K, j->ldx, j->q, j->ldq, j->s, j->stream)
            : j->kind == 1 ? vit_ln_quant_int8(j->x, j->M, j->K, j->ldx, j->gamma, j->beta, 1e-6f, j->q, j->ldq, j->s, j->stream)
            : j->kind == 2 ? vit_gelu_quant_int8(j->x, j->M, j->K, j->ldx, j->q, j->ldq, j->s, j->stream)
            : j->kind == 4 ? int8_gemm(j->x, j->ldx, j->beta, j->gamma, j->ldw, j->sW, 0, 0, 0, j->q, j->ldq, j->dtype, j->M, j->N,
                                       j->K, j->stream)
            : j->kind == 5 ? vit_rope_axes(j->rope, j->x, j->q, 0, 0, (const int32_t*)j->beta, j->M, j->stream)
                           : vit_ln_quant(j->x, j->M, j->K, j->ldx, j->gamma, j->beta, 1e-6f, (uint8_t*)j->q, j->s, j->ldq, j->stream);
    if (r) j->failed++, j->status = r;
  }
  return 0;
}
int hammer(job* jobs, int threads) {
  pthread_barrier_t start;
  pthread_t t[8];
  int failed = 0;
  pthread_barrier_init(&start, 0, (unsigned)threads);
  for (int i = 0; i < threads; ++i) jobs[i].start = &start;
  for (int i = 0; i < threads; ++i) pthread_create(&t[i], 0, work, &jobs[i]);
  for (int i = 0; i < threads; ++i) {
    pthread_join(t[i], 0);
    failed += jobs[i].failed;
  }
  pthread_barrier_destroy(&start);
  return failed;
}
"""


class Job(C.Structure):
    _fields_ = ([(n, C.c_int) for n in ("kind", "dtype", "M", "K", "ldx", "ldq", "n", "failed", "status")] +
                [(n, C.c_void_p) for n in ("x", "gamma", "beta", "q", "s", "stream")] + [("N", C.c_int), ("ldw", C.c_int)] +
                [(n, C.c_void_p) for n in ("sW", "rope", "start")])


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    """A C function that makes calls from host threads at once (Python's lock would keep them apart)."""
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    vitq.load()
    d = tmp_path_factory.mktemp("hammer")
    (d / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-pthread", "-I", os.path.join(ROOT, "include"), str(d / "hammer.c"),
                    "-o", str(d / "hammer.so"), vitq.LIB_PATH, "-Wl,-rpath," + os.path.dirname(vitq.LIB_PATH)], check=True)
    return C.CDLL(str(d / "hammer.so")).hammer


QUANT, LN, GELU, LN_FP8, GEMM, ROPE = range(6)
# pairs of calls that run one kernel with different amounts of shared memory
TOGETHER = {
    "ln_1152_by_rows": [(LN, BF, 256, 1152), (LN, BF, 6256, 1152)],
    "ln_by_width": [(LN, BF, 300, 4608), (LN, BF, 300, 16000)],
    "ln_any_alignment": [(LN, BF, 300, 1145), (LN, BF, 3000, 1151)],
    "quant_any_alignment": [(QUANT, BF, 40, 2101), (QUANT, BF, 40, 2303)],
    "quant_fp32_wide": [(QUANT, F32, 20, 9301), (QUANT, F32, 20, 32767)],
    "gelu_any_alignment": [(GELU, BF, 40, 2101), (GELU, BF, 40, 2303)],
    "ln_fp8_by_width": [(LN_FP8, BF, 300, 4224), (LN_FP8, BF, 300, 4608)],
}


@pytest.mark.parametrize("name", TOGETHER)
def test_two_host_threads(name, hammer):
    """Two threads call the same operator at different sizes, each on its own stream: no call fails, and
    every result is the one of a call alone."""
    jobs, keep = (Job * 2)(), []
    for i, (kind, t, M, K) in enumerate(TOGETHER[name]):
        x, g, b = _randn(i, M, K).to(t), (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
        call = {QUANT: lambda: vitq.quant_int8(x), LN: lambda: vitq.ln_quant_int8(x, g, b), GELU: lambda: vitq.gelu_quant_int8(x),
                LN_FP8: lambda: vitq.ln_quant(x, g, b)}[kind]
        want, got, st = call(), [w.zero_() for w in call()], torch.cuda.Stream()
        keep.append((x, g, b, want, got, st))
        jobs[i] = Job(kind, vitq._DTYPES[t], M, K, K, got[1].stride(0) if kind == LN_FP8 else got[0].stride(0), 5000, 0, 0,
                      x.data_ptr(), g.data_ptr(), b.data_ptr(), got[0].data_ptr(), got[1].data_ptr(), st.cuda_stream)
    _hammer(hammer, jobs, keep)


def _hammer(hammer, jobs, keep):
    torch.cuda.synchronize()
    failed = hammer(jobs, 2)
    torch.cuda.synchronize()
    assert failed == 0, f"{failed} of {sum(j.n for j in jobs)} calls failed, status {[j.status for j in jobs]}"
    for *_, want, got, _ in keep:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert vitq.device_error() == 0


# products that share a kernel (split K by 4 and 8, single tiles, pairs), or a code path
@pytest.mark.parametrize("shapes", [((243, 2048, 4600), (121, 1104, 5001)), ((301, 4304, 1151), (972, 1152, 1152)),
                                    ((2100, 1160, 1100), (5001, 2688, 203)), ((7, 200, 303), (30, 1160, 1000))])
def test_two_host_threads_of_products(shapes, hammer):
    jobs, keep = (Job * 2)(), []
    for i, (M, N, K) in enumerate(shapes):
        qa, sa = vitq.quant_int8(_randn(i, M, K))
        qw, sw = vitq.quant_int8(_randn(i + 2, N, K))
        want, st = vitq.int8_gemm(qa, sa, qw, sw), torch.cuda.Stream()
        got = torch.zeros_like(want)
        keep.append((qa, sa, qw, sw, (want,), (got,), st))
        jobs[i] = Job(GEMM, vitq._DTYPES[BF], M, K, qa.stride(0), N, 3000, 0, 0, qa.data_ptr(), qw.data_ptr(), sa.data_ptr(),
                      got.data_ptr(), None, st.cuda_stream, N, qw.stride(0), sw.data_ptr())
    _hammer(hammer, jobs, keep)


def test_two_host_threads_of_the_rotary(hammer):
    jobs, keep = (Job * 2)(), []
    for i, (n, h, sections) in enumerate(((16, 8, (12, 12, 12)), (4096, 16, (24, 20, 20)))):
        d = 2 * sum(sections)
        x = _randn(i, n, h, d).to(BF)
        pos = torch.arange(3 * n, device="cuda", dtype=torch.int32).view(n, 3)
        p = vitq.RopeAxes(vitq._DTYPES[BF], 3, (C.c_int32 * 4)(*sections, 0), h, 0, d, 0, 10000.0, h * d, d, h * d, d,
                          0, 0, 0, 0, 3, 1)
        want, st = vitq.rope_axes(x, None, pos, sections)[0], torch.cuda.Stream()
        got = torch.zeros_like(want)
        keep.append((x, pos, p, (want,), (got,), st))
        jobs[i] = Job(ROPE, 0, n, 0, 0, 0, 3000, 0, 0, x.data_ptr(), None, pos.data_ptr(), got.data_ptr(), None, st.cuda_stream,
                      0, 0, None, C.addressof(p))
    _hammer(hammer, jobs, keep)


# ------------------------------------------------------------------ LayerNorm
# widths whose reciprocal in 64 bits times a constant row's sum is not that constant, and plain ones
@pytest.mark.parametrize("K", [49, 103, 300, 1000, 1001, 1152, 1960, 2056, 3000, 4608, 15987, 16400])
def test_ln_quant_constant_rows_come_out_as_beta(K):
    values = [0.0, 1.0, 1.9921875, -1.9921875, 1.0078125, 3.140625, 1.9921875 * 2.0 ** 50, -1.9921875 * 2.0 ** 100,
              1.9921875 * 2.0 ** 120, 1.9921875 * 2.0 ** -100]
    x = torch.tensor(values, device="cuda").to(BF)[:, None].expand(-1, K).contiguous()
    gamma, beta = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    for b in (beta, torch.zeros_like(beta)):
        for eps in (1e-6, 1.0, 1e-12):
            _same(vitq.ln_quant_int8(x, gamma, b, eps=eps), _codes_ref(b[None].expand(len(values), K)), (K, eps))
    q, s = vitq.ln_quant_int8(x, gamma, beta, eps=0.0)          # 0 / 0
    assert torch.isnan(s).all() and not q.any()


@pytest.mark.parametrize("K", [50, 98, 206, 1152, 1960, 4606, 16400])
def test_ln_quant_results_that_are_exact_ties(K):
    """Rows of +c and -c in turn: the mean is 0, (x - mean) rstd is +-1 exactly with eps = 0, and with
    gamma = 1 and beta half a step of bf16 every positive result is an exact tie, which goes to even."""
    sign = torch.ones(K, device="cuda")
    sign[1::2] = -1
    x = torch.stack([sign, sign * 0.5, -sign * 4096, sign * 2.0 ** -60]).to(BF)
    gamma = torch.ones(K, dtype=BF, device="cuda")
    for beta, up, down in ((2.0 ** -8, 1.0, -1 + 2.0 ** -8), (3 * 2.0 ** -8, 1 + 2.0 ** -6, -1 + 3 * 2.0 ** -8)):
        y = torch.where(x.float() > 0, up, down)
        b = torch.full((K,), beta, device="cuda").to(BF)
        _same(vitq.ln_quant_int8(x, gamma, b, eps=0.0), _codes_ref(y), (K, beta))


@pytest.mark.parametrize("K", [40, 100, 1100, 1153, 2001, 4700])
def test_ln_quant_constant_rows_with_a_tiny_eps(K):
    """mean times rstd is past fp32's range, also in the columns that a thread has behind the last one."""
    x = torch.tensor([2.0 ** 99, -2.0 ** 90, 1.0], device="cuda").to(BF)[:, None].expand(-1, K).contiguous()
    gamma, beta = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    for eps in (1e-20, 1e-38):
        _same(vitq.ln_quant_int8(x, gamma, beta, eps=eps), _codes_ref(beta[None].expand(3, K)), (K, eps))


def _bf16_any(y):
    """fp64 -> bf16 with one rounding, subnormal results included."""
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp_min(-125) - 8)
    return (torch.round(y / step) * step).to(F32).to(BF)


@pytest.mark.parametrize("K", [1152, 1153, 2048, 4608])
def test_ln_quant_results_below_the_normal_range(K):
    """gamma so small that results are subnormal: the error of fp32 arithmetic is then absolute, not relative."""
    M = 3000 if K < 4000 else 1000
    x = _randn(K, M, K).to(BF)
    for scale in (2.0 ** -130, 2.0 ** -127, 2.0 ** -120):
        gamma = ((1 + 0.1 * _randn(1, K)).double() * scale).to(F32).to(BF)
        c = x.double() - x.double().mean(1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6) * gamma.double()
        _same(vitq.ln_quant_int8(x, gamma, torch.zeros_like(gamma)), _codes_ref(_bf16_any(y)), (K, scale))


@pytest.mark.parametrize("K", [1152, 4608])
def test_ln_quant_results_of_inputs_below_the_normal_range(K):
    """Rows of subnormal inputs under a large eps: (x - mean) rstd is subnormal, and a large gamma brings
    the result back to the middle of the range."""
    x = (_randn(K, 2000, K).double() * 2.0 ** -128).to(F32).to(BF)
    for scale in (2.0 ** -4, 1.0, 2.0 ** 40, 2.0 ** 100):
        gamma = ((1 + 0.1 * _randn(1, K)).double() * scale).to(F32).to(BF)
        c = x.double() - x.double().mean(1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 4.0) * gamma.double()
        _same(vitq.ln_quant_int8(x, gamma, torch.zeros_like(gamma), eps=4.0), _codes_ref(_bf16_any(y)), (K, scale))


# ------------------------------------------------------------------ widths at the limits of the kernels
# chunks (16 bytes) of a row up to which each number of threads a row is used: the widths just below, at and
# above, where a row fills its threads' chunks (and its shared memory, where rows start anywhere) or spills
# over into the next kernel
ROW_LIMITS, LN_LIMITS = (160, 288, 576, 1152, 2304, 8192), (144, 256, 2048)


def _limit_widths(limits, per, most=65536):
    return sorted({k for c in limits for k in (c * per - 1, c * per, c * per + 1, (c + 1) * per) if k <= most})


def _ln_ref(x, gamma, beta):
    c = x.double() - x.double().mean(1, keepdim=True)
    return _bf16_any(c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6) * gamma.double() + beta.double())


def _gelu_ref(f):
    x = f.double()
    return _bf16_any(x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("op,t,K", [("quant", t, k) for t in (BF, HF, F32) for k in _limit_widths(ROW_LIMITS, 4 if t == F32 else 8)] +
                         [("gelu", BF, k) for k in _limit_widths(ROW_LIMITS, 8)] +
                         [("ln", BF, k) for k in _limit_widths(LN_LIMITS, 8)])
def test_widths_at_the_limits(op, t, K, shift):
    """Rows of x from their storage's first element on (shift 1: one element in, so that rows start anywhere)
    to its last; sentinels around the codes and scales."""
    M, ldq = 9, (K + 15) // 16 * 16 + 16
    x = torch.empty(shift + M * K, dtype=t, device="cuda")[shift:].view(M, K)
    x.copy_(_randn(K, M, K) * torch.exp(_randn(K + 1, M, 1)))
    codes, scales = torch.full((M + 2, ldq), 99, dtype=torch.int8, device="cuda"), torch.full((M + 2,), -1.0, device="cuda")
    out = codes[1:M + 1, :K], scales[1:M + 1]
    if op == "quant":
        got, y = vitq.quant_int8(x, out=out), x
    elif op == "gelu":
        got, y = vitq.gelu_quant_int8(x, out=out), _gelu_ref(x)
    else:
        g, b = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
        got, y = vitq.ln_quant_int8(x, g, b, out=out), _ln_ref(x, g, b)
    _same(got, _codes_ref(y), (op, t, K))
    assert (codes[0] == 99).all() and (codes[-1] == 99).all() and (codes[:, K:] == 99).all()
    assert scales[0] == scales[-1] == -1


@pytest.mark.parametrize("op", ["quant", "ln", "gelu"])
@pytest.mark.parametrize("K", [8, 3])
def test_most_rows(op, K):
    """2^24 rows, the entry points' limit; every row is one of 1000."""
    M, few = 1 << 24, _randn(K, 1000, K).to(BF)
    x = few.repeat(-(-M // 1000), 1)[:M]
    g, b = (1 + 0.1 * _randn(1, K)).to(BF), (0.1 * _randn(2, K)).to(BF)
    call = {"quant": vitq.quant_int8, "gelu": vitq.gelu_quant_int8, "ln": lambda a: vitq.ln_quant_int8(a, g, b)}[op]
    (q, s), (wq, ws) = call(x), call(few)
    for a in range(0, M, 1000 << 10):
        n = min(M - a, 1000 << 10)
        assert torch.equal(q[a:a + n], wq.repeat(1024, 1)[:n]) and torch.equal(s[a:a + n], ws.repeat(1024)[:n]), a
    with pytest.raises(vitq.VitqError, match="unsupported shape"):
        call(x.new_zeros((M + 1, K)))
