"""Argument checks of the INT8 entry points and of vit_rope_axes, on CPU: the C ABI's
refusals (found before any device query), the struct's layout, and the binding's checks
and marshalling against a stub of the library."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, SHAPE, ALIGN = vitq.ERR_INVALID_ARG, vitq.ERR_SHAPE, vitq.ERR_ALIGN
V = ctypes.c_void_p
P = V(4096)                       # aligned, never read: each call below is refused first


@pytest.fixture(scope="module")
def lib():
    from quantized_vit_encoder_b200 import build
    build.build(verbose=False)
    return vitq.load()


# ------------------------------------------------------------------ C ABI
def _quant(lib, x=P, dtype=0, M=4, K=32, ldx=32, q=P, ldq=32, s=P):
    return lib.vit_quant_int8(x, dtype, M, K, ldx, q, ldq, s, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(ldx=31), INVALID),
    (dict(ldq=31), INVALID), (dict(ldq=40), SHAPE), (dict(M=(1 << 24) + 1), SHAPE),
    (dict(K=(1 << 16) + 1, ldx=1 << 17, ldq=1 << 17), SHAPE), (dict(x=V(4097)), ALIGN), (dict(q=V(4104)), ALIGN),
    (dict(s=V(4098)), ALIGN), (dict(x=V(4098), dtype=2), ALIGN)])
def test_quant_int8_refusals(lib, bad, code):
    assert _quant(lib, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INVALID), (dict(g=None), INVALID), (dict(b=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(K=0), INVALID), (dict(ldq=24), INVALID), (dict(g=V(4097)), ALIGN),
    (dict(M=(1 << 24) + 1), SHAPE)])
def test_ln_quant_int8_refusals(lib, bad, code):
    a = dict(x=P, M=4, K=32, ldx=32, g=P, b=P, eps=1e-6, q=P, ldq=32, s=P) | bad
    assert lib.vit_ln_quant_int8(a["x"], a["M"], a["K"], a["ldx"], a["g"], a["b"], ctypes.c_float(a["eps"]), a["q"],
                                 a["ldq"], a["s"], None) == code


@pytest.mark.parametrize("bad,code", [(dict(f=None), INVALID), (dict(K=-3), INVALID), (dict(ldf=8), INVALID),
                                      (dict(ldq=33), SHAPE), (dict(f=V(4097)), ALIGN)])
def test_gelu_quant_int8_refusals(lib, bad, code):
    a = dict(f=P, M=4, K=32, ldf=32, q=P, ldq=32, s=P) | bad
    assert lib.vit_gelu_quant_int8(a["f"], a["M"], a["K"], a["ldf"], a["q"], a["ldq"], a["s"], None) == code


GEMM = dict(A=P, lda=64, sA=P, W=P, ldw=64, sW=P, bias=None, res=None, ldr=0, C=P, ldc=40, dtype=0, M=8, N=40, K=64)


@pytest.mark.parametrize("bad,code", [
    (dict(A=None), INVALID), (dict(W=None), INVALID), (dict(sA=None), INVALID), (dict(sW=None), INVALID),
    (dict(C=None), INVALID), (dict(dtype=7), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(lda=48), INVALID), (dict(ldw=48), INVALID), (dict(ldc=39), INVALID), (dict(res=P, ldr=39), INVALID),
    (dict(lda=72), SHAPE), (dict(ldw=72), SHAPE), (dict(M=(1 << 24) + 1), SHAPE), (dict(M=(1 << 31) - 1), SHAPE),
    (dict(N=(1 << 16) + 8, ldc=1 << 17), SHAPE), (dict(K=(1 << 16) + 16, lda=1 << 17, ldw=1 << 17), SHAPE),
    (dict(A=V(4104)), ALIGN), (dict(W=V(4104)), ALIGN), (dict(C=V(4097)), ALIGN), (dict(C=V(4098), dtype=2), ALIGN),
    (dict(bias=V(4097)), ALIGN), (dict(res=V(4097), ldr=40), ALIGN), (dict(sA=V(4098)), ALIGN),
    (dict(res=P, ldr=48), INVALID)])                # the residual in place, but with another row stride than C's
def test_int8_gemm_refusals(lib, bad, code):
    a = GEMM | bad
    assert lib.int8_gemm(*[a[k] for k in GEMM], None) == code


def _rope(**kw):
    a = dict(dtype=0, n_axes=3, sections=(12, 12, 12), heads_q=4, heads_k=2, head_dim=72, flags=0, theta=10000.0,
             q=(288, 72), q_out=(288, 72), k=(144, 72), k_out=(144, 72), pos=(3, 1)) | kw
    sec = (ctypes.c_int32 * 4)(*(list(a["sections"]) + [0] * 4)[:4])
    return vitq.RopeAxes(a["dtype"], a["n_axes"], sec, a["heads_q"], a["heads_k"], a["head_dim"], a["flags"], a["theta"],
                         *a["q"], *a["q_out"], *a["k"], *a["k_out"], *a["pos"])


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=5), INVALID), (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE), (dict(sections=(-1, 12, 12)), SHAPE),
    (dict(sections=(0, 0, 0)), SHAPE), (dict(sections=(13, 12, 12)), SHAPE), (dict(head_dim=0), INVALID),
    (dict(head_dim=514), SHAPE), (dict(heads_q=-1), INVALID), (dict(heads_k=1025), SHAPE), (dict(flags=16), INVALID),
    (dict(theta=0.0), INVALID), (dict(theta=float("inf")), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(q=(-1, 72)), SHAPE), (dict(pos=(3, -1)), SHAPE), (dict(q=(1 << 31, 72)), SHAPE),
    (dict(q_out=(72, 71)), SHAPE), (dict(q_out=(200, 72)), SHAPE), (dict(k_out=(0, 72)), SHAPE),
    # interleaved: axis 2 has no pair 2 + 3 * 12 in 36
    (dict(sections=(10, 13, 13), flags=vitq.ROPE_INTERLEAVED), SHAPE)])
def test_rope_axes_refusals(lib, bad, code):
    p = _rope(**bad)
    assert lib.vit_rope_axes(ctypes.byref(p), P, V(8192), P, V(8192), P, 5, None) == code


def test_rope_axes_pointer_refusals(lib):
    ref, f = ctypes.byref, lib.vit_rope_axes
    p = _rope()
    assert f(None, P, P, P, P, P, 5, None) == INVALID
    assert f(ref(p), None, P, P, P, P, 5, None) == INVALID
    assert f(ref(p), P, P, P, None, P, 5, None) == INVALID
    assert f(ref(p), P, P, P, P, None, 5, None) == INVALID
    assert f(ref(p), P, P, P, P, P, -1, None) == INVALID
    assert f(ref(p), P, P, P, P, P, (1 << 24) + 1, None) == SHAPE
    assert f(ref(p), V(4097), P, P, P, P, 5, None) == ALIGN
    assert f(ref(p), P, P, P, P, V(4098), 5, None) == ALIGN
    moved = _rope(q=(1000, 72))                     # in place, but with other strides than the input's
    assert f(ref(moved), P, P, P, P, P, 5, None) == INVALID


def test_rope_axes_struct_layout(lib, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    fields = [n for n, _ in vitq.RopeAxes._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "vitq.h"\nint main(void) {\n' + \
        ''.join(f'printf("%zu\\n", offsetof(vitq_rope_axes, {n}));\n' for n in fields) + \
        'printf("%zu\\n", sizeof(vitq_rope_axes)); return 0; }\n'
    (tmp_path / "l.c").write_text(src)
    exe = str(tmp_path / "l")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"),
                    "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(vitq.RopeAxes, n).offset for n in fields] + [ctypes.sizeof(vitq.RopeAxes)]


def test_header_constants_match_the_binding():
    src = open(os.path.join(ROOT, "include", "vitq.h")).read()
    for name, value in (("VITQ_BF16", 0), ("VITQ_FP16", 1), ("VITQ_FP32", 2), ("VITQ_ROPE_MAX_AXES", 4),
                        ("VITQ_ROPE_INTERLEAVED", vitq.ROPE_INTERLEAVED), ("VITQ_ROPE_AXIS_FREQ", vitq.ROPE_AXIS_FREQ),
                        ("VITQ_ROPE_ADJACENT", vitq.ROPE_ADJACENT), ("VITQ_ROPE_INVERSE", vitq.ROPE_INVERSE)):
        assert re.search(rf"#define {name} {value}\b", src), name


# ------------------------------------------------------------------ binding
class _Stub:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, [getattr(a, "value", a) for a in args]))
            return 0
        return fn


@pytest.fixture
def on_cpu(monkeypatch):
    s = _Stub()
    monkeypatch.setattr(vitq, "_lib", s)
    monkeypatch.setattr(vitq, "_stream", lambda stream=None: None)
    monkeypatch.setattr(vitq, "_DEVICE_TYPE", "cpu")
    return s


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i8(m, k):
    return torch.zeros((m, (k + 15) // 16 * 16), dtype=torch.int8)[:, :k]


def test_binding_marshals_rows(on_cpu):
    q, s = vitq.quant_int8(torch.zeros((7, 100)))
    name, a = on_cpu.calls[-1]
    assert name == "vit_quant_int8" and a[1:5] == [2, 7, 100, 100] and a[6] == 112
    assert q.shape == (7, 100) and q.stride() == (112, 1) and q.dtype == torch.int8 and s.shape == (7,)
    vitq.quant_int8(_bf(9, 64)[:, 3:35])
    assert on_cpu.calls[-1][1][1:5] == [0, 9, 32, 64]
    vitq.ln_quant_int8(_bf(5, 48), _bf(48), _bf(48), eps=1e-5)
    a = on_cpu.calls[-1][1]
    assert a[1:4] == [5, 48, 48] and a[6] == 1e-5 and a[8] == 48
    out = (torch.zeros((5, 64), dtype=torch.int8)[:, :48], torch.zeros(5))
    assert vitq.gelu_quant_int8(_bf(5, 48), out=out)[0] is out[0]
    assert on_cpu.calls[-1][1][1:4] == [5, 48, 48] and on_cpu.calls[-1][1][5] == 64


def test_binding_marshals_gemm(on_cpu):
    y = vitq.int8_gemm(_i8(6, 50), torch.zeros(6), _i8(11, 50), torch.zeros(11), bias=_bf(11))
    a = on_cpu.calls[-1][1]
    assert y.shape == (6, 11) and y.dtype == torch.bfloat16 and a[1] == 64 and a[4] == 64 and a[7] is None
    assert a[10:15] == [11, 0, 6, 11, 50]
    wide = torch.zeros((6, 32), dtype=torch.float16)
    vitq.int8_gemm(_i8(6, 50), torch.zeros(6), _i8(11, 50), torch.zeros(11), residual=wide[:, :11], out=wide[:, 16:27])
    a = on_cpu.calls[-1][1]
    assert a[8] == 32 and a[10:15] == [32, 1, 6, 11, 50]


def test_binding_marshals_rope(on_cpu):
    qkv = _bf(10, 3456)
    q, k = qkv[:, :1152].view(10, 16, 72), qkv[:, 1152:2304].view(10, 16, 72)
    pos = torch.zeros((3, 10), dtype=torch.int32).t()
    yq, yk = vitq.rope_axes(q, k, pos, (12, 12, 12), axis_freq=True, inverse=True)
    name, a = on_cpu.calls[-1]
    p = vitq.RopeAxes.from_buffer_copy(a[0])
    assert name == "vit_rope_axes" and a[6] == 10 and yq.is_contiguous() and yk.shape == (10, 16, 72)
    assert (p.q_token, p.q_head, p.q_out_token, p.q_out_head) == (3456, 72, 1152, 72)
    assert (p.pos_token, p.pos_axis, p.flags, p.head_dim) == (1, 10, 2 | 8, 72)
    assert vitq.rope_axes_(q, None, pos, (36, 0, 0))[0] is q
    p = vitq.RopeAxes.from_buffer_copy(on_cpu.calls[-1][1][0])
    assert p.heads_k == 0 and p.q_out_token == 3456 and list(p.sections) == [36, 0, 0, 0]


@pytest.mark.parametrize("call", [
    lambda: vitq.quant_int8(torch.zeros((4, 8), dtype=torch.float64)),
    lambda: vitq.quant_int8(torch.zeros(8)),
    lambda: vitq.quant_int8(torch.zeros((8, 4)).t()),
    lambda: vitq.quant_int8(torch.zeros((1, 8)).expand(4, 8)),
    lambda: vitq.quant_int8(_bf(4, 32), out=(torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4))),
    lambda: vitq.ln_quant_int8(torch.zeros((4, 8)), _bf(8), _bf(8)),
    lambda: vitq.ln_quant_int8(_bf(4, 8), _bf(7), _bf(8)),
    lambda: vitq.gelu_quant_int8(torch.zeros((4, 8), dtype=torch.float16)),
    lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(4), _i8(8, 48), torch.zeros(8)),
    lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(5), _i8(8, 32), torch.zeros(8)),
    lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(4), _i8(8, 32), torch.zeros(8), bias=torch.zeros(8)),
    lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(4), _i8(8, 32), torch.zeros(8), out=torch.zeros((4, 8), dtype=torch.int8)),
    lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(4), _i8(8, 32), torch.zeros(8), out_dtype=torch.int32),
    lambda: vitq.int8_gemm(_i8(4, 32).to(torch.uint8), torch.zeros(4), _i8(8, 32), torch.zeros(8)),
    lambda: vitq.rope_axes(_bf(4, 2, 8), _bf(5, 2, 8), torch.zeros((4, 1), dtype=torch.int32), (4,)),
    lambda: vitq.rope_axes(_bf(4, 2, 8), _bf(4, 2, 8), torch.zeros((4, 2), dtype=torch.int32), (4,)),
    lambda: vitq.rope_axes(_bf(4, 2, 8), _bf(4, 2, 8), torch.zeros((4, 1), dtype=torch.int64), (4,)),
    lambda: vitq.rope_axes(_bf(4, 8, 2).transpose(1, 2), None, torch.zeros((4, 1), dtype=torch.int32), (4,)),
    lambda: vitq.rope_axes(_bf(4, 2, 8), None, torch.zeros((4, 5), dtype=torch.int32), (1, 1, 1, 1, 0)),
])
def test_binding_refusals(on_cpu, call):
    with pytest.raises(vitq.VitqError):
        call()
    assert not on_cpu.calls


def test_binding_refuses_sizes_past_int32(on_cpu, monkeypatch):
    """Sizes and strides that would wrap around in a C int (meta tensors: no memory behind them)."""
    monkeypatch.setattr(vitq, "_DEVICE_TYPE", "meta")
    big = 1 << 31

    def meta(shape, strides, t=torch.bfloat16):
        return torch.empty_strided(shape, strides, dtype=t, device="meta")
    for call in (lambda: vitq.quant_int8(meta((2, 32), (big + 32, 1))),
                 lambda: vitq.quant_int8(meta((2 * big + 4, 32), (32, 1))),
                 lambda: vitq.gelu_quant_int8(meta((2, 32), (2 * big + 32, 1))),
                 lambda: vitq.int8_gemm(meta((4, 32), (big + 32, 1), torch.int8), torch.zeros(4), _i8(8, 32), torch.zeros(8)),
                 lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(4), _i8(8, 32), torch.zeros(8),
                                        out=meta((4, 8), (2 * big + 8, 1))),
                 lambda: vitq.rope_axes(meta((2 * big + 4, 2, 8), (16, 8, 1)), None,
                                        meta((2 * big + 4, 1), (1, 1), torch.int32), (4,))):
        with pytest.raises(vitq.VitqError, match="2\\^31"):
            call()
    assert not on_cpu.calls


def test_host_tensors_never_reach_the_library(monkeypatch):
    s = _Stub()
    monkeypatch.setattr(vitq, "_lib", s)
    for call in (lambda: vitq.quant_int8(_bf(4, 32)), lambda: vitq.gelu_quant_int8(_bf(4, 32)),
                 lambda: vitq.int8_gemm(_i8(4, 32), torch.zeros(4), _i8(8, 32), torch.zeros(8)),
                 lambda: vitq.rope_axes(_bf(4, 2, 8), None, torch.zeros((4, 1), dtype=torch.int32), (4,))):
        with pytest.raises(vitq.VitqError):
            call()
    assert not s.calls
