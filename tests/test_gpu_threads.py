"""Calls from host threads that have made no CUDA call before: such a thread has no context current, which the
encoding of a tensor map needs."""
import threading

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _int8(M, N, K):
    qa, qw = vitq.quant_int8(_randn(1, M, K)), vitq.quant_int8(_randn(2, N, K))
    out = torch.zeros((M, N), dtype=BF, device="cuda")
    return out, lambda: vitq.load().int8_gemm(qa[0].data_ptr(), qa[0].stride(0), qa[1].data_ptr(), qw[0].data_ptr(),
                                              qw[0].stride(0), qw[1].data_ptr(), None, None, 0, out.data_ptr(), N, 0, M, N, K, None)


def _fp8(M, N, K):
    qa, qw = vitq.quant_act(_randn(1, M, K).to(BF)), vitq.quant_weight(_randn(2, N, K).to(BF))
    out = torch.zeros((M, N), dtype=BF, device="cuda")
    return out, lambda: vitq.load().fp8_block_gemm(qa[0].data_ptr(), qa[1].data_ptr(), qa[1].stride(0), qw[0].data_ptr(),
                                                   qw[1].data_ptr(), None, None, out.data_ptr(), M, N, K, None)


def _bf16(M, N, K):
    a, w = _randn(1, M, K).to(BF), _randn(2, N, K).to(BF)
    out = torch.zeros((M, N), dtype=BF, device="cuda")
    return out, lambda: vitq.load().bf16_gemm(a.data_ptr(), w.data_ptr(), None, None, out.data_ptr(), M, N, K, None)


def _attention(n):
    qkv, cu = _randn(1, n, 3456).to(BF), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = torch.zeros((n, 1152), dtype=BF, device="cuda")
    return out, lambda: vitq.load().vit_attention_varlen(qkv.data_ptr(), n, cu.data_ptr(), 1, n, 72 ** -0.5, 0, out.data_ptr(), None)


CALLS = {"int8_gemm tiles": lambda: _int8(301, 4304, 1152), "int8_gemm pairs": lambda: _int8(2100, 1160, 1104),
         "int8_gemm split K": lambda: _int8(243, 2048, 4608), "fp8_block_gemm": lambda: _fp8(256, 1152, 1152),
         "bf16_gemm": lambda: _bf16(256, 1152, 1152), "attention": lambda: _attention(256)}


@pytest.mark.parametrize("name", CALLS)
def test_first_call_of_a_host_thread(name):
    out, call = CALLS[name]()
    assert call() == vitq.OK
    torch.cuda.synchronize()
    want, got = out.clone(), []
    out.zero_()
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got == [vitq.OK] and torch.equal(out, want) and vitq.device_error() == 0
