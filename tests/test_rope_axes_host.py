"""vit_rope_axes refuses outputs that are another tensor of the call: q and k turned in place as one tensor would
be turned twice, in no order.  On CPU: the refusals come before any device query."""
import ctypes

import pytest
import torch

from quantized_vit_encoder_b200 import vitq

A, B, D, E = (ctypes.c_void_p(4096 * i) for i in (1, 2, 3, 4))


@pytest.fixture(scope="module")
def lib():
    from quantized_vit_encoder_b200 import build
    build.build(verbose=False)
    return vitq.load()


def _call(lib, q, q_out, k, k_out, heads_q=4, heads_k=4, n=5):
    p = vitq.RopeAxes(0, 1, (ctypes.c_int32 * 4)(8, 0, 0, 0), heads_q, heads_k, 16, 0, 10000.0,
                      64, 16, 64, 16, 64, 16, 64, 16, 1, 1)
    return lib.vit_rope_axes(ctypes.byref(p), q, q_out, k, k_out, ctypes.c_void_p(4096 * 9), n, None)


@pytest.mark.parametrize("q,q_out,k,k_out", [(A, A, A, A), (A, D, B, D), (A, B, B, D), (A, D, B, A), (A, A, A, D), (A, D, A, A)])
def test_shared_outputs_are_refused(lib, q, q_out, k, k_out):
    assert _call(lib, q, q_out, k, k_out) == vitq.ERR_INVALID_ARG


def test_pointers_that_are_not_used_may_be_anything(lib):
    assert _call(lib, A, A, A, A, n=0) != vitq.ERR_INVALID_ARG       # (launches nothing)


@pytest.mark.gpu
def test_one_tensor_as_both_inputs():
    x = torch.randn((33, 4, 72), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    pos = torch.arange(33, device="cuda", dtype=torch.int32)[:, None].expand(33, 3)
    want = vitq.rope_axes(x, None, pos, (12, 12, 12))[0]
    q, k = vitq.rope_axes(x, x, pos, (12, 12, 12))
    assert torch.equal(q, want) and torch.equal(k, want)
    with pytest.raises(vitq.VitqError, match="invalid argument"):
        vitq.rope_axes_(x, x, pos, (12, 12, 12))
    vitq.rope_axes_(x, None, pos, (12, 12, 12))
    assert torch.equal(x, want)
