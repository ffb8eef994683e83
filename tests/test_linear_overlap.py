"""Results of the dense quantised products that would overwrite their own operands are
refused; column slices of one buffer are not."""
import ctypes

import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe

A = 0x10000000
W = moe.QMatrixC(A, A, A, 256, 256, 128, 4)


def _linear(x, y, T=4, ldx=256, ldy=256, t=moe.BF16, rb=None, res=None, ldr=256):
    return moe.lib().moe_linear(ctypes.byref(W), T, x, ldx, rb, res, ldr, y, ldy, t, A, 1 << 40, None)


def _grad(dy, dx, T=4, lddy=256, lddx=256, t=moe.BF16):
    return moe.lib().moe_linear_grad(ctypes.byref(W), T, dy, lddy, t, dx, lddx, A, 1 << 40, A, None)


@pytest.mark.parametrize("kw", [
    dict(x=A, y=A), dict(x=A, y=A, T=1), dict(x=A, y=A, t=moe.F32), dict(x=A, y=A + 510, T=1), dict(x=A + 512, y=A, T=2),
    dict(x=A, y=A + 256, ldx=512, ldy=512), dict(x=A + 768, y=A, ldx=512, ldy=512, T=2),
    dict(x=A, y=A + (1 << 20), res=A + (1 << 20) + 2), dict(x=A, y=A + (1 << 20), res=A + (1 << 20) - 512),
    dict(x=A, y=A + (1 << 20), rb=A + (1 << 20) + 4), dict(x=A, y=A + 512, T=2, ldx=1024, ldy=256),
])
def test_linear_refuses_to_overwrite(kw):
    assert _linear(**kw) == moe.ERR_INVALID_ARG
    assert "overlaps" in moe.last_error()


@pytest.mark.parametrize("kw", [dict(dy=A, dx=A), dict(dy=A + 512, dx=A), dict(dy=A, dx=A + 16, T=1),
                                dict(dy=A, dx=A + 256, t=moe.F32, lddy=512, lddx=1024)])
def test_linear_grad_refuses_to_overwrite(kw):
    assert _grad(**kw) == moe.ERR_INVALID_ARG
    assert "overlaps" in moe.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 40])
def test_slices_of_one_buffer(T):
    g = torch.Generator("cuda").manual_seed(T)
    w = moe.QMatrix(4, 128, torch.randint(0, 256, (2, 256, 64), dtype=torch.uint8, device="cuda", generator=g),
                    *(0.01 * torch.rand(256, 2, device="cuda", generator=g).half() for _ in range(2)))
    wide = torch.randn(T, 768, device="cuda", generator=g).bfloat16()
    x, y, r = wide[:, 256:512], wide[:, :256], wide[:, 512:]
    apart = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
    moe.linear(w, x.contiguous(), apart, residual=r.contiguous())
    moe.linear(w, x, y, residual=r)
    assert torch.equal(y, apart)
    buf = moe.LinearBuffers.allocate(w, T, torch.bfloat16, grad=True)
    moe.linear_grad(w, r.contiguous(), apart, buf)
    moe.linear_grad(w, r, y, buf)
    assert torch.equal(y, apart)
