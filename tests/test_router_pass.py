"""The router's way back agrees with the step it goes back through: how the gates were
made, and the counts that the losses' gradient needs."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref


def _cpu():
    d = moe.dims(4, 256, 512, 8, 2)
    buf, grads = moe.LayerBuffers.allocate(d, 4, device="cpu"), moe.RouterGradBuffers.allocate(d, device="cpu")
    return buf, grads, torch.zeros(4, 256, dtype=torch.bfloat16)


def test_losses_gradient_needs_the_losses():
    buf, grads, out = _cpu()
    with pytest.raises(ValueError, match="router_losses"):
        moe.router_backward(buf, grads, out, torch.ones(2))
    grads.counted = True                                     # (as router_losses() leaves it)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.router_backward(buf, grads, out, torch.ones(2))
    grads.counted = False
    with pytest.raises(ValueError, match="on the GPU"):
        moe.router_backward(buf, grads, out)


@pytest.mark.parametrize("made", [True, False])
def test_gates_of_another_kind_are_refused(made):
    buf, grads, out = _cpu()
    buf.renormalize = made
    with pytest.raises(ValueError, match="renormalize"):
        moe.router_backward(buf, grads, out, renormalize=not made)
    for ask in (made, None):
        with pytest.raises(ValueError, match="on the GPU"):
            moe.router_backward(buf, grads, out, renormalize=ask)


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("fused", [True, False])
def test_the_way_back_goes_by_the_step(renormalize, fused):
    from gpu_util import upload_layer
    sh, T, dev = mi.CONFIGS["tiny"], 6, "cuda"
    L = upload_layer(sh, 4, 0)
    d = moe.dims(T, sh.H, sh.I, sh.E, sh.k, sh.group)
    buf, grads = moe.LayerBuffers.allocate(d, 4), moe.RouterGradBuffers.allocate(d)
    x = torch.randn(T, sh.H, device=dev).bfloat16().view(torch.int16)
    out = torch.empty_like(x)
    moe.layer_forward(buf, x, L.Wr_d, L.bias_d, L.weights_d, L.table_d, sh.E, x, out, renormalize=renormalize, fused=fused)
    assert buf.renormalize is renormalize
    out_grad = torch.randn(T, sh.H, device=dev).bfloat16()
    got = moe.router_backward(buf, grads, out_grad).double().cpu().numpy()
    f = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    want, mag = ref.route_backward(f(buf.logits), buf.topk_ids.cpu().numpy(), f(buf.topk_w), renormalize, f(grads.topk_w_grad))
    L64 = f(buf.logits)
    # the bound of the route's own test: 64 roundings, and the size of exp's argument
    assert np.all(np.abs(got - want) <= (64 + 4 * ref.spread(L64)) * ref.U32 * mag + 1e-37)
    with pytest.raises(ValueError, match="renormalize"):
        moe.router_backward(buf, grads, out_grad, renormalize=not renormalize)
