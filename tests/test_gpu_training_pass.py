"""The operators together, as a user tunes the router over frozen quantised weights:

    x0 -> linear (quantised projection) -> layer step -> linear (quantised head, float32 logits)
    loss = <logits, r> + a balance + z z-loss
    head logits' gradient -> linear_grad -> router_backward (combine, route) -> d router logits

checked against float64 autograd from the GPU's own intermediate values (each stage's
inputs as the GPU had them, so that only that stage's roundings are left)."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref
from gpu_util import to_dev, upload_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu()


@pytest.mark.parametrize("T,shared", [(4, False), (150, False), (8, True)])
def test_router_training_pass(T, shared):
    sh = mi.CONFIGS["tiny"]
    H, E, k, V = sh.H, sh.E, sh.k, 203
    L = upload_layer(sh, 4, 0)
    rng = np.random.default_rng(T)
    mats = []
    for N, K, bits, group in ((H, 384, 2, 64), (V, H, 4, 128)):
        q, s, b = ref.make_matrix(rng, N, K, bits, group)
        mats.append((moe.QMatrix(bits, group, *(torch.from_numpy(a).to(DEV) for a in (q, s, b))),
                     *ref.weights(q, s, b, bits, group)))
    (proj, Wp, magp), (head, Wh, magh) = mats
    x0 = ref.bf16_round(rng.standard_normal((T, 384)).astype(np.float32))
    x0_d = torch.from_numpy(x0).to(DEV, torch.bfloat16)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    moe.linear(proj, x0_d, x, moe.LinearBuffers.allocate(proj, T, x.dtype))
    want = ref.linear(x0, Wp)
    assert np.all(np.abs(f64(x).numpy() - want) <= ref.linear_bound(x0, Wp, magp, want, False))

    d = moe.dims(T, H, sh.I, E, k, sh.group)
    buf = moe.LayerBuffers.allocate(d, 4, shared_rows=shared)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    xs, outs = x.view(torch.int16), out.view(torch.int16)
    kw = {}
    if shared:
        W = mi.make_expert_weights(sh, 4, 1, experts=[0])
        one = moe.QWeights(4, [to_dev(moe.group_major(W.q[m], 4)) for m in mi.MATRICES],
                           [to_dev(W.scale[m]) for m in mi.MATRICES], [to_dev(W.bias[m]) for m in mi.MATRICES])
        fused = moe.QWeights(4, *[[torch.cat([a, b]) for a, b in zip(getattr(L.weights_d, n), getattr(one, n))]
                                  for n in ("q", "scale", "bias")])
        kw = dict(shared=moe.SharedExpert(one, torch.randn(H, device=DEV) * 0.02, sh.I, fused))
    moe.layer_forward(buf, xs, L.Wr_d, L.bias_d, L.weights_d, L.table_d, E, xs, outs, **kw)
    logits = torch.empty(T, V, device=DEV)
    moe.linear(head, out, logits, moe.LinearBuffers.allocate(head, T, logits.dtype))
    out_np = f64(out).numpy()
    want = ref.linear(out_np, Wh)
    assert np.all(np.abs(f64(logits).numpy() - want) <= ref.linear_bound(out_np, Wh, magh, want, True))

    grads = moe.RouterGradBuffers.allocate(d)
    valid = torch.ones(T, dtype=torch.bool, device=DEV)
    valid[T - 1] = False
    losses = moe.router_losses(buf, grads, valid)
    c, P, n, bal, z = ref.balance(f64(buf.logits).numpy(), buf.topk_ids.cpu().numpy(), k, valid.cpu().numpy())
    assert np.array_equal(grads.counts.cpu().numpy(), c) and int(grads.n_valid) == n == T - 1
    np.testing.assert_allclose(f64(losses).numpy(), [bal, z], rtol=(64 + T) * ref.U32 * 4)

    # backward
    r = rng.standard_normal((T, V)).astype(np.float32) * 1e-2
    out_grad = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    r_d = torch.from_numpy(r).to(DEV)
    moe.linear_grad(head, r_d, out_grad, moe.LinearBuffers.allocate(head, T, r_d.dtype, grad=True))
    want = r.astype(np.float64) @ Wh
    assert np.all(np.abs(f64(out_grad).numpy() - want) <= ref.linear_grad_bound(r, Wh, magh, want))
    y_grad = torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV)
    a, zc = 0.05, 0.01
    dl = moe.router_backward(buf, grads, out_grad, torch.tensor([a, zc], device=DEV), valid, y_grad)
    torch.cuda.synchronize()
    assert buf.counters_clean()

    # the same through autograd in float64, from the GPU's logits, rows and output gradient
    Lg = f64(buf.logits).requires_grad_(True)
    ids = buf.topk_ids.cpu().long()
    g = torch.softmax(torch.gather(Lg, 1, ids), 1)
    Y = f64(buf.y_rows.view(torch.bfloat16))[buf.pair_to_row.cpu().long()[:T * k]].view(T, k, H)
    dout = f64(out_grad)
    m = f64(valid)
    f = torch.from_numpy(c / (n * k))
    total = ((g[:, :, None] * Y).sum(1) * dout).sum() + a * E * (f * (torch.softmax(Lg, 1) * m[:, None]).sum(0) / n).sum() \
        + zc * (torch.logsumexp(Lg, 1) ** 2 * m).sum() / n
    total.backward()
    dg_mag = (Y.abs() * dout.abs()[:, None]).sum(2)
    # dg is a sum of H products (H U of their sizes), g off by 2e-6; the rest as in the route's own test
    bound = (2 * H * ref.U32 + 4e-6) * dg_mag.sum(1, keepdim=True) + (64 + 4 * 16) * ref.U32 * (a * E + zc * 16 * 2)
    assert bool(((f64(dl) - Lg.grad).abs() <= bound).all())
    rows = buf.pair_to_row.cpu().long()[:T * k]
    want = (f64(buf.topk_w)[:, :, None] * dout[:, None]).view(T * k, H)
    got = f64(y_grad)[rows]
    assert bool(((got - want).abs() <= (ref.HALF_BF16 + 2 * ref.U32) * want.abs() + 1e-38).all())
    # the router weight's gradient, as a user takes it
    dW = f64(dl).t() @ f64(x)
    assert dW.shape == (E, H) and bool(torch.isfinite(dW).all()) and float(dW.abs().max()) > 0
