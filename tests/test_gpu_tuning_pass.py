"""The operators together, as a user tunes adapters and the router over frozen quantised weights:

    x0 -> quantised projection with each request's adapter -> layer step -> quantised head
    -> token log probabilities and entropy
    gradient: logits -> head's input -> router (gates from 8-bit expert rows, weight from the 8-bit
    layer input) and, by the residual, projection's input and the adapters' factors

each stage checked in 64 bits from the values the GPU had before it."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import quantized_expert_ffn_gemv_amd as moe
import tuning_ref as ref
import weights_ref as wref
from gpu_util import upload_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    worst = float(np.max(np.abs(f64(got) - want) / bound))
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


@pytest.mark.parametrize("T,graph", [(6, True), (150, False), (600, False)])
def test_tuning_pass(T, graph):
    sh = mi.CONFIGS["tiny"]
    H, E, k, V, K0, n, R = sh.H, sh.E, sh.k, 211, 384, 5, 12
    L = upload_layer(sh, 4, 0)
    rng = np.random.default_rng(T)
    mats = []
    for N, K, bits, group in ((H, K0, 2, 64), (V, H, 4, 128)):
        q, s, b = wref.make_matrix(rng, N, K, bits, group)
        mats.append((moe.QMatrix(bits, group, *(torch.from_numpy(a).to(DEV) for a in (q, s, b))), *wref.weights(q, s, b, bits, group)))
    (proj, Wp, magp), (head, Wh, magh) = mats
    ranks = rng.integers(1, R + 1, n)
    downs = [wref.bf16_round((rng.standard_normal((r, K0)) / 20).astype(np.float32)) for r in ranks]
    ups = [wref.bf16_round((0.3 * rng.standard_normal((H, r))).astype(np.float32)) for r in ranks]
    scales = rng.uniform(0.5, 2, n).astype(np.float32)
    m = moe.Adapters.pack([torch.from_numpy(a) for a in downs], [torch.from_numpy(a) for a in ups], scales)
    f = ref.Factors(rng, n, m.R, K0, H)
    f.a, f.b = m.a.float().cpu().numpy(), m.b.float().cpu().numpy()
    f.scale, f.rank = scales, None if m.rank is None else m.rank.cpu().numpy()
    ids_np = rng.integers(-1, n, T).astype(np.int32)
    ids = torch.from_numpy(ids_np).to(DEV)
    x0 = torch.from_numpy(wref.bf16_round(rng.standard_normal((T, K0)).astype(np.float32))).to(DEV, BF)
    tok = torch.from_numpy(rng.integers(-1, V, T).astype(np.int32)).to(DEV)

    d = moe.dims(T, H, sh.I, E, k, sh.group)
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    x, out, out_grad, dx0 = e(T, H, dt=BF), e(T, H, dt=BF), e(T, H, dt=BF), e(T, K0, dt=BF)
    h, logits, dlogits = e(T, m.R), e(T, V), e(T, V)
    logp, stats, ent, top_ids, top = e(T), e(T, 2), e(T), e(T, 3, dt=torch.int32), e(T, 3)
    da, db, dw, dbias = e(n, m.R, K0), e(n, m.R, H), e(E, H), e(E)
    w, u = torch.full((T,), -1.0 / T, device=DEV), torch.full((T,), -0.01 / T, device=DEV)
    cx0, cx, cy = moe.Checkpoint.allocate(T, K0), moe.Checkpoint.allocate(T, H), moe.Checkpoint.allocate(T * k, H)
    buf, grads = moe.LayerBuffers.allocate(d, 4), moe.RouterGradBuffers.allocate(d)
    ab = moe.AdaptedBuffers.allocate(proj, m, T, BF, grad=True)
    hb, hgb = moe.LinearBuffers.allocate(head, T, torch.float32), moe.LinearBuffers.allocate(head, T, torch.float32, grad=True)
    lb, rb = moe.LogprobBuffers.allocate(T, V, 3), moe.RouterWeightBuffers.allocate(d)
    xs, outs = x.view(torch.int16), out.view(torch.int16)
    kept_rows = e(T * k, H, dt=BF)

    def step():
        moe.adapted_linear(proj, m, ids, x0, x, ab, h=h)
        moe.checkpoint_save(x0, cx0)
        moe.layer_forward(buf, xs, L.Wr_d, L.bias_d, L.weights_d, L.table_d, E, xs, outs)
        moe.checkpoint_save(x, cx)
        moe.checkpoint_save(buf.y_rows[:T * k], cy)
        kept_rows.copy_(buf.y_rows[:T * k].view(BF))
        buf.y_rows.zero_()                                   # (another layer's step would use them)
        moe.linear(head, out, logits, hb)
        moe.logprobs(logits, tok, logp, stats, lb, entropy=ent, top_ids=top_ids, top_logp=top)
        moe.logprobs_grad(logits, tok, stats, dlogits, logp_grad=w, entropy=ent, entropy_grad=u)
        moe.linear_grad(head, dlogits, out_grad, hgb)
        moe.router_backward(buf, grads, out_grad, y_saved=cy, x=cx, w_router_grad=dw, router_bias_grad=dbias, weight_buffers=rb)
        moe.adapted_linear_backward(proj, m, ids, out_grad, cx0, h, ab, dx=dx0, da=da, db=db)

    step()
    torch.cuda.synchronize()
    assert buf.counters_clean()

    # the projection with its adapters: the projection is rounded to bf16 first
    xa = f64(x0)
    yp = wref.linear(xa, Wp)
    pb = wref.linear_bound(xa, Wp, magp, yp, False)
    wy, wh, yb, hbnd = ref.adapter(f, ids_np, xa, yp)
    within(h, wh, hbnd, "h")
    within(x, wy, ref.rounded(wy, yb + pb, False), "x")
    # scores
    Lg = f64(logits)
    wl, we, ws, wi, wt = ref.logprobs(Lg, tok.cpu().numpy(), 3)
    rel = (V / 32 + 80) * wref.U32
    assert np.all(np.abs(f64(logp) - wl) <= rel + 8 * wref.U32 * (1 + np.abs(wl)))
    assert np.array_equal(top_ids.cpu().numpy(), wi)
    # the loss' gradient: every probability off by a relative rel and its exponent's 2 U |log p|, the
    # entropy and log p by rel (2 + 2 log V) and their own roundings
    wd, mag = ref.logprobs_grad(Lg, tok.cpu().numpy(), f64(w), f64(u))
    lp = Lg - ws[:, :1] - ws[:, 1:]
    p = np.exp(lp)
    tol = rel + wref.U32 * (2 * np.abs(lp) + 24)
    both = np.abs(f64(w))[:, None] + np.abs(f64(u))[:, None] * (4 + 4 * np.log(V) + 2 * np.abs(lp))
    within(dlogits, wd, mag * tol + both * p * tol + 1e-37, "dlogits")
    want = f64(dlogits) @ Wh
    within(out_grad, want, wref.linear_grad_bound(f64(dlogits).astype(np.float32), Wh, magh, want), "out_grad")
    # gates' gradient from the saved rows, the router's from that, and its weight's
    Y = ref.restored(*ref.save(kept_rows.float().cpu().numpy()))
    p2r = buf.pair_to_row.cpu().numpy()[:T * k]
    terms = Y[p2r].reshape(T, k, H) * f64(out_grad)[:, None, :]
    within(grads.topk_w_grad, terms.sum(2), (H + 16) * wref.U32 * np.abs(terms).sum(2) + 1e-37, "gates")
    D, X = f64(grads.logits_grad), ref.restored(*ref.save(x.float().cpu().numpy()))
    within(dw, D.T @ X, (T + 64) * ref.SUM * (np.abs(D).T @ np.abs(X)) + 1e-37, "router weight")
    within(dbias, D.sum(0), (T + 16) * wref.U32 * np.abs(D).sum(0) + 1e-37, "router bias")
    # by the residual: the projection's input and the adapters
    dy = f64(out_grad)
    base = dy @ Wp
    bb = wref.linear_grad_bound(dy.astype(np.float32), Wp, magp, base)
    wx, wa, wb, xb, abnd, bbnd = ref.adapter_grad(f, ids_np, dy, ref.restored(*ref.save(x0.float().cpu().numpy())), f64(h), base)
    within(dx0, wx, ref.rounded(wx, xb + bb, False), "dx0")
    within(da, wa, abnd, "da")
    within(db, wb, bbnd, "db")

    if graph:
        outs_all = (x, h, out, logits, logp, ent, top_ids, dlogits, out_grad, dw, dbias, dx0, da, db)
        want = [o.clone() for o in outs_all]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for _ in range(3):
            for o in outs_all:
                o.fill_(5)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs_all, want))
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs_all, want))
