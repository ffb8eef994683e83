"""Activations kept in 8 bits, the combine's gates gradient from them and the router's weight
gradient on the GPU against the 64-bit forms of tuning_ref.py."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import tuning_ref as ref
from weights_ref import HALF_BF16, U32, bf16_round

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")
BF, F32 = torch.bfloat16, torch.float32


def dev(a, dtype=BF):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def strided(a, pad, shift):
    T, K = a.shape
    flat = torch.full((shift + T * (K + pad) + 8,), 7.0, dtype=BF, device=DEV)
    v = flat.as_strided((T, K), (K + pad, 1), shift)
    v.copy_(dev(a))
    return flat, v


def rows_of(rng, T, K):
    big = 1 + 12 * (rng.random(K) < 0.02)
    return bf16_round((rng.standard_normal((T, K)) * big * np.exp(3 * rng.standard_normal((T, 1)))).astype(np.float32))


def save(x, pad=0, shift=0):
    T, K = x.shape
    c = moe.Checkpoint(torch.full((T, K), 99, dtype=torch.int8, device=DEV), torch.full((T, K // 128), -7.0, device=DEV))
    moe.checkpoint_save(strided(x, pad, shift)[1], c)
    torch.cuda.synchronize()
    return c


@pytest.mark.parametrize("T,K,pad,shift", [(1, 128, 0, 0), (3, 384, 8, 8), (5, 128, 3, 1), (17, 2048, 1, 3), (64, 1152, 0, 0), (1000, 640, 5, 7), (3, 32768, 0, 0)])
def test_save_and_restore(T, K, pad, shift):
    x = rows_of(np.random.default_rng(T + K), T, K)
    c = save(x, pad, shift)
    q, s = ref.save(x)
    assert np.array_equal(c.q.cpu().numpy(), q) and np.array_equal(c.scale.cpu().numpy(), s)
    flat, out = strided(np.zeros_like(x), pad, shift)
    moe.checkpoint_restore(c, out)
    want = bf16_round((q.astype(np.float32) * np.repeat(s, 128, 1)))
    assert np.array_equal(out.float().cpu().numpy(), want)
    assert int((flat == 7.0).sum()) >= shift + (T - 1) * pad + 8        # nothing written around the rows


def test_ties_zeros_tiny_and_large():
    rng = np.random.default_rng(0)
    # every pair of 8-bit significands, among them all ties
    m = np.arange(128, 256)
    rows = []
    for k in (0, 1, 2, 3, 5, 6, 7, 9):
        rows += [np.concatenate([[a], np.minimum(m[1:] * 2.0 ** -k, a)]) for a in m[::5]]
    x = bf16_round(np.stack(rows).astype(np.float32))
    x *= np.where(rng.random(x.shape) < 0.5, -1, 1).astype(np.float32)
    for factor in (1.0, 2.0 ** -90, 2.0 ** -126, 2.0 ** 119):
        y = bf16_round((x.astype(np.float64) * factor).astype(np.float32))
        q, s = ref.save(y)
        c = save(y)
        assert np.array_equal(c.q.cpu().numpy(), q), factor
        assert np.array_equal(c.scale.cpu().numpy(), s), factor
    small = (rng.integers(-127, 128, (4, 256)) * 2.0 ** -133).astype(np.float32)          # below the smallest normal
    small[0, :128] = 0
    small[1, 128:] = 0
    small[1, 200] = 2.0 ** -133
    c = save(small)
    q, s = ref.save(small)
    assert np.array_equal(c.q.cpu().numpy(), q) and np.array_equal(c.scale.cpu().numpy(), s)


def test_groups_with_infinities_and_nans_read_as_nan():
    x = rows_of(np.random.default_rng(1), 6, 384)
    good = save(x)
    bad = x.copy()
    bad[1, 5], bad[2, 130], bad[3, 383], bad[3, 0] = np.nan, np.inf, -np.inf, np.nan
    c = save(bad)
    hit = np.zeros((6, 3), bool)
    hit[1, 0] = hit[2, 1] = hit[3, 2] = hit[3, 0] = True
    s = c.scale.cpu().numpy()
    assert np.isnan(s[hit]).all() and np.array_equal(s[~hit], good.scale.cpu().numpy()[~hit])
    wide = np.repeat(hit, 128, 1)
    q = c.q.cpu().numpy()
    assert (q[wide] == 0).all() and np.array_equal(q[~wide], good.q.cpu().numpy()[~wide])
    out = torch.empty(6, 384, dtype=BF, device=DEV)
    moe.checkpoint_restore(c, out)
    assert np.array_equal(np.isnan(out.float().cpu().numpy()), wide)


def test_rows_past_32_bits():
    """A checkpoint of more than 2^31 codes, rows far apart in the last ones."""
    T, K = 66000, 32768
    x = torch.zeros(T, K, dtype=BF, device=DEV)
    last = rows_of(np.random.default_rng(2), 4, K)
    x[-4:] = dev(last)
    c = moe.Checkpoint(torch.full((T, K), 5, dtype=torch.int8, device=DEV), torch.full((T, K // 128), NAN, device=DEV))
    moe.checkpoint_save(x, c)
    q, s = ref.save(last)
    assert np.array_equal(c.q[-4:].cpu().numpy(), q) and np.array_equal(c.scale[-4:].cpu().numpy(), s)
    assert int(c.q[:-4].any()) == 0 and float(c.scale[:-4].abs().max()) == 0
    x.fill_(1.0)
    moe.checkpoint_restore(c, x)
    assert np.array_equal(x[-4:].float().cpu().numpy(), bf16_round(q.astype(np.float32) * np.repeat(s, 128, 1)))
    assert float(x[:-4].float().abs().max()) == 0


@pytest.mark.parametrize("T,H,k,more", [(1, 128, 1, 0), (3, 256, 3, 2), (8, 5120, 2, 0), (60, 640, 9, 0), (300, 128, 4, 5), (200, 256, 5, 0), (700, 2048, 2, 0)])
def test_gates_gradient_from_a_checkpoint(T, H, k, more):
    rng = np.random.default_rng(T + H)
    P = T * k
    y = rows_of(rng, P + more, H)
    c = save(y)
    dout = bf16_round((1e-3 * rng.standard_normal((T, H))).astype(np.float32))
    p2r = rng.permutation(P).astype(np.int32)
    g = rng.random((T, k)).astype(np.float32)
    Y = ref.restored(*ref.save(y))
    if P > 2:
        p2r[1], p2r[2] = P + 3, -1                          # rows out of range
    d = moe.dims(T, H, 128, 64, k)
    for rows_grad in (False, True):
        dg = torch.full((T, k), NAN, device=DEV)
        dy = torch.full((P, H), 7.0, dtype=BF, device=DEV) if rows_grad else None
        moe.combine_backward(d, dev(dout), c, dev(p2r, torch.int32), dev(g, F32), dg, dy)
        ok = (p2r >= 0) & (p2r < P)
        at = np.where(ok, p2r, 0)
        terms = Y[at].reshape(T, k, H) * dout.astype(np.float64)[:, None, :]
        want = np.where(ok.reshape(T, k), terms.sum(2), 0.0)
        bound = np.where(ok.reshape(T, k), (H + 16) * U32 * np.abs(terms).sum(2), 0.0) + 1e-37
        got = dg.double().cpu().numpy()
        assert (np.abs(got - want) <= bound).all()
        if rows_grad:
            full = np.full((P, H), 7.0)
            vals = (g[:, :, None].astype(np.float64) * dout[:, None, :]).reshape(P, H)
            full[p2r[ok]] = vals[ok]
            o = dy.double().cpu().numpy()
            assert (np.abs(o - full) <= (HALF_BF16 + 2 * U32) * np.abs(full) * (full != 7.0) + 1e-37).all()


@pytest.mark.parametrize("T,E,H", [(0, 5, 128), (1, 1, 128), (7, 16, 256), (33, 17, 128), (100, 64, 384), (257, 33, 128), (700, 130, 256),
                                   (5000, 8, 128), (2100, 1024, 128), (300, 40, 8192)])
@pytest.mark.parametrize("saved", [False, True])
def test_router_weight_gradient(T, E, H, saved):
    rng = np.random.default_rng(T + E)
    x = rows_of(rng, T, H)
    dl = (1e-3 * np.exp(2 * rng.standard_normal((T, 1))) * rng.standard_normal((T, E))).astype(np.float32)
    d = moe.dims(T, H, 128, E, 1)
    buf = moe.RouterWeightBuffers.allocate(d)
    buf.workspace.fill_(0xFF)
    kept = (save(x) if T else moe.Checkpoint.allocate(0, H)) if saved else strided(x, 3, 1)[1] if T else torch.empty(0, H, dtype=BF, device=DEV)
    X = (ref.restored(*ref.save(x)) if saved else x.astype(np.float64)) if T else np.zeros((0, H))
    outs = []
    for bias in (True, False, True):
        dw = torch.full((E, H), NAN, device=DEV)
        db = torch.full((E,), NAN, device=DEV) if bias else None
        moe.router_weight_grad(d, dev(dl, F32), kept, dw, buf, bias_grad=db)
        torch.cuda.synchronize()
        D = dl.astype(np.float64)
        # a checkpoint's scale goes into d logits by one product more
        bound = (T + 64) * ref.SUM * (np.abs(D).T @ np.abs(X)) + 1e-37
        got = dw.double().cpu().numpy()
        assert np.isfinite(got).all() and (np.abs(got - D.T @ X) <= bound).all()
        if bias:
            assert (np.abs(db.double().cpu().numpy() - D.sum(0)) <= (T + 16) * U32 * np.abs(D).sum(0) + 1e-37).all()
        outs.append((dw, db))
    assert torch.equal(outs[0][0], outs[2][0]) and torch.equal(outs[0][1], outs[2][1]) and torch.equal(outs[0][0], outs[1][0])


def test_router_weight_gradient_keeps_bad_rows_in_their_columns():
    rng = np.random.default_rng(4)
    T, E, H = 90, 20, 384
    x, dl = rows_of(rng, T, H), rng.standard_normal((T, E)).astype(np.float32)
    d = moe.dims(T, H, 128, E, 1)
    buf = moe.RouterWeightBuffers.allocate(d)
    good, got = torch.empty(E, H, device=DEV), torch.empty(E, H, device=DEV)
    for saved in (False, True):
        bad = x.copy()
        bad[17, 200] = np.nan
        a, b = (save(x), save(bad)) if saved else (dev(x), dev(bad))
        moe.router_weight_grad(d, dev(dl, F32), a, good, buf)
        moe.router_weight_grad(d, dev(dl, F32), b, got, buf)
        hit = torch.zeros(H, dtype=torch.bool, device=DEV)
        hit[128:256] = saved
        hit[200] = True
        assert bool(torch.isnan(got[:, hit]).all()) and torch.equal(got[:, ~hit], good[:, ~hit])


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(5)
    T, H, k, E = 40, 256, 3, 24
    d = moe.dims(T, H, 128, E, k)
    x, y = dev(rows_of(rng, T, H)), dev(rows_of(rng, T * k, H))
    cx, cy = moe.Checkpoint.allocate(T, H), moe.Checkpoint.allocate(T * k, H)
    back, dout = torch.empty_like(x), dev(rng.standard_normal((T, H)).astype(np.float32))
    p2r, g = dev(rng.permutation(T * k).astype(np.int32), torch.int32), torch.rand(T, k, device=DEV)
    dg, dl = torch.empty(T, k, device=DEV), torch.randn(T, E, device=DEV)
    dw, db = torch.empty(E, H, device=DEV), torch.empty(E, device=DEV)
    buf = moe.RouterWeightBuffers.allocate(d)

    def step():
        moe.checkpoint_save(x, cx)
        moe.checkpoint_save(y, cy)
        moe.checkpoint_restore(cx, back)
        moe.combine_backward(d, dout, cy, p2r, g, dg)
        moe.router_weight_grad(d, dl, cx, dw, buf, bias_grad=db)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (cx.q, cx.scale, cy.q, cy.scale, back, dg, dw, db)
    for k2 in range(4):
        x.copy_(dev(rows_of(rng, T, H)))
        dl.normal_()
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {k2}"
