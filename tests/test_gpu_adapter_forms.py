"""Every kernel form of the adapters and of the router's weight gradient, at the sizes of
adapter_forms.py: dense operands within the bounds of tuning_ref.py, and operands few of which are
not zero, whose results show all 24 bits of h, g and a float32 dy."""
import numpy as np
import pytest
import torch

import adapter_forms as forms
import quantized_expert_ffn_gemv_amd as moe
import test_gpu_adapters as gpu
import tuning_ref as ref
from weights_ref import U32, bf16_round

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", forms.CASES, ids=str)
def test_dense(case):
    T, n, R, K, N, f32 = case
    rng = np.random.default_rng(T + n + R)
    f = ref.Factors(rng, n, R, K, N, ragged=n > 2)
    m = gpu.upload(f, 1)
    ids = gpu.make_ids(rng, T, n, none=True, skew=n == 3)
    x = bf16_round(rng.standard_normal((T, K)).astype(np.float32))
    base = rng.standard_normal((T, N)).astype(np.float32)
    base = base if f32 else bf16_round(base)
    y, h = gpu.run_forward(f, m, ids, x, base, f32, 3, in_place=True)
    wy, wh, yb, hb = ref.adapter(f, ids, x, base)
    gpu.check(h, wh, hb, "h")
    gpu.check(y, wy, ref.rounded(wy, yb, f32), "y")
    dy = (1e-3 * np.exp(2 * rng.standard_normal((T, 1))) * rng.standard_normal((T, N))).astype(np.float32)
    dy = dy if f32 else bf16_round(dy)
    hv = rng.standard_normal((T, R)).astype(np.float32)
    xs = ref.restored(*ref.save(x))
    for saved in (False, True):
        dx, da, db = gpu.run_grad(f, m, ids, dy, x, hv, None, f32, 5, saved=saved)
        wx, wa, wb, xb, ab, bb = ref.adapter_grad(f, ids, dy, xs if saved else x, hv)
        gpu.check(dx, wx, ref.rounded(wx, xb, False), "dx")
        gpu.check(da, wa, ab, f"da saved={saved}")
        gpu.check(db, wb, bb, "db")


@pytest.mark.parametrize("case", forms.CASES, ids=str)
def test_every_bit(case):
    f32 = case[-1]
    s = forms.Sparse(*case)
    m = gpu.upload(s.f)
    _, h = gpu.run_forward(s.f, m, s.ids, s.x_dense, None, f32)
    part, bound = s.y(h.cpu().numpy())
    # a bf16 y: what the adapters' part nearly cancels, so that rounding hides little of it
    base = np.zeros_like(part, np.float32) if f32 else bf16_round(-part.astype(np.float32))
    y, again = gpu.run_forward(s.f, m, s.ids, s.x_dense, base, f32)
    assert torch.equal(h, again)
    want = base + part
    gpu.check(y, want, ref.rounded(want, bound + 2 * U32 * (np.abs(base) + np.abs(want)), f32), "y")
    for saved in (False, True):
        dx, da, db = gpu.run_grad(s.f, m, s.ids, s.dy, s.x, s.h, s.base, f32, saved=saved)
        wx, wa, wb, xb, ab, bb = s.gradients(ref.restored(*ref.save(s.x)) if saved else s.x.astype(np.float64))
        gpu.check(dx, wx, xb, "dx")
        gpu.check(da, wa, ab, f"da saved={saved}")
        gpu.check(db, wb, bb, "db")


@pytest.mark.parametrize("T,E,H", forms.ROUTER)
@pytest.mark.parametrize("saved", [False, True])
def test_router_weight(T, E, H, saved):
    rng = np.random.default_rng(T + H)
    d = moe.dims(T, H, 128, E, 1)
    buf = moe.RouterWeightBuffers.allocate(d)
    sparse, some, steps = forms.router_operands(T, E, H)
    dense = (1e-3 * np.exp(2 * rng.standard_normal((T, 1))) * rng.standard_normal((T, E))).astype(np.float32)
    rows = bf16_round(rng.standard_normal((T, H)).astype(np.float32))
    for dl, x, step in ((dense, rows, (T + 64) * ref.SUM), (sparse, some, steps)):
        kept, X = gpu.dev(x), x.astype(np.float64)
        if saved:
            c = moe.Checkpoint.allocate(T, H)
            moe.checkpoint_save(kept, c)
            kept, X = c, ref.restored(*ref.save(x))
        buf.workspace.fill_(0xFF)
        dw, db = torch.full((E, H), float("nan"), device="cuda"), torch.full((E,), float("nan"), device="cuda")
        moe.router_weight_grad(d, gpu.dev(dl, torch.float32), kept, dw, buf, bias_grad=db)
        D = dl.astype(np.float64)
        gpu.check(dw, D.T @ X, step * (np.abs(D).T @ np.abs(X)) + ref.TINY, "weight")
        gpu.check(db, D.sum(0), (T + 16) * U32 * np.abs(D).sum(0) + ref.TINY, "bias")


@pytest.mark.parametrize("T", [30, 600])
@pytest.mark.parametrize("f32", [False, True])
def test_infinities_are_nan_where_they_enter(T, f32):
    """As the header says: an infinite h, g or float32 dy is three parts that are no numbers, an infinite
    bf16 operand may give either; everything else keeps its bits."""
    rng = np.random.default_rng(T)
    f = ref.Factors(rng, 3, 8, 128, 24)
    m = gpu.upload(f)
    ids = gpu.make_ids(rng, T, 3)
    t, i = 5, int(ids[5])
    x, dy = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (128, 24))
    hv = rng.standard_normal((T, 8)).astype(np.float32)
    others, rest = [k for k in range(3) if k != i], torch.arange(T, device="cuda") != t
    good = gpu.run_forward(f, m, ids, x, None, f32), gpu.run_grad(f, m, ids, dy, x, hv, None, f32)
    bad = x.copy()
    bad[t, 9] = np.inf
    y, h = gpu.run_forward(f, m, ids, bad, None, f32)
    assert bool(torch.isinf(h[t]).all()) and bool(torch.isnan(y[t]).all())
    assert torch.equal(y[rest], good[0][0][rest]) and torch.equal(h[rest], good[0][1][rest])
    dx, da, db = gpu.run_grad(f, m, ids, dy, bad, hv, None, f32)
    assert torch.equal(dx, good[1][0]) and torch.equal(db, good[1][2]) and torch.equal(da[others], good[1][1][others])
    keep = torch.arange(128, device="cuda") != 9
    assert not bool(torch.isfinite(da[i, :, 9]).any()) and torch.equal(da[i][:, keep], good[1][1][i][:, keep])
    bad = dy.copy()
    bad[t, 3] = -np.inf
    dx, da, db = gpu.run_grad(f, m, ids, bad, x, hv, None, f32)
    assert bool(torch.isnan(dx[t]).all()) and torch.equal(dx[rest], good[1][0][rest])
    assert bool(torch.isnan(da[i]).all()) and torch.equal(da[others], good[1][1][others])
    keep = torch.arange(24, device="cuda") != 3
    assert not bool(torch.isfinite(db[i, :, 3]).any()) and torch.equal(db[:, :, keep], good[1][2][:, :, keep])
    assert torch.equal(db[others], good[1][2][others])
    d = moe.dims(T, 128, 128, 8, 1)
    buf, dl = moe.RouterWeightBuffers.allocate(d), gpu.dev(hv, torch.float32)
    a, b = torch.empty(8, 128, device="cuda"), torch.empty(8, 128, device="cuda")
    moe.router_weight_grad(d, dl, gpu.dev(x), a, buf)
    dl[t, 2] = float("inf")
    moe.router_weight_grad(d, dl, gpu.dev(x), b, buf)
    rows = torch.arange(8, device="cuda") != 2
    assert bool(torch.isnan(b[2]).all()) and torch.equal(a[rows], b[rows])


@pytest.mark.parametrize("T,n,R", [(3, 5, 8), (40, 200, 8), (40, 200, 24), (700, 7, 8), (700, 7, 40), (600, 150, 8)])
def test_adapters_without_a_token_may_hold_anything(T, n, R):
    """An empty slot of a set: its factors' gradients are 0 whatever its scale, rank and factors are."""
    rng = np.random.default_rng(T + R)
    f = ref.Factors(rng, n, R, 384, 264)
    used = rng.choice(n, max(1, n // 3), False)
    ids = used[rng.integers(0, len(used), T)].astype(np.int32)
    empty = np.setdiff1d(np.arange(n), ids)
    x, dy = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (384, 264))
    h = rng.standard_normal((T, R)).astype(np.float32)
    want = gpu.run_grad(f, gpu.upload(f), ids, dy, x, h, None, False)
    f.rank = np.full(n, R, np.int32)
    f.scale[empty] = rng.choice(np.array([np.nan, np.inf, -np.inf], np.float32), len(empty))
    f.a[empty], f.b[empty], f.rank[empty] = np.nan, np.inf, rng.integers(-3, 2 * R, len(empty))
    got = gpu.run_grad(f, gpu.upload(f), ids, dy, x, h, None, False)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    assert bool((got[1][empty] == 0).all()) and bool((got[2][empty] == 0).all())
