"""Low-rank adapters and their gradients on the GPU against the 64-bit forms of
tuning_ref.py, with its bounds."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import tuning_ref as ref
from weights_ref import bf16_round

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")
BF, F32 = torch.bfloat16, torch.float32


def dev(a, dtype=BF):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def wide(a, pad, dtype=BF):
    """a's values as the first columns of a wider buffer of NaNs."""
    buf = torch.full((a.shape[0], a.shape[1] + pad), NAN, dtype=dtype, device=DEV)
    buf[:, :a.shape[1]] = dev(a, dtype)
    return buf[:, :a.shape[1]]


def upload(f, pad=0):
    """The set on the GPU; what is past the ranks and in b's padding is NaN."""
    a, b = f.a.copy(), np.full((f.n, f.R, (f.N + 7) // 8 * 8 + 8 * pad), np.nan, np.float32)
    b[:, :, :f.N] = f.b
    if f.rank is not None:
        for i, r in enumerate(f.rank):
            a[i, max(int(r), 0):], b[i, max(int(r), 0):] = np.nan, np.nan
    return moe.Adapters(dev(a), dev(b)[:, :, :f.N], dev(f.scale, F32), None if f.rank is None else dev(f.rank, torch.int32))


def make_ids(rng, T, n, mixed=True, none=False, skew=False):
    ids = rng.integers(0, n, T)
    if skew:
        ids[rng.random(T) < 0.8] = n // 2
    if not mixed:
        ids = np.sort(ids)
    if none:
        ids[rng.random(T) < 0.15] = -1
    return ids.astype(np.int32)


def check(got, want, bound, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    worst = float(np.max(np.abs(got - want) / bound)) if want.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def run_forward(f, m, ids, x, base, f32, pad=0, in_place=False, buf=None, rows=3):
    T = len(ids)
    dt = F32 if f32 else BF
    ybuf = torch.full((T + rows, f.N + pad + 1), 7.0, dtype=dt, device=DEV)
    y = ybuf[:T, :f.N]
    bd = None
    if base is not None:
        bd = wide(base, pad, dt)
        if in_place:
            y.copy_(bd)
            bd = y
    h = torch.full((T, f.R), NAN, device=DEV)
    if buf is None:
        buf = moe.AdapterBuffers.allocate(m, T)
        buf.workspace.fill_(0xFF)
    if not in_place:
        y.fill_(NAN)
    moe.adapter(m, dev(ids, torch.int32), wide(x, pad), y, buf, base=bd, h=h)
    torch.cuda.synchronize()
    assert bool((ybuf[T:] == 7.0).all()) and bool((ybuf[:, f.N:] == 7.0).all()), "wrote outside y"
    return y, h


def run_grad(f, m, ids, dy, x, h, base, f32, pad=0, in_place=False, saved=False, buf=None, want=("dx", "da", "db")):
    T = len(ids)
    dxbuf = torch.full((T + 2, f.K + pad), 7.0, dtype=BF, device=DEV)
    dx = dxbuf[:T, :f.K]
    bd = None
    if base is not None:
        bd = wide(base, pad)
        if in_place:
            dx.copy_(bd)
            bd = dx
    if not in_place:
        dx.fill_(NAN)
    da, db = torch.full((f.n, f.R, f.K), NAN, device=DEV), torch.full((f.n, f.R, f.N), NAN, device=DEV)
    if buf is None:
        buf = moe.AdapterBuffers.allocate(m, T, grad=True)
        buf.workspace.fill_(0xFF)
    kept = wide(x, pad)
    if saved:
        c = moe.Checkpoint.allocate(T, f.K)
        moe.checkpoint_save(kept, c)
        kept = c
    kw = {k: v for k, v in (("dx", dx), ("da", da), ("db", db)) if k in want}
    if "dx" in want:
        kw["dx_base"] = bd
    moe.adapter_grad(m, dev(ids, torch.int32), wide(dy, pad, F32 if f32 else BF), kept, dev(h, F32), buf, **kw)
    torch.cuda.synchronize()
    assert bool((dxbuf[T:] == 7.0).all()) and bool((dxbuf[:, f.K:] == 7.0).all()), "wrote outside dx"
    return dx, da, db


# T, n, R, K, N, ragged, mixed, none, skew, f32, pad
CASES = [
    (1, 1, 16, 128, 8, False, True, False, False, False, 0),
    (1, 3, 1, 384, 9, False, True, False, False, True, 8),
    (2, 5, 3, 128, 17, True, True, False, False, False, 3),
    (15, 1, 16, 2048, 130, False, True, False, False, False, 0),
    (17, 1, 17, 256, 129, False, True, True, False, True, 1),
    (33, 2, 32, 640, 513, True, False, True, False, False, 5),
    (48, 32, 16, 1024, 1000, True, True, True, False, False, 0),
    (64, 200, 33, 384, 250, True, True, False, False, False, 8),
    (100, 4, 64, 512, 264, False, True, True, True, True, 0),
    (129, 3, 128, 256, 1025, True, False, False, False, False, 2),
    (512, 7, 8, 256, 72, False, True, True, True, False, 0),
    (513, 7, 8, 256, 72, True, True, True, True, False, 0),
    (513, 1, 128, 128, 15, False, True, False, False, True, 1),
    (700, 64, 16, 384, 136, True, True, True, False, False, 8),
    (1500, 5, 48, 256, 200, True, False, True, True, False, 0),
    (3001, 2, 20, 128, 24, False, True, True, True, True, 3),
    (2600, 1024, 4, 128, 33, True, True, True, False, False, 0),
]


@pytest.mark.parametrize("T,n,R,K,N,ragged,mixed,none,skew,f32,pad", CASES)
def test_forward(T, n, R, K, N, ragged, mixed, none, skew, f32, pad):
    rng = np.random.default_rng(T + n)
    f = ref.Factors(rng, n, R, K, N, ragged)
    m = upload(f, pad % 3)
    ids = make_ids(rng, T, n, mixed, none, skew)
    x = bf16_round(rng.standard_normal((T, K)).astype(np.float32))
    base = rng.standard_normal((T, N)).astype(np.float32)
    base = base if f32 else bf16_round(base)
    for b, in_place in ((base, False), (base, True), (None, False)):
        y, h = run_forward(f, m, ids, x, b, f32, pad, in_place)
        wy, wh, yb, hb = ref.adapter(f, ids, x, b)
        check(h, wh, hb, "h")
        check(y, wy, ref.rounded(wy, yb, f32), f"y {in_place}")
    if none:
        off = torch.from_numpy(ids < 0).to(DEV)
        y, h = run_forward(f, m, ids, x, base, f32, pad)
        assert bool((h[off] == 0).all()) and torch.equal(y[off], dev(base, y.dtype)[off])


@pytest.mark.parametrize("T,n,R,K,N,ragged,mixed,none,skew,f32,pad", CASES)
def test_gradients(T, n, R, K, N, ragged, mixed, none, skew, f32, pad):
    rng = np.random.default_rng(T + n + 1)
    f = ref.Factors(rng, n, R, K, N, ragged)
    m = upload(f, pad % 3)
    ids = make_ids(rng, T, n, mixed, none, skew)
    x = bf16_round(rng.standard_normal((T, K)).astype(np.float32))
    dy = (1e-3 * np.exp(2 * rng.standard_normal((T, 1))) * rng.standard_normal((T, N))).astype(np.float32)
    dy = dy if f32 else bf16_round(dy)
    h = rng.standard_normal((T, R)).astype(np.float32)
    base = bf16_round((1e-3 * rng.standard_normal((T, K))).astype(np.float32))
    xs = ref.restored(*ref.save(x))
    for saved, in_place, b in ((False, False, base), (True, True, base), (False, False, None)):
        dx, da, db = run_grad(f, m, ids, dy, x, h, b, f32, pad, in_place, saved)
        wx, wa, wb, xb, ab, bb = ref.adapter_grad(f, ids, dy, xs if saved else x, h, b)
        check(dx, wx, ref.rounded(wx, xb, False), "dx")
        check(da, wa, ab, f"da saved={saved}")
        check(db, wb, bb, "db")
        again = run_grad(f, m, ids, dy, x, h, b, f32, pad, in_place, saved)
        assert all(torch.equal(p, q) for p, q in zip((dx, da, db), again)), "equal calls differ"


def test_each_gradient_alone():
    rng = np.random.default_rng(9)
    f = ref.Factors(rng, 3, 8, 256, 40)
    m = upload(f)
    for T in (20, 600):
        ids = make_ids(rng, T, 3, none=True)
        x, dy = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (256, 40))
        h = rng.standard_normal((T, 8)).astype(np.float32)
        every = run_grad(f, m, ids, dy, x, h, None, False)
        for k, name in enumerate(("dx", "da", "db")):
            got = run_grad(f, m, ids, dy, x, h, None, False, want=(name,))
            assert torch.equal(got[k], every[k])
            assert all(bool(torch.isnan(got[o]).all()) for o in range(3) if o != k)


def test_no_adapter_and_ids_out_of_range():
    rng = np.random.default_rng(10)
    f = ref.Factors(rng, 4, 8, 128, 24)
    m = upload(f)
    for T in (6, 520):
        ids = rng.choice(np.array([-1, 4, 1000, -2 ** 31, 2 ** 31 - 1], np.int64), T).astype(np.int32)
        x, base = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (128, 24))
        y, h = run_forward(f, m, ids, x, base, False)
        assert torch.equal(y, dev(base)) and bool((h == 0).all())
        dx, da, db = run_grad(f, m, ids, base, x, np.ones((T, 8), np.float32), x, False)
        assert torch.equal(dx, dev(x)) and bool((da == 0).all()) and bool((db == 0).all())


def test_ranks_out_of_range_count_as_the_nearer_end():
    rng = np.random.default_rng(11)
    f = ref.Factors(rng, 3, 8, 128, 24)
    f.rank = np.array([-5, 100, 3], np.int32)
    m = upload(f)
    ids = np.array([0, 1, 2, 1, 0], np.int32)
    x = bf16_round(rng.standard_normal((5, 128)).astype(np.float32))
    y, h = run_forward(f, m, ids, x, None, True)
    wy, wh, yb, hb = ref.adapter(f, ids, x)
    check(y, wy, yb, "y")
    assert bool((h[ids == 0] == 0).all())


def test_bad_rows_stay_with_their_token_and_adapter():
    rng = np.random.default_rng(12)
    f = ref.Factors(rng, 3, 16, 256, 40)
    m = upload(f)
    for T in (30, 600):
        ids = make_ids(rng, T, 3)
        x, dy = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (256, 40))
        h = rng.standard_normal((T, 16)).astype(np.float32)
        good = run_forward(f, m, ids, x, None, False)
        ggood = run_grad(f, m, ids, dy, x, h, None, False)
        bad = x.copy()
        bad[4, 7], bad[4, 9] = np.inf, np.nan
        y, hh = run_forward(f, m, ids, bad, None, False)
        rest = torch.arange(T, device=DEV) != 4
        assert torch.equal(y[rest], good[0][rest]) and torch.equal(hh[rest], good[1][rest])
        assert not bool(torch.isfinite(y[4]).any())
        for saved in (False, True):
            g = run_grad(f, m, ids, dy, bad, h, None, False, saved=saved)
            others = [i for i in range(3) if i != ids[4]]
            if not saved:
                assert torch.equal(g[1][others], ggood[1][others])
            assert bool(torch.isfinite(g[1][others]).all()) and bool(torch.isnan(g[1][ids[4], :, 9]).all())
            assert torch.equal(g[0], ggood[0]) and torch.equal(g[2], ggood[2])
        bad = dy.copy()
        bad[4, 3] = np.nan
        g = run_grad(f, m, ids, bad, x, h, None, False)
        assert torch.equal(g[0][rest], ggood[0][rest]) and bool(torch.isnan(g[0][4]).all())
        assert torch.equal(g[2][others], ggood[2][others]) and torch.equal(g[2][:, :, 4], ggood[2][:, :, 4])


def test_no_tokens_clear_the_gradients():
    rng = np.random.default_rng(13)
    f = ref.Factors(rng, 3, 20, 128, 24)
    m = upload(f)
    da, db = torch.full((3, 20, 128), NAN, device=DEV), torch.full((3, 20, 24), NAN, device=DEV)
    e = lambda c, dt=BF: torch.empty(0, c, dtype=dt, device=DEV)  # noqa: E731
    moe.adapter_grad(m, torch.empty(0, dtype=torch.int32, device=DEV), e(24), e(128), e(20, F32),
                     moe.AdapterBuffers.allocate(m, 0, grad=True), dx=e(128), da=da, db=db)
    assert bool((da == 0).all()) and bool((db == 0).all())


def test_buffers_serve_fewer_tokens_and_streams():
    rng = np.random.default_rng(14)
    f = ref.Factors(rng, 6, 16, 256, 72)
    m = upload(f)
    buf, gbuf = moe.AdapterBuffers.allocate(m, 2000), moe.AdapterBuffers.allocate(m, 2000, grad=True)
    side = torch.cuda.Stream()
    for T in (2000, 513, 512, 3, 700, 1):
        ids = make_ids(rng, T, 6, none=True)
        x, dy = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (256, 72))
        h = rng.standard_normal((T, 16)).astype(np.float32)
        fresh, gfresh = run_forward(f, m, ids, x, None, False), run_grad(f, m, ids, dy, x, h, None, False)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got, ggot = run_forward(f, m, ids, x, None, False, buf=buf), run_grad(f, m, ids, dy, x, h, None, False, buf=gbuf)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(fresh + gfresh, got + ggot))


@pytest.mark.parametrize("T", [24, 1100])
def test_captured_and_replayed(T):
    rng = np.random.default_rng(15)
    f = ref.Factors(rng, 4, 16, 256, 136)
    m = upload(f)
    ids = dev(make_ids(rng, T, 4, none=True), torch.int32)
    x, dy = (dev(rng.standard_normal((T, c)).astype(np.float32)) for c in (256, 136))
    y, dx = torch.empty(T, 136, dtype=BF, device=DEV), torch.empty(T, 256, dtype=BF, device=DEV)
    h = torch.empty(T, 16, device=DEV)
    da, db = torch.empty(4, 16, 256, device=DEV), torch.empty(4, 16, 136, device=DEV)
    buf, gbuf = moe.AdapterBuffers.allocate(m, T), moe.AdapterBuffers.allocate(m, T, grad=True)

    def step():
        moe.adapter(m, ids, x, y, buf, h=h)
        moe.adapter_grad(m, ids, dy, x, h, gbuf, dx=dx, da=da, db=db)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (y, h, dx, da, db)
    for k in range(4):
        x.copy_(torch.randn_like(x, dtype=F32))
        ids.copy_(dev(make_ids(rng, T, 4, none=True, skew=k % 2 == 1), torch.int32))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {k}"


def test_far_row_strides():
    """Rows more than 2^31 elements from the first."""
    rng = np.random.default_rng(16)
    f = ref.Factors(rng, 2, 8, 128, 16)
    m = upload(f)
    T, ld = 67, (1 << 25) + 8
    flat = torch.empty(T * ld, dtype=BF, device=DEV)
    far = lambda off, c: flat[off:].as_strided((T, c), (ld, 1), flat.storage_offset() + off)  # noqa: E731
    x, y, dy, dx = far(0, 128), far(256, 16), far(512, 16), far(1024, 128)
    xv, dyv = (bf16_round(rng.standard_normal((T, c)).astype(np.float32)) for c in (128, 16))
    x.copy_(dev(xv)), dy.copy_(dev(dyv)), y.zero_(), dx.zero_()
    ids = make_ids(rng, T, 2)
    h = torch.empty(T, 8, device=DEV)
    moe.adapter(m, dev(ids, torch.int32), x, y, moe.AdapterBuffers.allocate(m, T), base=y, h=h)
    wy, wh, yb, _ = ref.adapter(f, ids, xv)
    check(y, wy, ref.rounded(wy, yb, False), "y")
    da = torch.empty(2, 8, 128, device=DEV)
    moe.adapter_grad(m, dev(ids, torch.int32), dy, x, h, moe.AdapterBuffers.allocate(m, T, grad=True), dx=dx, dx_base=dx, da=da)
    wx, wa, _, xb, ab, _ = ref.adapter_grad(f, ids, dyv, xv, wh)
    check(dx, wx, ref.rounded(wx, xb, False), "dx")
    check(da, wa, ab, "da")


def test_gradient_of_broadcast_tokens():
    """One token's row given to every token (equal rows): the factors' gradients are T times one's."""
    rng = np.random.default_rng(17)
    f = ref.Factors(rng, 1, 4, 128, 16)
    m = upload(f)
    T = 256
    x, dy = (np.repeat(bf16_round(rng.standard_normal((1, c)).astype(np.float32)), T, 0) for c in (128, 16))
    h = np.repeat(rng.standard_normal((1, 4)).astype(np.float32), T, 0)
    ids = np.zeros(T, np.int32)
    _, da, db = run_grad(f, m, ids, dy, x, h, None, False)
    _, wa, wb, _, ab, bb = ref.adapter_grad(f, ids, dy, x, h)
    check(da, wa, ab, "da"), check(db, wb, bb, "db")


def test_largest_sizes():
    """The longest rows and the highest rank, few tokens."""
    rng = np.random.default_rng(18)
    f = ref.Factors(rng, 2, 128, 32768, 20011)
    m = upload(f)
    ids = np.array([1, 0, 1], np.int32)
    x, dy = (bf16_round(rng.standard_normal((3, c)).astype(np.float32)) for c in (32768, 20011))
    y, h = run_forward(f, m, ids, x, None, True)
    wy, wh, yb, hb = ref.adapter(f, ids, x)
    check(h, wh, hb, "h"), check(y, wy, yb, "y")
    hv = rng.standard_normal((3, 128)).astype(np.float32)
    dx, da, db = run_grad(f, m, ids, dy, x, hv, None, False)
    wx, wa, wb, xb, ab, bb = ref.adapter_grad(f, ids, dy, x, hv)
    check(dx, wx, ref.rounded(wx, xb, False), "dx"), check(da, wa, ab, "da"), check(db, wb, bb, "db")
