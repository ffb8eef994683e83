"""The router's losses, its backward pass and the combine's on the GPU against the
64-bit forms of weights_ref.py.

Bounds (float32 half step U = 2^-24): a logit difference of size D is off by D U, so
its exponential by a relative D U, plus a few U of its own and the sum's; ACC (64)
such roundings cover exp, division, the row's sums (at most 16 values a lane, then a
tree) and the products.  A mean over T tokens adds at most T U relative (any order).
"""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U32
ACC = 64
NAN = float("nan")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(seed, T, E, k, off=0):
    rng = np.random.default_rng(seed)
    L = (1.5 * rng.standard_normal((T, E)) - np.log(1 + np.arange(E))).astype(np.float32)
    if off:
        L[:, rng.choice(E, off, replace=False)] = -np.inf
    ids = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, L, ids


def gates_of(L, ids, renorm):
    p, _, some = ref.softmax(L)
    g = np.take_along_axis(p, np.clip(ids, 0, L.shape[1] - 1), 1)
    if renorm:
        g = g / np.maximum(g.sum(1, keepdims=True), 1e-300)
    return g.astype(np.float32)


def run_balance(L, ids, k, valid=None, buf=None, misalign=False):
    T, E = L.shape
    d = moe.dims(T, 128, 128, E, k)
    c = torch.full((E,), -7, dtype=torch.int32, device=DEV)
    P = torch.full((E,), NAN, device=DEV)
    n = torch.full((1,), -7, dtype=torch.int32, device=DEV)
    loss = torch.full((2,), NAN, device=DEV)
    if buf is None:
        buf = moe.BalanceBuffers.allocate(d)
        buf.workspace.fill_(0xFF)
    Ld = dev(L)
    if misalign:
        Ld = torch.empty(T * E + 1, device=DEV)[1:].view(T, E).copy_(Ld)
    moe.balance_loss(d, Ld, dev(ids), c, P, n, loss, buf, valid=None if valid is None else dev(valid))
    torch.cuda.synchronize()
    assert int(buf.sync.abs().sum()) == 0
    return c.cpu().numpy(), P.cpu().numpy(), int(n), loss.cpu().numpy()


def check_balance(L, ids, k, valid=None, **kw):
    c, P, n, loss = run_balance(L, ids, k, valid, **kw)
    wc, wP, wn, wb, wz = ref.balance(L, ids, k, valid)
    assert np.array_equal(c, wc) and n == wn
    rel = (ACC + 4 * ref.spread(L) + n) * U
    assert np.all(np.abs(P - wP) <= rel * wP + 1e-37), np.max(np.abs(P - wP) / (rel * wP + 1e-37))
    assert abs(loss[0] - wb) <= (rel + L.shape[1] * U) * wb + 1e-37
    # lse's absolute error: a few U of its size and of 1 (the logarithm of a sum with relative error ACC U)
    size = ref.spread(L) + np.log(L.shape[1]) + 1
    assert abs(loss[1] - wz) <= (ACC + n) * U * wz + 2 * size * ACC * U * np.sqrt(wz) + (size * ACC * U) ** 2
    return loss


SHAPES = [(1, 1, 1), (1, 4, 2), (2, 8, 8), (3, 5, 2), (7, 16, 3), (9, 17, 4), (33, 64, 2), (32, 256, 8), (20, 100, 32),
          (5, 128, 6), (64, 129, 7), (11, 300, 5), (17, 512, 4), (8, 513, 10), (40, 1000, 32), (130, 1024, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
def test_balance_shapes(T, E, k):
    rng, L, ids = make(T + E, T, E, k, off=(E - k) // 3)
    check_balance(L, ids, k)
    check_balance(L, ids, k, (rng.random(T) < 0.6).astype(np.uint8))
    check_balance(L, ids, k, misalign=True)


@pytest.mark.parametrize("T,E,k", [(8191, 128, 8), (16385, 7, 3), (5000, 64, 2), (4100, 1000, 4), (65536, 4, 1)])
def test_balance_many_tokens(T, E, k):
    rng, L, ids = make(T, T, E, k)
    valid = np.ones(T, np.uint8)
    valid[T // 3:T // 2] = 0
    first = check_balance(L, ids, k, valid)
    again = check_balance(L, ids, k, valid)
    assert np.array_equal(first, again), "equal calls give equal bits"


def test_balance_of_nothing():
    _, L, ids = make(0, 6, 9, 2)
    for valid, rows in ((np.zeros(6, np.uint8), L), (None, np.full_like(L, -np.inf)), (None, L[:0])):
        c, P, n, loss = run_balance(rows, ids[:len(rows)], 2, valid)
        assert not c.any() and not P.any() and n == 0 and not loss.any()


def test_balance_masks_and_bad_picks():
    rng, L, ids = make(1, 40, 33, 4, off=8)
    L[3] = -np.inf
    L[8, 1:] = -np.inf                                   # one expert left
    L[9] = np.finfo(np.float32).min                      # masks of the type's lowest value
    L[10, 5:] = np.finfo(np.float32).min
    ids[12] = [-1, 33, 2, 1 << 30]
    ids[13] = 4                                          # one expert four times
    valid = np.ones(40, np.uint8)
    valid[9] = 0                                         # its lse^2 alone would be past float32
    valid[20:] = 255
    check_balance(L, ids, 4, valid)
    c, P, n, loss = run_balance(L, ids, 4)
    assert n == 39 and np.isinf(loss[1])
    L[15, 2] = NAN
    c, P, n, loss = run_balance(L, ids, 4, valid)
    assert n == ref.balance(L, ids, 4, valid)[2] and np.isnan(loss).all() and np.isnan(P).all()


def run_route(L, ids, g, renorm, dg=None, dl=None, counts=None, n=0, valid=None, misalign=False):
    T, E = L.shape
    d = moe.dims(T, 128, 128, E, ids.shape[1])
    out = torch.full((T * E + 1,), NAN, device=DEV)
    out = out[1:].view(T, E) if misalign else out[:-1].view(T, E)
    moe.route_backward(d, dev(L), dev(ids), dev(g), renorm, out, None if dg is None else dev(dg),
                       None if dl is None else torch.tensor(dl, device=DEV),
                       None if counts is None else dev(counts.astype(np.int32)),
                       torch.tensor([n], dtype=torch.int32, device=DEV), None if valid is None else dev(valid))
    torch.cuda.synchronize()
    return out.cpu().numpy()


def check_route(L, ids, renorm, dg=None, dl=None, counts=None, n=0, valid=None, **kw):
    g = gates_of(L, ids, renorm)
    got = run_route(L, ids, g, renorm, dg, dl, counts, n, valid, **kw)
    want, mag = ref.route_backward(L, ids, g, renorm, dg, None if dl is None else np.float32(dl), counts, n, valid)
    bound = (ACC + 4 * ref.spread(L)) * U * mag + 1e-37
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", SHAPES + [(3000, 64, 2), (9001, 16, 7), (2100, 1024, 3)])
def test_route_backward_shapes(T, E, k, renorm):
    rng, L, ids = make(T + E + 1, T, E, k, off=(E - k) // 3)
    dg = rng.standard_normal((T, k)).astype(np.float32)
    valid = (rng.random(T) < 0.6).astype(np.uint8)
    counts, _, n, _, _ = ref.balance(L, ids, k, valid)
    check_route(L, ids, renorm, dg, (0.5, 0.02), counts, n, valid)
    check_route(L, ids, renorm, dg, misalign=True)
    check_route(L, ids, renorm, None, (0.0, 1.0), counts, n)


def test_route_backward_masks():
    rng, L, ids = make(2, 20, 24, 3, off=4)
    L[2] = -np.inf
    L[3, 1:] = -np.inf
    L[4] = np.finfo(np.float32).min
    ids[5] = [7, 7, 7]                                   # one expert three times
    ids[6] = [-1, 24, 3]
    dg = rng.standard_normal((20, 3)).astype(np.float32)
    counts, _, n, _, _ = ref.balance(L, ids, 3)
    valid = np.ones(20, np.uint8)
    valid[4] = 0
    for renorm in (True, False):
        check_route(L, ids, renorm, dg, (1.0, 0.1), counts, n, valid)
    # no tokens counted (an all-padding batch): |V| is taken as 1, padded tokens get the gates' part only
    none = np.zeros(20, np.uint8)
    check_route(L, ids, False, dg, (1.0, 0.1), np.zeros(24, np.int64), 0, none)
    assert not run_route(L, ids, gates_of(L, ids, True), True, None, (1.0, 0.1), np.zeros(24), 0, none).any()
    assert not run_route(L, ids, gates_of(L, ids, True), True).any()


def test_route_backward_by_differences():
    """Central differences of the losses' and gates' sum in 64 bits against the kernel."""
    T, E, k = 4, 12, 3
    rng, L, ids = make(3, T, E, k)
    dg = rng.standard_normal((T, k)).astype(np.float32)
    a, z = 0.8, 0.05
    counts, _, n, _, _ = ref.balance(L, ids, k)
    f = counts / (n * k)

    def loss(X, renorm):
        p, lse, _ = ref.softmax(X)
        g = np.take_along_axis(p, ids, 1)
        g = g / g.sum(1, keepdims=True) if renorm else g
        return a * E * (f * p.mean(0)).sum() + z * (lse ** 2).mean() + (g * dg).sum()

    h = 1e-4
    for renorm in (True, False):
        got = run_route(L, ids, gates_of(L, ids, renorm), renorm, dg, (a, z), counts, n)
        for t in range(T):
            for e in range(E):
                X = L.astype(np.float64)
                X[t, e] += h
                hi = loss(X, renorm)
                X[t, e] -= 2 * h
                # h^2 / 6 times the third derivative (below 10 here), and the kernel's own float32 roundings
                assert abs((hi - loss(X, renorm)) / (2 * h) - got[t, e]) < 2e-8 + ACC * U * 4


# ---------------------------------------------------------------- combine

def run_combine(seed, T, H, k, dy=True, rows=None, extra_rows=0):
    rng = np.random.default_rng(seed)
    P = T * k
    dout = ref.bf16_round(1e-3 * rng.standard_normal((T, H)).astype(np.float32))
    y = ref.bf16_round(rng.standard_normal((P + extra_rows, H)).astype(np.float32))
    p2r = rng.permutation(P).astype(np.int32) if rows is None else rows
    g = rng.random((T, k)).astype(np.float32)
    d = moe.dims(T, H, 128, 1024, k)
    b16 = lambda a: dev(a).to(torch.bfloat16)  # noqa: E731
    dg = torch.full((T, k), NAN, device=DEV)
    out = torch.full((P + extra_rows, H), 7.0, dtype=torch.bfloat16, device=DEV) if dy else None
    moe.combine_backward(d, b16(dout), b16(y), dev(p2r), dev(g), dg, out)
    torch.cuda.synchronize()
    ok = (p2r >= 0) & (p2r < P)
    r = np.where(ok, p2r, 0)
    yr = y.astype(np.float64)[r] * ok[:, None]
    dt = np.repeat(dout.astype(np.float64), k, axis=0)
    want = (yr * dt).sum(1).reshape(T, k)
    bound = H * U * (np.abs(yr) * np.abs(dt)).sum(1).reshape(T, k) + 1e-37
    assert np.all(np.abs(dg.double().cpu().numpy() - want) <= bound)
    if dy:
        got = out.double().cpu().numpy()
        ref_dy = np.full((P + extra_rows, H), 7.0)
        ref_dy[p2r[ok]] = (g.astype(np.float64).reshape(-1, 1) * dt)[ok]
        # one rounding to float32, one to bf16
        assert np.all(np.abs(got - ref_dy) <= (ref.HALF_BF16 + 2 * U) * np.abs(ref_dy) + 1e-38)


@pytest.mark.parametrize("T,H,k", [(1, 128, 1), (1, 5120, 2), (2, 256, 32), (8, 8192, 4), (37, 384, 3), (130, 2048, 8),
                                   (700, 640, 1), (513, 1152, 5), (1, 4096, 4), (300, 128, 2)])
def test_combine_backward_shapes(T, H, k):
    run_combine(T, T, H, k)
    run_combine(T + 1, T, H, k, dy=False)


def test_combine_backward_rows_out_of_range():
    T, k = 40, 4
    rows = np.random.default_rng(0).permutation(T * k).astype(np.int32)
    rows[5], rows[17], rows[99] = -1, T * k, 1 << 30
    run_combine(9, T, 256, k, rows=rows, extra_rows=3)
    T, k = 300, 4
    rows = np.random.default_rng(1).permutation(T * k).astype(np.int32)
    rows[::7] = -5
    run_combine(10, T, 256, k, rows=rows, extra_rows=300)


def test_graph_replay_and_streams():
    """All three captured together; replays against eager, with new inputs and eager work between."""
    T, E, k, H = 600, 96, 4, 512
    d = moe.dims(T, H, 128, E, k)
    s = torch.cuda.Stream()
    buf = moe.BalanceBuffers.allocate(d)
    _, L, ids = make(5, T, E, k)
    Ld, idd, g = dev(L), dev(ids), dev(gates_of(L, ids, True))
    dout, y = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(T * k, H, device=DEV).bfloat16()
    p2r = torch.randperm(T * k, device=DEV).int()
    outs = [torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV),
            torch.empty(1, dtype=torch.int32, device=DEV), torch.empty(2, device=DEV), torch.empty(T, k, device=DEV),
            torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, E, device=DEV)]
    dl = torch.tensor([0.1, 0.01], device=DEV)

    def step(stream=None):
        c, P, n, loss, dg, dy, dL = outs
        moe.balance_loss(d, Ld, idd, c, P, n, loss, buf, stream=stream)
        moe.combine_backward(d, dout, y, p2r, g, dg, dy, stream=stream)
        moe.route_backward(d, Ld, idd, g, True, dL, dg, dl, c, n, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        _, L, ids = make(50 + i, T, E, k)
        Ld.copy_(dev(L))
        idd.copy_(dev(ids))
        g.copy_(dev(gates_of(L, ids, True)))
        dout.normal_()
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {i}"
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        step(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"stream {i}"


@pytest.mark.parametrize("T,H,k", [(171, 128, 3), (700, 256, 3), (5001, 128, 5), (65536, 128, 1), (900, 384, 1)])
def test_combine_backward_short_rows(T, H, k):
    """Several pairs a wave, a partial last wave, and rows out of range among them."""
    run_combine(T, T, H, k)
    rows = np.random.default_rng(T).permutation(T * k).astype(np.int32)
    rows[::11], rows[-1] = -1, T * k
    run_combine(T + 1, T, H, k, rows=rows, extra_rows=1)
