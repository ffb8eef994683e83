"""The plain 64-bit forms of tuning_ref.py on the CPU against independent definitions:
autograd in float64, central differences, and fractions."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import tuning_ref as ref
from weights_ref import bf16_round


@pytest.mark.parametrize("ragged", [False, True])
def test_adapter_gradients(ragged):
    rng = np.random.default_rng(3)
    f = ref.Factors(rng, 3, 5, 128, 11, ragged)
    ids = np.array([2, 0, -1, 0, 7, 2, 2])
    x, dy = rng.standard_normal((7, 128)), rng.standard_normal((7, 11))
    base, dbase = rng.standard_normal((7, 11)), rng.standard_normal((7, 128))
    a, b = torch.tensor(f.a, dtype=torch.float64, requires_grad=True), torch.tensor(f.b, dtype=torch.float64, requires_grad=True)
    X = torch.tensor(x, requires_grad=True)
    rows = []
    for t, i in enumerate(ids):
        r = 0 if not 0 <= i < 3 else f.R if f.rank is None else int(f.rank[i])
        y = torch.tensor(base[t])
        if r:
            y = y + float(f.scale[i]) * ((X[t] @ a[i, :r].T) @ b[i, :r])
        rows.append(y)
    Y = torch.stack(rows)
    y, h, _, _ = ref.adapter(f, ids, x, base)
    np.testing.assert_allclose(y, Y.detach().numpy(), atol=1e-12)
    (Y * torch.tensor(dy)).sum().backward()
    dx, da, db, *_ = ref.adapter_grad(f, ids, dy, x, h, dbase)
    np.testing.assert_allclose(dx, X.grad.numpy() + dbase, atol=1e-12)
    np.testing.assert_allclose(da, a.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(db, b.grad.numpy(), atol=1e-12)


def test_adapter_gradient_by_differences():
    rng = np.random.default_rng(4)
    f = ref.Factors(rng, 2, 3, 128, 9)
    ids = np.array([1, 1, 0])
    x, dy = rng.standard_normal((3, 128)), rng.standard_normal((3, 9))
    _, h, _, _ = ref.adapter(f, ids, x)
    dx, da, db, *_ = ref.adapter_grad(f, ids, dy, x, h)
    f.a, f.b = f.a.astype(np.float64), f.b.astype(np.float64)
    for arr, grad, at in ((x, dx, (1, 7)), (f.a, da, (1, 2, 5)), (f.b, db, (0, 1, 8))):
        keep = arr[at]
        arr[at] = keep + 1e-5
        up = (ref.adapter(f, ids, x)[0] * dy).sum()
        arr[at] = keep - 1e-5
        down = (ref.adapter(f, ids, x)[0] * dy).sum()
        arr[at] = keep
        assert abs((up - down) / 2e-5 - grad[at]) < 1e-6


def test_logprobs_and_gradient():
    rng = np.random.default_rng(5)
    L = 3 * rng.standard_normal((4, 13))
    L[1, 2:5] = -np.inf
    L[3] = -np.inf
    tokens = np.array([3, 0, -1, 2])
    w, u = rng.standard_normal(4), rng.standard_normal(4)
    logp, ent, stats, ids, top = ref.logprobs(L, tokens, 12)
    T = torch.tensor(L[:3], requires_grad=True)
    lp = torch.log_softmax(T, 1)
    p = lp.exp()
    H = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    want = torch.stack((lp[0, 3], lp[1, 0], torch.zeros((), dtype=torch.float64)))
    np.testing.assert_allclose(logp[:3], want.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(ent[:3], H.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(stats[:3].sum(1), torch.logsumexp(T, 1).detach().numpy(), atol=1e-12)
    assert logp[3] == -np.inf and ent[3] == 0 and (ids[3] == -1).all() and (top[3] == -np.inf).all()
    assert (ids[1] >= 0).sum() == 10 and ids[0, 0] == int(L[0].argmax())
    d, _ = ref.logprobs_grad(L, tokens, w, u)
    assert (d[3] == 0).all() and (d[1, 2:5] == 0).all()
    # by differences
    for t, v in ((0, 3), (0, 7), (1, 0), (2, 12)):
        val = []
        for step in (1e-5, -1e-5):
            M = L.copy()
            M[t, v] += step
            lo, en, *_ = ref.logprobs(M, tokens)
            val.append(lo[t] * w[t] + en[t] * u[t])
        assert abs((val[0] - val[1]) / 2e-5 - d[t, v]) < 1e-7


def test_logprobs_order_and_ends_of_the_type():
    row = np.array([[2.0, -0.0, 5.0, 0.0, 5.0, np.nan, 2.0]])
    assert ref.logprobs(row, np.array([0]), 6)[3].tolist() == [[2, 4, 0, 6, 1, 3]]
    low = np.finfo(np.float32).min
    logp, ent, stats, *_ = ref.logprobs(np.full((1, 8), low, np.float32), np.array([3]))
    np.testing.assert_allclose([logp[0], ent[0]], [-np.log(8), np.log(8)])


def test_codes_are_the_nearest_with_ties_to_even():
    rng = np.random.default_rng(6)
    x = bf16_round(rng.standard_normal((3, 256)).astype(np.float32))
    x[0, :8] = [4.0, 2.0, -2.0, 1.0, 0.5, -0.5, 0.25, 4.0]       # 127 / 2 = 63.5: a tie
    x[1, 128:] = 0
    q, s = ref.save(x)
    assert q[0, 1] == 64 and q[0, 2] == -64
    for t in range(3):
        for g in range(2):
            v = [Fraction(float(e)) for e in x[t, 128 * g:128 * g + 128]]
            m = max(abs(e) for e in v)
            for j, e in enumerate(v):
                assert int(q[t, 128 * g + j]) == (round(127 * e / m) if m else 0)    # (Python rounds ties to even)
    assert (s[1, 1] == 0) and np.all(np.abs(ref.restored(q, s) - x) <= np.repeat(s, 128, 1) * 0.5001)


def test_kernel_arithmetic_of_the_codes():
    """The float32 steps of the kernel (a product with the rounded quotient, rounded to 18 bits, to the
    nearest whole number) give the exact quotient's rounding for every pair of 8-bit significands."""
    A = np.arange(128, 256)
    for k in range(16):
        for X in range(128, 256):
            x, a = np.float32(X * 2.0 ** -k), A.astype(np.float32)
            fits = x <= a
            q = (x * (np.float32(127) / a)).astype(np.float32)
            q = ((q.view(np.uint32) + np.uint32(0x20)) & np.uint32(0xFFFFFFC0)).view(np.float32)
            num, den = 127 * X, A.astype(np.int64) << k
            whole, rest = num // den, 2 * (num % den)
            want = whole + ((rest > den) | ((rest == den) & (whole % 2 == 1)))
            assert np.array_equal(np.rint(q)[fits], want[fits])
