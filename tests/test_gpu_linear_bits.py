"""Dense quantised products whose terms cancel: what is left shows the bits that the
operands were carried with, whichever kernels the sizes take.

Only m terms of each sum differ from 0 (adding zeros rounds nothing), so the bound is
that of weights_ref.py for a sum of m terms without any rounding of the operands:
(m + 16) U32 of the terms' magnitudes, then half a step of the result's type.  The 16
hold what a weight or a float32 dy may leave out, 2^-22 or 4 U32 of a term each.
"""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"

# few tokens, many, and one token with a long K and few rows (which the estimates give to the laid-out product)
SIZES = [(3, 90, 256), (40, 90, 256), (1, 24, 32768), (1000, 2500, 640), (3000, 700, 1152)]


def pack(codes, bits):
    """Codes [N, K] in the library's layout [K/128, N, 16 bits]."""
    N, K = codes.shape
    per = 8 // bits
    c = codes.reshape(N, K // per, per).astype(np.uint32)
    row = sum(c[:, :, i] << (bits * i) for i in range(per)).astype(np.uint8)
    return np.ascontiguousarray(row.reshape(N, K // 128, 16 * bits).transpose(1, 0, 2))


class Matrix:
    def __init__(self, codes, s, b, bits, group):
        q = pack(codes, bits)
        assert np.array_equal(ref.codes(q, bits), codes)
        self.N, self.K = codes.shape
        self.W, self.mag = ref.weights(q, s, b, bits, group)
        self.q = moe.QMatrix(bits, group, *(torch.from_numpy(a).to(DEV) for a in (q, s, b)))


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def scales(rng, N, n):
    return rng.uniform(0.005, 0.02, (N, n)).astype(np.float16)


def check(got, want, terms, m, f32, what):
    bound = (m + 16) * ref.U32 * terms
    if not f32:
        bound = bound + ref.HALF_BF16 * (np.abs(want) + bound)
    worst = float(np.max(np.abs(got.double().cpu().numpy() - want) / (bound + 1e-37)))
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 64)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_forward(T, N, K, f32, bits, group):
    """a (w1 + w2 - w3 - w4), the four weights of one group with equal sums of codes: exactly 0."""
    rng = np.random.default_rng(T + bits)
    codes = rng.integers(0, 1 << bits, (N, K))
    x = np.zeros((T, K), np.float32)
    for g in range(K // group):                          # columns g G .. g G + 3 of every group
        at = g * group
        codes[:, at + 2] = rng.integers(0, 1 << bits, N)
        total = codes[:, at] + codes[:, at + 1]
        top = (1 << bits) - 1
        codes[:, at + 2] = np.clip(codes[:, at + 2], np.maximum(total - top, 0), np.minimum(total, top))
        codes[:, at + 3] = total - codes[:, at + 2]
    s = scales(rng, N, K // group)
    b = (-rng.uniform(0, 9, s.shape) * s.astype(np.float32)).astype(np.float16)
    m = Matrix(codes, s, b, bits, group)
    a = ref.bf16_round(rng.standard_normal(T).astype(np.float32))
    at = group * rng.integers(0, K // group, T)
    for i, sign in enumerate((1, 1, -1, -1)):
        x[np.arange(T), at + i] = sign * a
    y = torch.empty(T, N, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    moe.linear(m.q, dev(x, torch.bfloat16), y, moe.LinearBuffers.allocate(m.q, T, y.dtype))
    want = x.astype(np.float64) @ m.W.T
    check(y, want, np.abs(x).astype(np.float64) @ m.mag.T, 4, f32, "forward")


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 64)])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gradient_of_a_weight_that_is_zero(T, N, K, bits, group):
    """One weight row a token, its codes at the zero point where w = q s - z s = 0."""
    rng = np.random.default_rng(T + bits + 1)
    s = scales(rng, N, K // group)
    z = rng.integers(0, 3, s.shape)
    b = (-z * s.astype(np.float32)).astype(np.float16)
    codes = np.where(rng.random((N, K)) < 0.9, np.repeat(z, group, axis=1), rng.integers(0, 1 << bits, (N, K)))
    m = Matrix(codes, s, b, bits, group)
    for f32 in (False, True):
        dy = np.zeros((T, N), np.float32)
        v = 1e-3 * rng.standard_normal(T).astype(np.float32)
        dy[np.arange(T), rng.integers(0, N, T)] = v if f32 else ref.bf16_round(v)
        run_grad(m, dy, 1, f32)


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 64)])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_gradient_of_weight_rows_that_cancel(T, N, K, bits, group):
    """a (w1 + w2 - w3) of three rows with one scale, no bias and codes q3 = q1 + q2: exactly 0."""
    rng = np.random.default_rng(T + bits + 2)
    codes = rng.integers(0, 1 << (bits - 1), (N, K))
    s = scales(rng, N, K // group)
    codes[2::3] = codes[0:N // 3 * 3:3] + codes[1:N // 3 * 3:3]
    s[1::3] = s[0::3][:len(s[1::3])]
    s[2::3] = s[0::3][:len(s[2::3])]
    m = Matrix(codes, s, np.zeros_like(s), bits, group)
    for f32 in (False, True):
        dy = np.zeros((T, N), np.float32)
        a = 1e-3 * rng.standard_normal(T).astype(np.float32)
        a = a if f32 else ref.bf16_round(a)
        n = 3 * rng.integers(0, N // 3, T)
        for i, sign in enumerate((1, 1, -1)):
            dy[np.arange(T), n + i] = sign * a
        run_grad(m, dy, 3, f32)


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 32), (2, 64)])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_float32_gradients_that_cancel(T, N, K, bits, group):
    """v w - v (1 + 2^-12) w of two equal rows: a float32 dy's own low bits are all that is left."""
    rng = np.random.default_rng(T + bits + 3)
    codes = rng.integers(0, 1 << bits, (N, K))
    s = scales(rng, N, K // group)
    b = (-rng.uniform(0, 9, s.shape) * s.astype(np.float32)).astype(np.float16)
    for a in (codes, s, b):
        a[1::2] = a[0::2][:len(a[1::2])]
    m = Matrix(codes, s, b, bits, group)
    dy = np.zeros((T, N), np.float32)
    v = 1e-3 * rng.standard_normal(T).astype(np.float32)
    n = 2 * rng.integers(0, N // 2, T)
    dy[np.arange(T), n] = v
    dy[np.arange(T), n + 1] = -v * np.float32(1 + 2.0 ** -12)
    run_grad(m, dy, 2, True)


def run_grad(m, dy, terms, f32):
    T = dy.shape[0]
    dt = torch.float32 if f32 else torch.bfloat16
    dx = torch.empty(T, m.K, dtype=torch.bfloat16, device=DEV)
    moe.linear_grad(m.q, dev(dy, dt), dx, moe.LinearBuffers.allocate(m.q, T, dt, grad=True))
    want = dy.astype(np.float64) @ m.W
    check(dx, want, np.abs(dy).astype(np.float64) @ m.mag, terms, False, f"gradient, float32 dy {f32}")
