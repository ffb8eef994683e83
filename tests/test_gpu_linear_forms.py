"""Every kernel form of the dense quantised products on the GPU (the sizes of
linear_forms.py, each asked which form it takes) against 64-bit products, with the
bound of a float32 sum of unrounded operands: (terms + 16) U32 of the terms'
magnitudes, as in weights_ref.py, then half a step of the result's type."""
import pytest
import torch

import linear_forms as forms
import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


class Matrix:
    """A matrix drawn on the GPU, its weights and the magnitudes of the kernels' terms in 64 bits."""

    def __init__(self, seed, N, K, bits, group, kind="plain"):
        self.gen = gen = torch.Generator(DEV).manual_seed(seed)
        q = torch.randint(0, 256, (K // 128, N, 16 * bits), dtype=torch.uint8, device=DEV, generator=gen)
        shape = (N, K // group)
        u = torch.rand(shape, device=DEV, generator=gen)
        s = 0.005 + 0.015 * u
        b = -torch.randint(0, 1 << bits, shape, device=DEV, generator=gen) * s
        if kind == "zero":
            s, b = s * (u > 0.3), b * (torch.rand(shape, device=DEV, generator=gen) > 0.3)
            s[::3], b[::3] = 0, 0
        elif kind == "large":
            s, b = torch.full_like(s, 60000), torch.full_like(s, -65504)
        elif kind == "tiny":
            s, b = torch.full_like(s, 6e-8), torch.full_like(s, -6e-8)
        elif kind == "mixed":
            s = torch.exp(-9.2 * u)                          # 1 .. 1e-4
            b = -s
        self.N, self.K = N, K
        s, b = s.half(), b.half()
        self.q = moe.QMatrix(bits, group, q, s, b)
        c = torch.stack([(q >> (bits * i)) & ((1 << bits) - 1) for i in range(8 // bits)], -1)
        c = c.permute(1, 0, 2, 3).reshape(N, K).double()
        S, B = (a.double().repeat_interleave(group, 1) for a in (s, b))
        self.W, self.mag = c * S + B, S.abs() * (c + 16) + B.abs()

    def rows(self, T, C, size=1.0):
        return size * torch.randn(T, C, device=DEV, generator=self.gen)

    def linear(self, T, f32, x=None, row_bias=False, residual=False, pad=0):
        x = (self.rows(T, self.K) if x is None else x).bfloat16()
        rb = self.rows(1, self.N)[0].contiguous() if row_bias else None
        res = self.rows(T, self.N).bfloat16() if residual else None
        dt = torch.float32 if f32 else torch.bfloat16
        y = torch.full((T, self.N + pad), 7.0, dtype=dt, device=DEV)
        moe.linear(self.q, x, y[:, :self.N], moe.LinearBuffers.allocate(self.q, T, dt), row_bias=rb, residual=res)
        assert bool((y[:, self.N:] == 7.0).all())
        want, terms = x.double() @ self.W.t(), x.double().abs() @ self.mag.t()
        for a in (rb, res):
            if a is not None:
                want, terms = want + a.double(), terms + a.double().abs()
        return self.check(y[:, :self.N], want, (self.K + 16) * ref.U32 * terms, f32)

    def grad(self, T, f32, dy=None, pad=0):
        dt = torch.float32 if f32 else torch.bfloat16
        dy = (self.rows(T, self.N + pad, 1e-3) if dy is None else dy).to(dt)[:, :self.N]
        dx = torch.full((T, self.K + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        buf = moe.LinearBuffers.allocate(self.q, T, dt, grad=True)
        buf.workspace.fill_(0xFF)
        moe.linear_grad(self.q, dy, dx[:, :self.K], buf)
        assert bool((dx[:, self.K:] == 7.0).all()) and not bool(buf.sync.any())
        terms = (self.N + 16) * ref.U32 * (dy.double().abs() @ self.mag)
        return self.check(dx[:, :self.K], dy.double() @ self.W, terms, False)

    @staticmethod
    def check(got, want, bound, f32):
        if not f32:
            bound = bound + ref.HALF_BF16 * (want.abs() + bound)
        off = (got.double() - want).abs() / (bound + 1e-37)
        worst = float(off.max())                             # (a NaN result is none)
        assert worst <= 1.0, f"{worst:.3g} times the bound"
        return got


@pytest.mark.parametrize("runs", forms.RUNS)
@pytest.mark.parametrize("bits,group", forms.FORMATS)
def test_streamed_forms(bits, group, runs):
    for i, (T, N) in enumerate(forms.TOKENS_ROWS):
        K = 128 * runs
        assert forms.kernels(T, N, K, bits, group)[0] == moe.LINEAR_STREAMED
        m = Matrix(N + runs, N, K, bits, group)
        m.linear(T, (i + runs) % 2 == 1, row_bias=i % 2 == 0, residual=i % 3 == 0, pad=i % 2)


@pytest.mark.parametrize("T,N,K,bits,group", forms.FORWARD)
def test_laid_out_tiles(T, N, K, bits, group):
    m = Matrix(T + N, N, K, bits, group)
    m.linear(T, f32=True, row_bias=True, residual=True, pad=1)
    m.linear(T, f32=False, residual=bits == 4)


@pytest.mark.parametrize("size,f32", [(s, False) for s in forms.GRAD_BF16] + [(s, True) for s in forms.GRAD_F32])
def test_laid_out_gradient_tiles(size, f32):
    T, N, K, bits, group = size
    Matrix(T + N, N, K, bits, group).grad(T, f32, pad=N % 3)


def test_tokens_in_turns():
    """More tokens than are laid out at once, the last turn a short one."""
    T, N, K, bits, group = forms.TURNS[0]
    Matrix(1, N, K, bits, group).linear(T, f32=False, row_bias=True, residual=True, pad=1)
    for (T, N, K, bits, group), f32 in ((forms.TURNS[1], False), (forms.TURNS[2], True)):
        Matrix(2, N, K, bits, group).grad(T, f32, pad=1)


def test_streamed_tokens_in_turns():
    """A long K's float32 sums of more than 1 GB: 256 tokens and 44, as two calls."""
    T, N, K = 300, 1048576, 8320
    assert forms.kernels(T, N, K, 2, 128)[0] == moe.LINEAR_STREAMED
    g = torch.Generator(DEV).manual_seed(3)
    q = torch.randint(0, 256, (K // 128, N, 32), dtype=torch.uint8, device=DEV, generator=g)
    s, b = (0.01 * torch.rand(N, K // 128, device=DEV, generator=g).half() for _ in range(2))
    w = moe.QMatrix(2, 128, q, s, b)
    x, res = torch.randn(T, K, device=DEV, generator=g).bfloat16(), torch.randn(T, N, device=DEV, generator=g).bfloat16()
    y, apart = torch.empty_like(res), torch.empty_like(res)
    buf = moe.LinearBuffers.allocate(w, T, y.dtype)
    moe.linear(w, x, y, buf, residual=res)
    for rows in (slice(0, 256), slice(256, T)):
        moe.linear(w, x[rows], apart[rows], buf, residual=res[rows])
    assert torch.equal(y, apart) and not torch.equal(y, res)


@pytest.mark.parametrize("T,N,K,bits,group", [(1, 31, 128, 4, 128), (3, 5000, 384, 4, 64), (16, 257, 1152, 2, 32),
                                              (17, 9001, 256, 4, 32), (40, 700, 2048, 2, 64), (100, 300, 128, 4, 128)])
def test_streamed_gradients(T, N, K, bits, group):
    for f32 in (False, True):
        assert forms.kernels(T, N, K, bits, group, f32, grad=True)[0] == moe.LINEAR_STREAMED
        Matrix(T + N, N, K, bits, group).grad(T, f32, pad=N % 3)


@pytest.mark.parametrize("kind", ["zero", "large", "tiny", "mixed", "rows"])
@pytest.mark.parametrize("f32", [False, True])
def test_extremes_laid_out(kind, f32):
    T, N, K, bits, group = forms.LAID_OUT
    for grad in (False, True):
        assert forms.kernels(*forms.LAID_OUT, f32, grad)[0] == moe.LINEAR_LAID_OUT
    m = Matrix(7, N, K, bits, group, kind)
    x, dy = m.rows(T, K), m.rows(T, N, 1e-3)
    if kind == "zero":
        dy[:, ::3] *= 2.0 ** 40                              # weight rows of zeros count nothing
    if kind == "rows":
        size = 2.0 ** torch.randint(-90, 90, (T, 1), device=DEV, generator=m.gen).float()
        x, dy = x * size, dy * size
        x[5], dy[6] = 0.0, 0.0
    m.linear(T, f32, x=x, residual=kind == "mixed")
    m.grad(T, f32, dy=dy)


@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("f32", [False, True])
def test_a_bad_row_laid_out(bad, f32):
    T, N, K, bits, group = forms.LAID_OUT
    m = Matrix(8, N, K, bits, group)
    x, dy = m.rows(T, K), m.rows(T, N, 1e-3)
    y0, dx0 = m.linear(T, f32, x=x), m.grad(T, f32, dy=dy)
    x[1, 70], dy[T - 1, 7] = bad, bad
    dt = torch.float32 if f32 else torch.bfloat16
    y, dx = torch.empty_like(y0), torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    moe.linear(m.q, x.bfloat16(), y, moe.LinearBuffers.allocate(m.q, T, dt))
    moe.linear_grad(m.q, dy.to(dt), dx, moe.LinearBuffers.allocate(m.q, T, dt, grad=True))
    assert not bool(torch.isfinite(y[1]).any()) and not bool(torch.isfinite(dx[T - 1]).any())
    t = torch.arange(T, device=DEV)
    assert torch.equal(y[t != 1], y0[t != 1]) and torch.equal(dx[t != T - 1], dx0[t != T - 1])


@pytest.mark.parametrize("size,f32,grad", [(forms.FORWARD[8], True, False), (forms.GRAD_F32[5], True, True),
                                           (forms.GRAD_BF16[7], False, True), (forms.LAID_OUT, True, True)])
def test_graph_replay_laid_out(size, f32, grad):
    """Split sums and two parts of dy, captured: replays with new inputs against eager calls."""
    T, N, K, bits, group = size
    m = Matrix(9, N, K, bits, group)
    dt = torch.float32 if f32 else torch.bfloat16
    a = m.rows(T, N, 1e-3).to(dt) if grad else m.rows(T, K).bfloat16()
    out = torch.empty(T, K if grad else N, dtype=torch.bfloat16 if grad else dt, device=DEV)
    buf = moe.LinearBuffers.allocate(m.q, T, dt, grad=grad)
    call = moe.linear_grad if grad else moe.linear
    call(m.q, a, out, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(m.q, a, out, buf)
    for i in range(4):
        a.copy_(m.rows(*a.shape, 1e-3))
        call(m.q, a, out, buf)
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(NAN)
        buf.workspace.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
