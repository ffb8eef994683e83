"""Dense quantised products and their input gradient on the GPU against the
64-bit forms of weights_ref.py, with its bounds."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


class Matrix:
    def __init__(self, seed, N, K, bits=4, group=128, scale=(0.005, 0.02), parts=None):
        rng = np.random.default_rng(seed)
        q, s, b = ref.make_matrix(rng, N, K, bits, group, scale) if parts is None else parts
        self.N, self.K, self.rng = N, K, rng
        self.W, self.mag = ref.weights(q, s, b, bits, group)
        self.q = moe.QMatrix(bits, group, torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV),
                             torch.from_numpy(b).to(DEV))

    def rows(self, T, C, size=1.0):
        return ref.bf16_round(size * self.rng.standard_normal((T, C)).astype(np.float32))


def dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def wide(a, pad, dtype=torch.bfloat16):
    """a's values as the first columns of a wider buffer of NaNs."""
    buf = torch.full((a.shape[0], a.shape[1] + pad), NAN, dtype=dtype, device=DEV)
    buf[:, :a.shape[1]] = dev(a, dtype)
    return buf[:, :a.shape[1]]


def check(got, want, bound, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    worst = float(np.max(np.abs(got - want) / bound)) if want.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def run_linear(m, T, f32=False, row_bias=False, residual=False, pad=0, x=None):
    dt = torch.float32 if f32 else torch.bfloat16
    x = m.rows(T, m.K) if x is None else x
    rb = (0.5 * m.rng.standard_normal(m.N)).astype(np.float32) if row_bias else None
    res = m.rows(T, m.N) if residual else None
    ybuf = torch.full((T + 1, m.N + pad + 1), 7.0, dtype=dt, device=DEV)
    y = ybuf[:T, :m.N]
    y.fill_(NAN)
    buf = moe.LinearBuffers.allocate(m.q, T, dt)
    moe.linear(m.q, wide(x, 8 * pad), y, buf, row_bias=None if rb is None else dev(rb, torch.float32),
               residual=None if res is None else wide(res, pad))
    torch.cuda.synchronize()
    assert bool((ybuf[T:] == 7.0).all()) and bool((ybuf[:, m.N:] == 7.0).all()), "wrote outside y"
    want = ref.linear(x, m.W, rb, res)
    extra = (0 if rb is None else np.abs(rb)) + (0 if res is None else np.abs(res))
    check(y, want, ref.linear_bound(x, m.W, m.mag, want, f32, extra), f"T={T} N={m.N} K={m.K}")
    return y


def run_grad(m, T, f32=False, pad=0, dy=None):
    dt = torch.float32 if f32 else torch.bfloat16
    if dy is None:
        dy = 1e-3 * np.exp(2 * m.rng.standard_normal((T, 1))) * m.rng.standard_normal((T, m.N))
        dy = dy.astype(np.float32) if f32 else ref.bf16_round(dy.astype(np.float32))
        dy[::5] = 0.0
    dxbuf = torch.full((T + 1, m.K + 8 * pad + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    dx = dxbuf[:T, :m.K]
    dx.fill_(NAN)
    buf = moe.LinearBuffers.allocate(m.q, T, dt, grad=True)
    buf.workspace.fill_(0xFF)
    moe.linear_grad(m.q, wide(dy, pad, dt), dx, buf)
    torch.cuda.synchronize()
    assert bool((dxbuf[T:] == 7.0).all()) and bool((dxbuf[:, m.K:] == 7.0).all()), "wrote outside dx"
    assert int(buf.sync.abs().sum()) == 0
    want = dy.astype(np.float64) @ m.W
    check(dx, want, ref.linear_grad_bound(dy, m.W, m.mag, want), f"T={T} N={m.N} K={m.K}")
    return dx


SHAPES = [(1, 1, 128), (1, 2048, 2048), (2, 15, 256), (3, 16, 384), (5, 17, 128), (8, 100, 1152), (16, 333, 640),
          (17, 128, 256), (31, 65, 512), (33, 47, 2048), (48, 200, 384), (64, 129, 256), (65, 64, 128), (97, 300, 512),
          (128, 256, 256), (129, 130, 384), (200, 77, 1024), (257, 513, 640), (330, 140, 512), (400, 1, 256),
          (513, 384, 1152), (700, 90, 256)]


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 64), (4, 32), (2, 128), (2, 64), (2, 32)])
def test_linear_shapes(bits, group):
    for i, (T, N, K) in enumerate(SHAPES):
        m = Matrix(100 * i + bits + group, N, K, bits, group)
        run_linear(m, T, f32=i % 3 == 1, row_bias=i % 2 == 0, residual=i % 4 < 2, pad=i % 3)


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 64), (4, 32), (2, 128), (2, 64), (2, 32)])
def test_linear_grad_shapes(bits, group):
    for i, (T, N, K) in enumerate(SHAPES):
        m = Matrix(100 * i + bits + group + 1, N, K, bits, group)
        run_grad(m, T, f32=i % 3 == 1, pad=i % 3)


@pytest.mark.parametrize("T", [1, 4, 16, 60])
def test_linear_tall_and_wide(T):
    """Many output rows (a vocabulary) and a long K, with partial last tiles."""
    run_linear(Matrix(T, 20011, 512), T, f32=True)
    run_grad(Matrix(T + 1, 20011, 256), T)
    run_linear(Matrix(T + 2, 40, 16384, 2), T, row_bias=True)
    run_grad(Matrix(T + 3, 40, 16384, 2, 32), T, f32=True)


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 64), (4, 32), (2, 128), (2, 64), (2, 32)])
def test_linear_every_share_of_k(bits, group):
    """K from one group to more than one launch's registers hold, odd counts of groups among them."""
    for NG in (1, 3, 8, 9, 13, 16, 17, 23, 32, 33, 41, 48, 49, 55, 64, 65, 79, 96, 131):
        for T, N in ((1, 33), (16, 47)) if NG % 2 else ((19, 31), (5, 4099)):
            run_linear(Matrix(NG + T, N, 128 * NG, bits, group), T, f32=NG % 3 == 0, row_bias=True, residual=True)


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 64), (4, 32), (2, 128), (2, 64), (2, 32)])
def test_linear_grad_every_share_of_rows(bits, group):
    """Weight rows from one to many rounds of a workgroup, several workgroups a run, partial last units."""
    for N, K, T in ((1, 128, 3), (31, 256, 17), (32, 128, 33), (33, 384, 1), (255, 128, 16), (256, 256, 20), (257, 128, 15),
                    (513, 384, 49), (2000, 128, 4), (4100, 256, 31), (9001, 128, 64), (3000, 1024, 100), (700, 4096, 2)):
        run_grad(Matrix(N + T, N, K, bits, group), T, f32=N % 2 == 0, pad=T % 4)


@pytest.mark.parametrize("T", [1024, 1500])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_prompt(T, f32):
    m = Matrix(T, 1030, 1280, 4, 128)
    run_linear(m, T, f32=f32, row_bias=True, residual=True, pad=1)
    run_grad(m, T, f32=f32, pad=1)


@pytest.mark.parametrize("T", [1, 9, 64, 400])
def test_residual_in_place(T):
    m = Matrix(T, 96, 256)
    x, res = m.rows(T, m.K), m.rows(T, m.N)
    y = dev(res)
    moe.linear(m.q, dev(x), y, moe.LinearBuffers.allocate(m.q, T, y.dtype), residual=y)
    want = ref.linear(x, m.W, None, res)
    check(y, want, ref.linear_bound(x, m.W, m.mag, want, False, np.abs(res)), "in place")


@pytest.mark.parametrize("T", [3, 40, 400])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_a_bad_row_stays_in_its_row(T, bad):
    m = Matrix(T, 80, 256)
    x = m.rows(T, m.K)
    clean = run_linear(m, T, x=x).clone()
    xb = x.copy()
    xb[1, 70] = bad
    y = torch.empty_like(clean)
    moe.linear(m.q, dev(xb), y, moe.LinearBuffers.allocate(m.q, T, y.dtype))
    assert not bool(torch.isfinite(y[1]).any())
    keep = torch.arange(T, device=DEV) != 1
    assert torch.equal(y[keep], clean[keep])
    dy = m.rows(T, m.N)
    clean = run_grad(m, T, dy=dy).clone()
    db = dy.copy()
    db[1, 7] = bad
    dx = torch.empty_like(clean)
    moe.linear_grad(m.q, dev(db), dx, moe.LinearBuffers.allocate(m.q, T, dx.dtype, grad=True))
    assert not bool(torch.isfinite(dx[1]).any())
    assert torch.equal(dx[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 20, 700])
@pytest.mark.parametrize("kind", ["zero", "large", "tiny", "mixed"])
def test_extreme_scales(T, kind):
    """Zero scales, the largest and smallest fp16 scales, and both in one matrix."""
    rng = np.random.default_rng(5)
    N, K, group = 50, 512, 64
    q, s, b = ref.make_matrix(rng, N, K, 4, group)
    if kind == "zero":
        s[rng.random(s.shape) < 0.3] = 0
    elif kind == "large":
        s[:] = np.float16(60000)
        b[:] = np.float16(-65504)
    elif kind == "tiny":
        s[:] = np.float16(6e-8)
        b[:] = np.float16(-6e-8)
    else:
        s[:] = np.exp(rng.uniform(np.log(1e-4), np.log(1.0), s.shape)).astype(np.float16)
        b[:] = -s
    m = Matrix(1, N, K, 4, group, parts=(q, s, b))
    run_linear(m, T)
    run_linear(m, T, f32=True)
    run_grad(m, T)


@pytest.mark.parametrize("T", [7, 400])
def test_gradient_of_zeros_and_of_very_different_rows(T):
    m = Matrix(T, 130, 256)
    assert bool((run_grad(m, T, dy=np.zeros((T, m.N), np.float32)) == 0).all())
    dy = m.rows(T, m.N) * np.float32(2.0) ** m.rng.integers(-90, 90, (T, 1)).astype(np.float32)
    run_grad(m, T, dy=ref.bf16_round(dy))
    x = m.rows(T, m.K) * np.float32(2.0) ** m.rng.integers(-90, 90, (T, 1)).astype(np.float32)
    run_linear(m, T, x=ref.bf16_round(x))


@pytest.mark.parametrize("T", [2, 40, 700])
def test_grad_is_the_transpose_of_linear(T):
    """<dy, W x> = <dx, x>: both sides by the kernels, each within its own bound."""
    m = Matrix(T, 120, 384)
    x, dy = m.rows(T, m.K), m.rows(T, m.N)
    y = run_linear(m, T, f32=True, x=x).double().cpu().numpy()
    dx = run_grad(m, T, dy=dy).double().cpu().numpy()
    for t in range(T):
        left, right = float(y[t] @ dy[t]), float(dx[t] @ x[t])
        by = ref.linear_bound(x, m.W, m.mag, y, True)[t]
        bx = ref.linear_grad_bound(dy, m.W, m.mag, dx)[t]
        assert abs(left - right) <= float(by @ np.abs(dy[t]) + bx @ np.abs(x[t]))


@pytest.mark.parametrize("T", [1, 24, 350])
def test_other_streams_and_two_calls_at_once(T):
    a, b = Matrix(1, 500, 512), Matrix(2, 300, 1024, 2, 64)
    jobs = []
    for m in (a, b):
        x, dy = dev(m.rows(T, m.K)), dev(m.rows(T, m.N))
        y, dx = torch.empty(T, m.N, dtype=torch.float32, device=DEV), torch.empty(T, m.K, dtype=torch.bfloat16, device=DEV)
        fb, gb = moe.LinearBuffers.allocate(m.q, T, y.dtype), moe.LinearBuffers.allocate(m.q, T, dy.dtype, grad=True)
        moe.linear(m.q, x, y, fb)
        moe.linear_grad(m.q, dy, dx, gb)
        jobs.append((m, x, dy, y, dx, fb, gb, y.clone(), dx.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for m, x, dy, y, dx, *_ in jobs:
        y.fill_(NAN)
        dx.fill_(NAN)
    torch.cuda.synchronize()
    for _ in range(4):
        for m, x, dy, y, dx, fb, gb, _, _, s in jobs:
            moe.linear(m.q, x, y, fb, stream=s)
            with torch.cuda.stream(s):
                moe.linear_grad(m.q, dy, dx, gb)
    torch.cuda.synchronize()
    for m, x, dy, y, dx, fb, gb, y0, dx0, s in jobs:
        assert torch.equal(y, y0) and torch.equal(dx, dx0)


@pytest.mark.parametrize("T", [1, 12, 70, 400])
def test_graph_replay(T):
    m = Matrix(T, 700, 768)
    x, dy = dev(m.rows(T, m.K)), dev(m.rows(T, m.N))
    y, dx = torch.empty(T, m.N, dtype=torch.bfloat16, device=DEV), torch.empty(T, m.K, dtype=torch.bfloat16, device=DEV)
    fb, gb = moe.LinearBuffers.allocate(m.q, T, y.dtype), moe.LinearBuffers.allocate(m.q, T, dy.dtype, grad=True)

    def step():
        moe.linear(m.q, x, y, fb)
        moe.linear_grad(m.q, dy, dx, gb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(dev(m.rows(T, m.K)))
        dy.copy_(dev(m.rows(T, m.N)))
        step()
        torch.cuda.synchronize()
        want = (y.clone(), dx.clone())
        y.fill_(NAN)
        dx.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1]), f"replay {i}"
    # two graphs that share the buffers, one after the other
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        step()
    for g in (graph, other, graph):
        y.fill_(NAN)
        dx.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])


def test_no_tokens():
    m = Matrix(0, 64, 128)
    y, dx = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    moe.linear(m.q, torch.empty(0, 128, dtype=torch.bfloat16, device=DEV), y)
    moe.linear_grad(m.q, y, dx, moe.LinearBuffers.allocate(m.q, 0, y.dtype, grad=True))


def test_bits_as_int16_are_the_same_call():
    m = Matrix(3, 48, 256)
    x = dev(m.rows(5, m.K))
    y = torch.empty(5, m.N, dtype=torch.bfloat16, device=DEV)
    moe.linear(m.q, x, y)
    q16 = moe.QMatrix(4, 128, m.q.q, m.q.scale.view(torch.int16), m.q.bias.view(torch.int16))
    y16 = torch.empty(5, m.N, dtype=torch.int16, device=DEV)
    moe.linear(q16, x.view(torch.int16), y16)
    assert torch.equal(y16, y.view(torch.int16))


@pytest.mark.parametrize("T", [5, 40, 400])
@pytest.mark.parametrize("f32", [False, True])
def test_zero_weight_rows_do_not_weigh(T, f32):
    """Rows of zeros (the padding of a vocabulary) count nothing in dx, whatever their dy."""
    q, s, b = ref.make_matrix(np.random.default_rng(6), 90, 256, 4, 128)
    s[::2] = 0
    b[::2] = 0
    m = Matrix(2, 90, 256, 4, 128, parts=(q, s, b))
    dy = m.rows(T, m.N)
    dy[:, ::2] *= np.float32(2.0) ** 40
    run_grad(m, T, f32=f32, dy=dy)
    dy[::3, 1::2] = 0.0
    dx = run_grad(m, T, f32=f32, dy=dy)
    assert bool((dx[::3] == 0).all())


@pytest.mark.parametrize("T,N,K,bits,group", [(2, 1048576, 128, 4, 128), (3, 40, 32768, 4, 32), (400, 24, 32768, 2, 128),
                                              (65536, 24, 128, 2, 64), (1, 1, 32768, 4, 64)])
def test_largest_sizes(T, N, K, bits, group):
    m = Matrix(N + K, N, K, bits, group)
    run_linear(m, T, f32=T % 2 == 0, row_bias=True)
    run_grad(m, T, f32=T % 2 == 0)


@pytest.mark.parametrize("T,step", [(3, (1 << 30) + 8), (400, (1 << 23) + 8)])
def test_rows_far_apart(T, step):
    """Row strides that carry offsets past 32 bits."""
    m = Matrix(T, 70, 256)
    far = torch.zeros((T - 1) * step + 256, dtype=torch.bfloat16, device=DEV)

    def rows(C):
        return far.as_strided((T, C), (step, 1))

    x, dy = m.rows(T, m.K), m.rows(T, m.N)
    y, dx = run_linear(m, T, x=x), run_grad(m, T, dy=dy)
    fb, gb = (moe.LinearBuffers.allocate(m.q, T, torch.bfloat16, grad=g) for g in (False, True))
    near = torch.empty_like(y)
    rows(m.K).copy_(dev(x))
    moe.linear(m.q, rows(m.K), near, fb)
    assert torch.equal(near, y)
    moe.linear(m.q, dev(x), rows(m.N), fb)
    assert torch.equal(rows(m.N), y)
    rows(m.N).copy_(dev(dy))
    near = torch.empty_like(dx)
    moe.linear_grad(m.q, rows(m.N), near, gb)
    assert torch.equal(near, dx)
    moe.linear_grad(m.q, dev(dy), rows(m.K), gb)
    assert torch.equal(rows(m.K), dx)


@pytest.mark.parametrize("bits,group,K", [(4, 128, 512), (2, 32, 16384)])
def test_buffers_serve_fewer_tokens(bits, group, K):
    m = Matrix(K, 600, K, bits, group)
    most = 700
    fb, gb = (moe.LinearBuffers.allocate(m.q, most, torch.bfloat16, grad=g) for g in (False, True))
    for T in (most, 300, 129, 90, 17, 16, 3, 1):
        x, dy = m.rows(T, m.K), m.rows(T, m.N)
        y, dx = run_linear(m, T, x=x), run_grad(m, T, dy=dy)
        y2, dx2 = torch.empty_like(y), torch.empty_like(dx)
        moe.linear(m.q, dev(x), y2, fb)
        moe.linear_grad(m.q, dev(dy), dx2, gb)
        assert torch.equal(y, y2) and torch.equal(dx, dx2)


class LargeMatrix:
    """A matrix of weights drawn, and multiplied in 64 bits, on the GPU."""

    def __init__(self, seed, N, K, bits, group):
        gen = torch.Generator(DEV).manual_seed(seed)
        q = torch.randint(0, 256, (K // 128, N, 16 * bits), dtype=torch.uint8, device=DEV, generator=gen)
        s = (0.005 + 0.015 * torch.rand(N, K // group, device=DEV, generator=gen)).half()
        b = (-torch.randint(0, 1 << bits, (N, K // group), device=DEV, generator=gen) * s.float()).half()
        self.N, self.K, self.gen, self.q = N, K, gen, moe.QMatrix(bits, group, q, s, b)
        c = torch.stack([(q >> (bits * i)) & ((1 << bits) - 1) for i in range(8 // bits)], -1)
        c = c.permute(1, 0, 2, 3).reshape(N, K).double()
        S, B = (a.double().repeat_interleave(group, 1) for a in (s, b))
        self.W, self.mag = c * S + B, S.abs() * (c + 16) + B.abs()

    def rows(self, T, C, size=1.0):
        return (size * torch.randn(T, C, device=DEV, generator=self.gen)).bfloat16()

    def linear(self, T, f32, row_bias, residual, pad):
        """weights_ref.linear_bound, on the GPU"""
        x = self.rows(T, self.K)
        rb = torch.randn(self.N, device=DEV, generator=self.gen) if row_bias else None
        res = self.rows(T, self.N) if residual else None
        dt = torch.float32 if f32 else torch.bfloat16
        y = torch.full((T, self.N + pad), 7.0, dtype=dt, device=DEV)
        moe.linear(self.q, x, y[:, :self.N], moe.LinearBuffers.allocate(self.q, T, dt), row_bias=rb, residual=res)
        assert bool((y[:, self.N:] == 7.0).all())
        ax = x.double().abs()
        want, bound = x.double() @ self.W.t(), (self.K + 16) * ref.U32 * (ax @ self.mag.t())
        for a in (rb, res):
            if a is not None:
                want, bound = want + a.double(), bound + (self.K + 16) * ref.U32 * a.double().abs()
        if not f32:
            bound = bound + 2.0 ** -11 * (ax @ self.W.abs().t())
            bound = bound + ref.HALF_BF16 * (want.abs() + bound)
        worst = float(((y[:, :self.N].double() - want).abs() / (bound + 1e-37)).max())
        assert worst <= 1.0, f"{worst:.3g} times the bound"

    def grad(self, T, f32, pad):
        """weights_ref.linear_grad_bound, on the GPU"""
        dt = torch.float32 if f32 else torch.bfloat16
        dy = self.rows(T, self.N + pad, 1e-3).to(dt)[:, :self.N]
        if f32:
            dy = dy * 1.001
        dx = torch.full((T, self.K + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        moe.linear_grad(self.q, dy, dx[:, :self.K], moe.LinearBuffers.allocate(self.q, T, dt, grad=True))
        assert bool((dx[:, self.K:] == 7.0).all())
        ad = dy.double().abs()
        want = dy.double() @ self.W
        bound = ((self.N + 16) * ref.U32 + 2.0 ** -16) * (ad @ self.mag) + (2 if f32 else 1) * 2.0 ** -11 * (ad @ self.W.abs())
        bound = bound + ref.HALF_BF16 * (want.abs() + bound) + 1e-37
        worst = float(((dx[:, :self.K].double() - want).abs() / bound).max())
        assert worst <= 1.0, f"{worst:.3g} times the bound"


@pytest.mark.parametrize("T,N,K,bits,group", [(4100, 4300, 128, 4, 128), (4000, 2100, 640, 4, 64), (1030, 4001, 384, 2, 32),
                                              (2100, 9000, 256, 4, 128), (600, 1000, 4096, 4, 32), (3000, 4096, 1152, 2, 128)])
def test_every_tile(T, N, K, bits, group):
    m = LargeMatrix(T, N, K, bits, group)
    m.linear(T, f32=False, row_bias=True, residual=True, pad=3)
    m.linear(T, f32=True, row_bias=bits == 4, residual=False, pad=0)
    m.grad(T, f32=bits == 4, pad=5)


@pytest.mark.parametrize("T,N,K,bits,group", [(4000, 16, 512, 4, 128), (3001, 130, 8192, 4, 64), (2500, 40, 16384, 2, 32),
                                              (4000, 417, 128, 4, 32), (1000, 30001, 256, 4, 128), (5000, 1, 256, 2, 128)])
def test_many_tokens_and_a_narrow_matrix(T, N, K, bits, group):
    m = LargeMatrix(T + N, N, K, bits, group)
    m.linear(T, f32=False, row_bias=False, residual=True, pad=1)
    m.grad(T, f32=False, pad=N % 2)


def test_a_matrix_in_chunks():
    """Laid-out weights past one chunk's bytes, forward and gradient."""
    LargeMatrix(1, 5000, 32768, 4, 128).linear(1500, f32=True, row_bias=True, residual=True, pad=0)
    LargeMatrix(2, 40000, 8192, 2, 64).linear(600, f32=False, row_bias=True, residual=False, pad=1)
    LargeMatrix(3, 300001, 1024, 4, 128).grad(1000, f32=False, pad=1)


@pytest.mark.parametrize("T,N,K,bits,group", [(700, 60, 8192, 4, 64), (500, 20001, 384, 2, 128), (260, 24471, 1152, 4, 128),
                                              (1100, 70, 4224, 4, 32), (1000, 900, 6400, 2, 128), (2100, 333, 9088, 4, 128)])
def test_long_sums_over_few_tiles(T, N, K, bits, group):
    """Sums split over workgroups, forward (two planes of the weights among them) and gradient."""
    m = LargeMatrix(T + K, N, K, bits, group)
    m.linear(T, f32=True, row_bias=True, residual=True, pad=1)
    m.linear(T, f32=False, row_bias=False, residual=bits == 4, pad=0)
    m.grad(T, f32=bits == 2, pad=N % 3)


@pytest.mark.parametrize("T,N,K", [(2000, 1500, 768), (260, 24471, 1152), (300, 4100, 9088)])
def test_graph_replay_and_streams_of_many_tokens(T, N, K):
    """The laid-out products, and split ones, captured; replays and another stream's calls against eager."""
    m = LargeMatrix(T, N, K, 4, 64)
    x, dy = m.rows(T, K), m.rows(T, N, 1e-3)
    y, dx = torch.empty(T, N, dtype=torch.bfloat16, device=DEV), torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    fb, gb = moe.LinearBuffers.allocate(m.q, T, y.dtype), moe.LinearBuffers.allocate(m.q, T, dy.dtype, grad=True)
    side = torch.cuda.Stream()

    def step(stream=None):
        moe.linear(m.q, x, y, fb, stream=stream)
        moe.linear_grad(m.q, dy, dx, gb, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(m.rows(T, K))
        dy.copy_(m.rows(T, N, 1e-3))
        step()
        torch.cuda.synchronize()
        want = (y.clone(), dx.clone())
        for again in (graph.replay, lambda: step(side)):
            y.fill_(NAN)
            dx.fill_(NAN)
            fb.workspace.fill_(0xFF)
            gb.workspace.fill_(0xFF)
            torch.cuda.synchronize()
            again()
            torch.cuda.synchronize()
            assert torch.equal(y, want[0]) and torch.equal(dx, want[1]), f"time {i}"


def laid_out(seed=1, parts=None):
    """A matrix and a token count whose products go through the laid-out copies."""
    T, N, K = 1000, 2500, 640
    m = Matrix(seed, N, K, 4, 64, parts=parts)
    assert moe.linear_workspace_bytes(m.q, T, torch.bfloat16) >= T * K * 2
    assert moe.linear_workspace_bytes(m.q, T, torch.bfloat16, grad=True) >= T * N * 2
    return m, T


@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_a_bad_row_of_many(bad):
    m, T = laid_out()
    x, dy = m.rows(T, m.K), m.rows(T, m.N)
    y0, dx0 = run_linear(m, T, x=x), run_grad(m, T, dy=dy)
    x[1, 70], dy[T - 1, 7] = bad, bad
    y, dx = torch.empty_like(y0), torch.empty_like(dx0)
    moe.linear(m.q, dev(x), y, moe.LinearBuffers.allocate(m.q, T, y.dtype))
    moe.linear_grad(m.q, dev(dy), dx, moe.LinearBuffers.allocate(m.q, T, dx.dtype, grad=True))
    assert not bool(torch.isfinite(y[1]).any()) and not bool(torch.isfinite(dx[T - 1]).any())
    keep = torch.arange(T, device=DEV)
    assert torch.equal(y[keep != 1], y0[keep != 1]) and torch.equal(dx[keep != T - 1], dx0[keep != T - 1])


@pytest.mark.parametrize("kind", ["zero", "large", "tiny", "mixed", "rows"])
def test_extremes_of_many_tokens(kind):
    rng = np.random.default_rng(7)
    q, s, b = ref.make_matrix(rng, 2500, 640, 4, 64)
    if kind == "zero":
        s[rng.random(s.shape) < 0.3] = 0
        b[rng.random(b.shape) < 0.3] = 0
        s[::3], b[::3] = 0, 0
    elif kind == "large":
        s[:] = np.float16(60000)
        b[:] = np.float16(-65504)
    elif kind == "tiny":
        s[:] = np.float16(6e-8)
        b[:] = np.float16(-6e-8)
    elif kind == "mixed":
        s[:] = np.exp(rng.uniform(np.log(1e-4), np.log(1.0), s.shape)).astype(np.float16)
        b[:] = -s
    m, T = laid_out(parts=(q, s, b))
    x, dy = m.rows(T, m.K), m.rows(T, m.N)
    if kind == "zero":
        dy[:, ::3] *= np.float32(2.0) ** 40
    if kind == "rows":
        x, dy = (ref.bf16_round(a * np.float32(2.0) ** rng.integers(-90, 90, (T, 1)).astype(np.float32)) for a in (x, dy))
        dy[5], x[6] = 0.0, 0.0
    run_linear(m, T, x=x)
    run_linear(m, T, f32=True, x=x)
    run_grad(m, T, dy=dy)
    run_grad(m, T, f32=True, pad=1, dy=dy)


@pytest.mark.parametrize("T,N,K", [(1000, 2500, 640), (260, 24471, 1152), (700, 60, 8192), (300, 4100, 9088)])
def test_residual_in_place_of_many_tokens(T, N, K):
    m = LargeMatrix(N, N, K, 4, 128)
    x, res = m.rows(T, K), m.rows(T, N)
    rb = torch.randn(N, device=DEV, generator=m.gen)
    buf = moe.LinearBuffers.allocate(m.q, T, torch.bfloat16)
    apart, y = torch.empty_like(res), res.clone()
    moe.linear(m.q, x, apart, buf, row_bias=rb, residual=res)
    moe.linear(m.q, x, y, buf, row_bias=rb, residual=y)
    assert torch.equal(y, apart) and not torch.equal(y, res)
