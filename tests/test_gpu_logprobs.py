"""Token log probabilities, entropy, alternatives and their gradient on the GPU against
the 64-bit forms of tuning_ref.py.

Bounds (U = 2^-24): d = L - max is off by U |d| (one subtraction); its exponential by a relative
2 U |d| + 2 U (two roundings of the argument, the hardware's two units), which weighed
with exp d is at most 2 U (1/e + 1) of the sum each way; the running sums of a lane take
V / 32 additions and rescalings at most, the joins 64 more.  REL counts those: the sum is
off by REL of itself, log S by REL, and the mean of d (W / S) by twice REL of the mean of |d|."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import tuning_ref as ref
from weights_ref import HALF_BF16, U32, bf16_round

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")
U = U32


def rel(V):
    return (V / 32 + 80) * U


def mean_d(L, stats):
    """sum p |d| of each row (0 where there is none)"""
    out = np.zeros(len(L))
    for t, row in enumerate(L.astype(np.float64)):
        if np.isfinite(stats[t, 1]):
            with np.errstate(over="ignore", invalid="ignore"):
                d = row - stats[t, 0]
                p = np.exp(d - stats[t, 1])
            out[t] = (p[p > 0] * np.abs(d[p > 0])).sum()
    return out


def upload(L, f32, pad=0, shift=0):
    """Rows `pad` elements wider, starting `shift` elements into the buffer; NaNs around them."""
    dt = torch.float32 if f32 else torch.bfloat16
    T, V = L.shape
    flat = torch.full((shift + T * (V + pad) + 8,), NAN, dtype=dt, device=DEV)
    v = flat[shift:].as_strided((T, V), (V + pad, 1), shift)
    v.copy_(torch.from_numpy(L))
    return v


def run(L, tokens, f32=True, n_top=0, pad=0, shift=0, entropy=True, buf=None):
    T, V = L.shape
    logits = upload(L, f32, pad, shift)
    e = lambda *s: torch.full(s, NAN, device=DEV)  # noqa: E731
    logp, stats, ent = e(T), e(T, 2), e(T) if entropy else None
    ids = torch.full((T, n_top), -7, dtype=torch.int32, device=DEV) if n_top else None
    top = e(T, n_top) if n_top else None
    if buf is None:
        buf = moe.LogprobBuffers.allocate(T, V, n_top)
        buf.workspace.fill_(0xFF)
    tok = torch.from_numpy(np.asarray(tokens, np.int32)).to(DEV)
    moe.logprobs(logits, tok, logp, stats, buf, entropy=ent, top_ids=ids, top_logp=top)
    torch.cuda.synchronize()
    assert int(buf.sync.abs().sum()) == 0
    host = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    return dict(logits=logits, tok=tok, stats_d=stats, ent_d=ent, logp=host(logp), stats=host(stats), ent=host(ent),
                ids=None if ids is None else ids.cpu().numpy(), top=host(top))


def near(got, want, bound, what):
    ok = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = ok | (np.abs(got - want) <= bound)
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:4].tolist()} {got[~ok][:4]} {want[~ok][:4]}"


def check(L, tokens, r, n_top=0):
    V = L.shape[1]
    logp, ent, stats, ids, top = ref.logprobs(L, tokens, n_top)
    R, md = rel(V), mean_d(L, stats)
    with np.errstate(invalid="ignore"):
        size = np.where(np.isfinite(logp), np.abs(logp), 0.0)
    near(r["stats"][:, 0], stats[:, 0], 0.0, "maximum")
    near(r["stats"][:, 1], stats[:, 1], R + 4 * U * np.abs(np.nan_to_num(stats[:, 1])), "log of the sum")
    near(r["logp"], logp, R + 4 * U * (size + 1), "logp")
    if r["ent"] is not None:
        near(r["ent"], ent, R + 2 * R * md + 4 * U * (1 + np.log(V)), "entropy")
    if n_top:
        assert np.array_equal(r["ids"], ids), f"alternatives of rows {np.flatnonzero((r['ids'] != ids).any(1))[:5]}"
        size = np.where(np.isfinite(top), np.abs(np.nan_to_num(top)), 0.0)
        near(r["top"], top, R + 4 * U * (size + 1), "alternatives")


def make(rng, T, V, f32, masked=False, empty=False):
    L = (rng.standard_normal((T, V)) * (1 + 3 * rng.random((T, 1)))).astype(np.float32)
    L[np.arange(T), rng.integers(0, V, T)] += (12 * rng.random(T)).astype(np.float32)
    if masked:
        L[rng.random((T, V)) < 0.3] = -np.inf
    if empty:
        L[T // 2] = -np.inf
    return L if f32 else bf16_round(L)


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (2, 9), (4, 63), (3, 257), (2, 1023), (3, 2048), (3, 2049), (1, 4096), (2, 5003), (1, 8191),
         (2, 20011), (1, 49999), (3, 50001), (600, 41), (520, 2300)]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,V", SIZES)
def test_values(T, V, f32):
    rng = np.random.default_rng(T * 7 + V)
    for n_top, masked, pad, shift in ((0, False, 0, 0), (1, True, 1, 1), (5, False, 3, 2), (20, True, 0, 5), (64, False, 8, 3)):
        L = make(rng, T, V, f32, masked, masked)
        tokens = rng.integers(-1, V, T)
        check(L, tokens, run(L, tokens, f32, n_top, pad, shift, entropy=n_top != 5), n_top)


def hard_rows(V, f32):
    rng = np.random.default_rng(V)
    low = float(np.finfo(np.float32).min) if f32 else -3.3895314e38
    rows = [
        np.full(V, 0.0), np.full(V, low), np.full(V, -np.inf), np.full(V, 3.3e38),                    # even, masked, empty, huge
        np.linspace(-20, 20, V), np.linspace(20, -20, V),                                             # ascending, descending
        np.where(np.arange(V) == V - 1, 1.0, low), np.where(np.arange(V) == 0, -1.0, -np.inf),        # one that is left
        np.where(np.arange(V) % 3 == 0, 2.0, 1.0), np.round(2 * rng.standard_normal(V)),              # thousands of ties
        np.where(np.arange(V) % 2 == 0, 0.0, -0.0), rng.standard_normal(V) * 1e-30,                   # both zeros, tiny
        np.where(np.arange(V) < V // 2, -3.3e38, 3.3e38), rng.standard_normal(V) * 60 - 200,          # differences past the type
    ]
    bad = rng.standard_normal((4, V))
    bad[0, V // 3] = np.nan
    bad[1, V - 1] = np.inf
    bad[2, 0], bad[2, V // 2] = np.nan, np.inf
    bad[3] = np.nan
    L = np.concatenate([np.stack(rows), bad]).astype(np.float32)
    with np.errstate(invalid="ignore"):
        return L if f32 else np.where(np.isnan(L), np.float32(np.nan), bf16_round(np.nan_to_num(L, nan=0.0, posinf=np.inf, neginf=-np.inf)))


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("V", [70, 2000, 2100, 9001])
def test_hard_rows(V, f32):
    L = hard_rows(V, f32)
    tokens = np.arange(len(L)) * 5 % V
    for n_top in (0, 3, 64):
        check(L, tokens, run(L, tokens, f32, n_top, shift=1), n_top)
    # few rows (several workgroups a row) and many
    check(L[:2], tokens[:2], run(L[:2], tokens[:2], f32, 64), 64)
    many = np.concatenate([L] * (1 + 600 // len(L)))
    tk = np.resize(tokens, len(many))
    r = run(many, tk, f32, 5)
    check(L, tokens, {k: (v[:len(L)] if isinstance(v, np.ndarray) else v) for k, v in r.items()}, 5)
    assert np.array_equal(r["ids"], np.resize(r["ids"][:len(L)], r["ids"].shape))


def test_tokens_out_of_range_are_not_scored():
    L = np.random.default_rng(0).standard_normal((6, 300)).astype(np.float32)
    tokens = np.array([-1, 300, 2 ** 31 - 1, -2 ** 31, 299, 0])
    r = run(L, tokens)
    check(L, tokens, r)
    assert (r["logp"][:4] == 0).all() and (r["logp"][4:] < 0).all()


def run_grad(r, w, u, g32, in_place=False, pad=0):
    T, V = r["logits"].shape
    dt = torch.float32 if g32 else torch.bfloat16
    if in_place:
        g = r["logits"]
    else:
        flat = torch.full((T, V + pad + 1), 7.0, dtype=dt, device=DEV)
        g = flat[:, 1:V + 1]
    d = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.float32)).to(DEV)  # noqa: E731
    moe.logprobs_grad(r["logits"], r["tok"], r["stats_d"], g, logp_grad=d(w), entropy=r["ent_d"] if u is not None else None, entropy_grad=d(u))
    torch.cuda.synchronize()
    if not in_place:
        assert bool((flat[:, V + 1:] == 7.0).all()) and bool((flat[:, :1] == 7.0).all()), "wrote outside"
    return g


def check_grad(L, tokens, r, w, u, got, g32):
    V = L.shape[1]
    want, mag = ref.logprobs_grad(L, tokens, w, u)
    _, ent, stats, _, _ = ref.logprobs(L, tokens)
    R, md = rel(V), mean_d(L, stats)
    with np.errstate(invalid="ignore", over="ignore"):
        lp = L.astype(np.float64) - stats[:, :1] - stats[:, 1:]
        p = np.nan_to_num(np.exp(lp))
        ad = np.where(p > 0, np.abs(lp), 0.0)
    relp = R + U * (2 * ad + 16)                                          # of p
    off = R * (2 + 2 * md)[:, None] + U * (4 * ad + 4 * ent[:, None] + 4)   # of log p + entropy
    aw = np.abs(w)[:, None] if w is not None else 0.0
    au = np.abs(u)[:, None] if u is not None else 0.0
    bound = mag * (relp + 8 * U) + au * p * off + aw * p * relp + 2e-38 * (1 + aw + 200 * au)
    if not g32:
        bound = bound + HALF_BF16 * (np.abs(want) + bound)
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    worst = np.max(np.abs(g - want) / bound)
    assert worst <= 1.0, f"{worst:.3g} times the bound at {np.unravel_index(np.argmax(np.abs(g - want) / bound), g.shape)}"


@pytest.mark.parametrize("f32,g32", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (2, 9), (4, 63), (3, 1023), (2, 8200), (2, 20011), (600, 41)])
def test_gradient(T, V, f32, g32):
    rng = np.random.default_rng(T + V)
    for masked, pad, shift in ((False, 0, 0), (True, 3, 1), (True, 6, 3)):
        L = make(rng, T, V, f32, masked, masked)
        tokens = rng.integers(-1, V, T)
        r = run(L, tokens, f32, 0, pad, shift)
        w, u = rng.standard_normal(T).astype(np.float32), rng.standard_normal(T).astype(np.float32)
        for ww, uu in ((w, u), (w, None), (None, u)):
            check_grad(L, tokens, r, ww, uu, run_grad(r, ww, uu, g32, pad=pad), g32)
        if f32 == g32:
            check_grad(L, tokens, r, w, u, run_grad(r, w, u, g32, in_place=True), g32)


def test_gradient_by_differences_of_the_forward():
    """(f(L + s e) - f(L - s e)) / 2 s with the GPU's own logp and entropy: f's float32 values are off
    by at most B = R (3 + 2 mean d) + 8 U (1 + |f|), the quotient by B / s and a third-order term."""
    rng = np.random.default_rng(3)
    V, s = 40, 2.0 ** -6
    L = (2 * rng.standard_normal((1, V))).astype(np.float32)
    tokens = np.array([7])
    w, u = np.array([1.5], np.float32), np.array([-0.75], np.float32)
    r = run(L, tokens)
    g = run_grad(r, w, u, True).double().cpu().numpy()[0]
    for v in (0, 7, 12, 39):
        f = []
        for sign in (1, -1):
            M = L.copy()
            M[0, v] += sign * s
            q = run(M, tokens)
            f.append(q["logp"][0] * 1.5 - 0.75 * q["ent"][0])
        step = (L[0, v] + np.float32(s)).astype(np.float64) - (L[0, v] - np.float32(s)).astype(np.float64)
        B = rel(V) * (3 + 2 * 10) * 2.25 + 8 * U * 20
        # third derivatives of log-softmax and entropy of p <= 1 over rows of |log p| <= 12: at most 2 and 40
        assert abs((f[0] - f[1]) / step - g[v]) <= 2 * B / step + (2 * 1.5 + 40 * 0.75) * s * s / 6


def test_rows_without_gradient_are_zeros_and_not_read():
    L = np.random.default_rng(1).standard_normal((5, 700)).astype(np.float32)
    tokens = np.array([3, 4, -1, 6, 7])
    r = run(L, tokens)
    r["logits"][1].fill_(NAN)
    r["logits"][2].fill_(NAN)
    w = np.array([1.0, 0.0, 2.0, 0.0, 1.0])
    u = np.array([0.0, 0.0, 0.0, 0.5, 0.0])
    g = run_grad(r, w, u, True)
    assert bool((g[1] == 0).all()) and bool((g[2] == 0).all()) and bool(torch.isfinite(g).all())
    rows = [0, 3, 4]
    sub = {k: v[rows] if isinstance(v, (np.ndarray, torch.Tensor)) else v for k, v in r.items()}
    check_grad(L[rows], tokens[rows], sub, w[rows], u[rows], g[rows], True)


def test_bad_rows_stay_their_own():
    L = hard_rows(2100, True)
    tokens = np.zeros(len(L), np.int64)
    r = run(L, tokens)
    w = np.ones(len(L))
    g = run_grad(r, w, 0.1 * w, True)
    bad = len(L) - 4
    assert bool(torch.isfinite(g[:bad]).all()) and bool(torch.isnan(g[bad:]).any(1).all())
    assert bool((g[2] == 0).all())                      # a row without a logit


@pytest.mark.parametrize("T,V", [(4, 6001), (700, 300)])
def test_captured_streams_and_shared_buffers(T, V):
    rng = np.random.default_rng(8)
    buf = moe.LogprobBuffers.allocate(T, V, 10)
    L = make(rng, T, V, True)
    r = run(L, rng.integers(0, V, T), True, 10, buf=buf)
    logits, tok, stats, ent = r["logits"], r["tok"], r["stats_d"], r["ent_d"]
    logp, ids, top = torch.empty(T, device=DEV), torch.empty(T, 10, dtype=torch.int32, device=DEV), torch.empty(T, 10, device=DEV)
    g, w = torch.empty(T, V, device=DEV), torch.randn(T, device=DEV)

    def step():
        moe.logprobs(logits, tok, logp, stats, buf, entropy=ent, top_ids=ids, top_logp=top)
        moe.logprobs_grad(logits, tok, stats, g, logp_grad=w, entropy=ent, entropy_grad=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (logp, stats, ent, ids, top, g)
    for k in range(4):
        logits.copy_(torch.from_numpy(make(rng, T, V, True, k % 2 == 1)))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, x) for o, x in zip(outs, want)), f"replay {k}"
        # a smaller call on the same buffers, other alternatives
        moe.logprobs(logits[:2], tok[:2], logp[:2], stats[:2], buf, top_ids=ids[:2, :3].contiguous(), top_logp=top[:2, :3].contiguous())
    assert int(buf.sync.abs().sum()) == 0


@pytest.mark.parametrize("T,V,n", [(40, 9000, 64), (300, 1500, 20), (3, 50001, 64), (700, 3001, 40)])
def test_alternatives_are_relative_to_the_same_sum(T, V, n):
    """top_logp is (logit - maximum) - log S in float32 of the very statistics that are returned, whichever
    thread wrote it, so that equal calls give equal bits."""
    rng = np.random.default_rng(33)
    L = (3 * rng.standard_normal((T, V))).astype(np.float32)
    r = run(L, rng.integers(0, V, T), True, n)
    m, log_s = r["stats"].astype(np.float32).T
    want = (np.take_along_axis(L, r["ids"], 1) - m[:, None]) - log_s[:, None]
    assert np.array_equal(r["top"].astype(np.float32), want)


def test_far_rows():
    """Rows more than 2^31 elements from the first."""
    rng = np.random.default_rng(9)
    T, V, ld = 70, 3001, (1 << 25) + 1
    L = make(rng, T, V, False)
    flat = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV)
    logits, g = flat.as_strided((T, V), (ld, 1), 1), flat.as_strided((T, V), (ld, 1), 8192)
    logits.copy_(torch.from_numpy(L))
    tokens = rng.integers(0, V, T)
    tok = torch.from_numpy(tokens.astype(np.int32)).to(DEV)
    logp, stats, ent = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV), torch.empty(T, device=DEV)
    ids, top = torch.empty(T, 4, dtype=torch.int32, device=DEV), torch.empty(T, 4, device=DEV)
    moe.logprobs(logits, tok, logp, stats, moe.LogprobBuffers.allocate(T, V, 4), entropy=ent, top_ids=ids, top_logp=top)
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    check(L, tokens, dict(logp=h(logp), stats=h(stats), ent=h(ent), ids=ids.cpu().numpy(), top=h(top)), 4)
    w = rng.standard_normal(T).astype(np.float32)
    moe.logprobs_grad(logits, tok, stats, g, logp_grad=torch.from_numpy(w).to(DEV))
    check_grad(L, tokens, None, w, None, g, False)


def test_longest_rows():
    rng = np.random.default_rng(10)
    L = make(rng, 2, 1 << 20, False)
    tokens = np.array([5, (1 << 20) - 1])
    r = run(L, tokens, False, 20)
    check(L, tokens, r, 20)
    w = np.array([1.0, -2.0])
    check_grad(L, tokens, r, w, w, run_grad(r, w, w, False), False)
