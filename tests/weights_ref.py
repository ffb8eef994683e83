"""Plain 64-bit forms of the operators around frozen quantised weights, and the
error bounds their GPU results are held to.

Bounds count roundings.  U32 = 2^-24 is half a step of float32, half a step of a
bf16 result is 2^-8 of it.  A float32 sum of K products in any order is off by at
most K U32 times the sum of the terms' absolute values; the code operands carry an
offset of 16 code units (32 quarter units at 2 bits), which is subtracted again, so
a term counts |x| (|s| (q + 16) + |b|) here.  Products of many tokens go through a
half-precision copy of the weights (2^-11 of each), only where the result is bf16,
and the input gradient's through one of a float32 dy too (2^-11 of each; bf16
values keep their bits).  The input gradient of few tokens splits dy s into two
bf16 parts (2^-16 of it left out).
"""
import numpy as np

U32 = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def bf16_round(a):
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)).view(np.float32)


def make_matrix(rng, N, K, bits, group, scale=(0.005, 0.02)):
    """(q [K/128, N, 16 bits] uint8, scale fp16 [N, K/G], bias fp16 [N, K/G])"""
    q = rng.integers(0, 256, (K // 128, N, 16 * bits), dtype=np.uint8)
    s = rng.uniform(*scale, (N, K // group)).astype(np.float16)
    z = rng.integers(0, 1 << bits, (N, K // group))
    b = (-z * s.astype(np.float32)).astype(np.float16)
    return q, s, b


def codes(q, bits):
    """Codes as float64 [N, K]."""
    G, N, _ = q.shape
    parts = [(q >> (bits * i)) & ((1 << bits) - 1) for i in range(8 // bits)]
    c = np.stack(parts, axis=-1).reshape(G, N, 128)
    return c.transpose(1, 0, 2).reshape(N, G * 128).astype(np.float64)


def weights(q, s, b, bits, group):
    """(W, magnitude of the kernels' terms) in float64 [N, K]."""
    c = codes(q, bits)
    S = np.repeat(s.astype(np.float64), group, axis=1)
    B = np.repeat(b.astype(np.float64), group, axis=1)
    return c * S + B, np.abs(S) * (c + 16) + np.abs(B)


def linear(x, W, row_bias=None, residual=None):
    y = x.astype(np.float64) @ W.T
    if row_bias is not None:
        y = y + row_bias.astype(np.float64)
    if residual is not None:
        y = y + residual.astype(np.float64)
    return y


def linear_bound(x, W, mag, y, f32, extra=0.0):
    """Bound on |linear() on the GPU - y|; extra: magnitude of the row bias and residual."""
    K = W.shape[1]
    ax = np.abs(x).astype(np.float64)
    bound = (K + 16) * U32 * (ax @ mag.T + extra)
    if not f32:
        half = 2.0 ** -11 * (ax @ np.abs(W).T)
        bound = bound + half
        bound = bound + HALF_BF16 * (np.abs(y) + bound)
    return bound + 1e-37


def linear_grad_bound(dy, W, mag, dx):
    N = W.shape[0]
    ad = np.abs(dy).astype(np.float64)
    halves = 1 if np.array_equal(bf16_round(dy), dy) else 2
    bound = ((N + 16) * U32 + 2.0 ** -16) * (ad @ mag) + halves * 2.0 ** -11 * (ad @ np.abs(W))
    return bound + HALF_BF16 * (np.abs(dx) + bound) + 1e-37


# ----------------------------------------------------------------- router

def softmax(L):
    """(p, lse, rows that have a logit) in float64; rows without one are 0."""
    L = L.astype(np.float64)
    m = L.max(1, keepdims=True)
    some = ~(m[:, 0] == -np.inf)
    with np.errstate(invalid="ignore", over="ignore"):
        base = np.where(some[:, None], m, 0.0)
        e = np.where(some[:, None], np.exp(L - base), 0.0)
        s = np.where(some[:, None], e.sum(1, keepdims=True), 1.0)
        return e / s, np.where(some, base[:, 0] + np.log(s[:, 0]), 0.0), some


def balance(L, ids, k, valid=None):
    """(counts, prob_mean, n_valid, balance, z)"""
    T, E = L.shape
    p, lse, some = softmax(L) if T else (np.zeros((0, E)), np.zeros(0), np.zeros(0, bool))
    take = some if valid is None else some & (valid != 0)
    n = int(take.sum())
    picked = ids[take].ravel()
    picked = picked[(picked >= 0) & (picked < E)]
    counts = np.bincount(picked, minlength=E).astype(np.int64)
    if n == 0:
        return counts, np.zeros(E), 0, 0.0, 0.0
    P = p[take].sum(0) / n
    return counts, P, n, E * float((counts / (n * k) * P).sum()), float((lse[take] ** 2).sum() / n)


def route_backward(L, ids, g, renorm, dg=None, dlosses=None, counts=None, n_valid=0, valid=None):
    """(d logits, sum of its terms' absolute values)"""
    T, E = L.shape
    k = ids.shape[1]
    p, lse, some = softmax(L)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if dlosses is not None:
        V = max(n_valid, 1)
        f = counts / (V * k)
        take = (some if valid is None else some & (valid != 0)).astype(np.float64)[:, None]
        pf = (p * f).sum(1, keepdims=True)
        a, z = float(dlosses[0]) * E / V, float(dlosses[1]) * 2 / V
        d += take * p * (a * (f - pf) + z * lse[:, None])
        # lse = m + log S: S is off by a relative ACC U, so log S by ACC U whatever its size, and the
        # sum by U (|m| + |log S|); a row whose lse is near 0 has that absolute error, so 1 joins |lse|
        mag += take * p * (abs(a) * (f + pf) + abs(z) * (np.abs(lse[:, None]) + 1))
    if dg is not None:
        g, dg = g.astype(np.float64), dg.astype(np.float64)
        inner, big = (g * dg).sum(1), np.abs(g * dg).sum(1)
        rows = np.repeat(np.arange(T), k)
        ok = ((ids >= 0) & (ids < E)).ravel()
        at = (rows[ok], ids.ravel()[ok])
        if renorm:
            np.add.at(d, at, (g * (dg - inner[:, None])).ravel()[ok])
            np.add.at(mag, at, (np.abs(g) * (np.abs(dg) + big[:, None])).ravel()[ok])
        else:
            d -= p * inner[:, None]
            mag += p * big[:, None]
            np.add.at(d, at, (g * dg).ravel()[ok])
            np.add.at(mag, at, np.abs(g * dg).ravel()[ok])
    return d, mag


def spread(L):
    """The largest finite |logit| difference and size of a row: exp's argument and the logits' own
    float32 roundings scale with it."""
    F = L[np.isfinite(L) & (np.abs(L) < 1e30)]
    return float(np.abs(F).max()) if F.size else 0.0
