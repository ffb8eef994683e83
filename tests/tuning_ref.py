"""Plain 64-bit forms of the operators that tune and score over frozen weights
(low-rank adapters, token log probabilities, 8-bit checkpoints, the router's weight
gradient), and the error bounds their GPU results are held to.

Bounds count roundings.  U32 = 2^-24 is half a step of float32.  A matrix-core sum
of K products may cut instead of rounding, a whole step each: at most 2 K U32 times
the sum of the terms' absolute values, in any order.  Three bf16 parts hold a
float32's 24 bits.  A result of bf16 is off by half a step (2^-8) more.
"""
import numpy as np

from weights_ref import HALF_BF16, U32, bf16_round

SUM = 2 * U32
TINY = 1e-37
FLOAT32_MAX = float(np.finfo(np.float32).max)


# --------------------------------------------------------------- adapters

class Factors:
    """Random adapters: a [n, R, K], b [n, R, N] (bf16 values), scale [n], ranks [n]."""

    def __init__(self, rng, n, R, K, N, ragged=False):
        self.n, self.R, self.K, self.N = n, R, K, N
        self.a = bf16_round((rng.standard_normal((n, R, K)) / np.sqrt(K)).astype(np.float32))
        self.b = bf16_round((0.5 * rng.standard_normal((n, R, N))).astype(np.float32))
        self.scale = (0.25 + 2 * rng.random(n)).astype(np.float32)
        self.rank = rng.integers(0, R + 1, n).astype(np.int32) if ragged else None

    def of(self, i):
        """(A, B) within the adapter's rank, float64"""
        r = self.R if self.rank is None else int(min(max(self.rank[i], 0), self.R))
        return self.a[i, :r].astype(np.float64), self.b[i, :r].astype(np.float64)


def tokens_of(ids, n):
    return {i: np.flatnonzero(ids == i) for i in range(n) if np.any(ids == i)}


def adapter(f, ids, x, base=None):
    """y, h and the bounds of both (y's before its own rounding)."""
    T = len(ids)
    x = x.astype(np.float64)
    y = np.zeros((T, f.N)) if base is None else base.astype(np.float64).copy()
    h, hb, yb = np.zeros((T, f.R)), np.zeros((T, f.R)), np.zeros((T, f.N))
    for i, t in tokens_of(ids, f.n).items():
        A, B = f.of(i)
        r, s = A.shape[0], float(f.scale[i])
        h[t, :r] = x[t] @ A.T
        hb[t, :r] = (f.K + 32) * SUM * (np.abs(x[t]) @ np.abs(A).T)
        y[t] += s * (h[t, :r] @ B)
        yb[t] = s * (hb[t, :r] @ np.abs(B) + (f.R + 8) * SUM * (np.abs(h[t, :r]) @ np.abs(B)))
    if base is not None:
        yb += 2 * U32 * np.abs(base)
    yb += 2 * U32 * np.abs(y)
    return y, h, yb + TINY, hb + TINY


def rounded(y, bound, f32):
    return bound if f32 else bound + HALF_BF16 * (np.abs(y) + bound)


def adapter_grad(f, ids, dy, x, h, base=None):
    """dx, da, db and the bounds of each (dx's before its own rounding)."""
    T = len(ids)
    dy, x, h = (v.astype(np.float64) for v in (dy, x, h))
    dx = np.zeros((T, f.K)) if base is None else base.astype(np.float64).copy()
    dxb = np.zeros((T, f.K)) if base is None else 2 * U32 * np.abs(base.astype(np.float64))
    da, db = np.zeros((f.n, f.R, f.K)), np.zeros((f.n, f.R, f.N))
    dab, dbb = np.zeros_like(da), np.zeros_like(db)
    for i, t in tokens_of(ids, f.n).items():
        A, B = f.of(i)
        r, s, cnt = A.shape[0], float(f.scale[i]), len(t)
        g = dy[t] @ B.T
        gb = (f.N + 32) * SUM * (np.abs(dy[t]) @ np.abs(B).T)
        dx[t] += s * (g @ A)
        dxb[t] += s * (gb @ np.abs(A) + (f.R + 8) * SUM * (np.abs(g) @ np.abs(A)))
        da[i, :r] = s * (g.T @ x[t])
        dab[i, :r] = s * ((gb + (cnt + 48) * SUM * np.abs(g)).T @ np.abs(x[t]))
        db[i, :r] = s * (h[t, :r].T @ dy[t])
        dbb[i, :r] = s * (cnt + 48) * SUM * (np.abs(h[t, :r]).T @ np.abs(dy[t]))
    return dx, da, db, dxb + 2 * U32 * np.abs(dx) + TINY, dab + TINY, dbb + TINY


# ---------------------------------------------------- token probabilities

def logprobs(L, tokens, n_top=0):
    """logp, entropy, stats [T, 2], top ids, top logp of float values L [T, V], float64."""
    T, V = L.shape
    L = L.astype(np.float64)
    logp, ent, stats = np.zeros(T), np.zeros(T), np.zeros((T, 2))
    ids, top = np.full((T, n_top), -1, np.int64), np.full((T, n_top), -np.inf)
    for t in range(T):
        row = L[t]
        bad = np.isnan(row).any() or np.isposinf(row).any()
        m = np.max(row[~np.isnan(row)], initial=-np.inf)
        scored = 0 <= tokens[t] < V
        with np.errstate(invalid="ignore", over="ignore"):
            taken = np.flatnonzero(row > -np.inf) if n_top else np.zeros(0, np.int64)
            order = taken[np.lexsort((taken, -row[taken]))][:n_top]
            if bad:
                ls, ent[t] = np.nan, np.nan
                logp[t] = np.nan if scored else 0.0
            elif m == -np.inf:
                ls, ent[t] = -np.inf, 0.0
                logp[t] = -np.inf if scored else 0.0
            else:
                d = row - m
                e = np.exp(d)
                S = e.sum()
                ls = np.log(S)
                ent[t] = ls - (e[e > 0] * d[e > 0]).sum() / S
                logp[t] = d[tokens[t]] - ls if scored else 0.0
            stats[t] = m, ls
            for j, v in enumerate(order):
                ids[t, j], top[t, j] = v, np.nan if bad else row[v] - m - ls
    # a difference of two float32 may pass the type (-3.3e38 - 3.3e38 < -3.41e38): it is -inf there
    top[top < -FLOAT32_MAX] = -np.inf
    logp[logp < -FLOAT32_MAX] = -np.inf
    return logp, ent, stats, ids, top


def logprobs_grad(L, tokens, w=None, u=None):
    """d logits and the size of its terms, float64, rows of finite logits and -inf."""
    T, V = L.shape
    logp, ent, stats, _, _ = logprobs(L, np.full(T, -1))
    d, mag = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if stats[t, 0] == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            lp = L[t].astype(np.float64) - stats[t, 0] - stats[t, 1]
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0.0)
        if w is not None and 0 <= tokens[t] < V:
            d[t] -= w[t] * p
            mag[t] += abs(w[t]) * p
            d[t, tokens[t]] += w[t]
            mag[t, tokens[t]] = abs(w[t]) * -np.expm1(lp[tokens[t]])
        if u is not None:
            d[t] -= u[t] * p * (lp + ent[t])
            mag[t] += abs(u[t]) * p * (np.abs(lp) + ent[t])
    return d, mag


# ------------------------------------------------------------ checkpoints

def save(x):
    """codes int8 [T, K] and scales float32 [T, K/128] of bf16 values x, in whole numbers: with
    q = 127 |x| / max, the code is the nearest whole number and the even one half way."""
    T, K = x.shape
    v = x.reshape(T, K // 128, 128).astype(np.float64)
    finite = np.isfinite(v).all(2)
    v = np.where(finite[:, :, None], v, 0.0)
    top = np.abs(v).max(2)
    _, e = np.frexp(top)                              # bf16: multiples of 2^(e - 40) in reach of int64, or too small to count
    unit = np.ldexp(1.0, e - 40)[:, :, None]
    num = np.rint(np.abs(v) / unit).astype(np.int64) * 127
    den = np.maximum(np.rint(top[:, :, None] / unit), 1).astype(np.int64)
    q, r = num // den, num % den
    q = q + ((2 * r > den) | ((2 * r == den) & (q % 2 == 1)))
    codes = (np.sign(v).astype(np.int64) * q).astype(np.int8)
    scale = top.astype(np.float32) / np.float32(127)
    return codes.reshape(T, K), np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def restored(q, scale):
    return q.astype(np.float64) * np.repeat(scale.astype(np.float64), 128, axis=1)
