"""Sizes that take each form of the adapters' and the shared matrices' kernels, the rules by
which a call takes them, and operands few of which are not zero, whose results are therefore
known to a few steps of float32.

With `live` products of a float32 operand in a sum (its tokens, columns or ranks that are not
zero), each taken as three bf16 parts, a matrix-core sum makes 3 live additions that may cut, a
step of 2 U32 each of the terms' absolute sum; additions of zeros are exact.  Eight steps more are for
scales, the joins of waves, splits and chunks, and what precedes the sum.  A form that kept two
parts would be off by up to 2^-15 of a term."""
import math

import numpy as np

import tuning_ref as ref
from weights_ref import U32, bf16_round

# T, n, R, K, N, float32 y and dy
CASES = [(T, n, R, K, N, f32) for T, n, R, K, N in [
    (9, 2, 8, 256, 72), (9, 2, 24, 256, 1100),                     # one launch
    (30, 3, 8, 1024, 100001), (20, 3, 4, 2304, 200),               # two: wide rows, many columns
    (20, 3, 16, 2176, 300), (30, 3, 32, 2176, 136),                # two, with more than four splits
    (40, 2, 64, 640, 200), (40, 2, 96, 384, 250),
    (200, 64, 8, 512, 700), (200, 64, 24, 512, 700),               # factors' gradients by waves
    (700, 3, 8, 1152, 1300), (700, 3, 24, 1152, 1300),             # planned, with several splits
    (700, 3, 48, 640, 600), (600, 2, 128, 640, 520),
    (600, 100, 8, 384, 300), (600, 100, 40, 384, 300),             # planned, by waves
] for f32 in (False, True)] + [
    (4097, 5, 4, 128, 40, False), (9000, 3, 4, 256, 24, True),     # several rounds of the plan
    (65536, 7, 2, 128, 9, False),
    (1500, 2, 128, 1024, 3000, False), (2700, 1, 128, 1024, 3000, True),     # chunks of 512, 768 and 1024 tokens
    (4200, 1, 4, 2048, 8192, False), (4200, 3, 128, 1024, 2900, True),
]

# T, E, H of the router's weight gradient: whole calls and chunks of 256, 512 and more tokens
ROUTER = [(4200, 128, 1024), (9000, 40, 4096), (2100, 1024, 2048), (5000, 8, 8192), (3000, 16, 128), (700, 130, 256), (65536, 3, 128), (1100, 40, 384)]


# ------------------------------------------------------------ launch rules

def up(a, b):
    return (a + b - 1) // b


def rank_tiles(R):
    return 1 if R <= 16 else 2 if R <= 32 else 4 if R <= 64 else 8


def planned(T):
    return T > 512


def splits(T, n, C):
    sets = max(1, min(n, T))
    tiles = up(T, 64) + sets // 2 if planned(T) else sets
    return min(up(512, tiles), up(up(C, 128), 4), 16)


def grad_chunk(T, R, C, ids=True):
    """(tokens a chunk, chunks of a set of all tokens)"""
    if ids and not planned(T):
        return T, 1
    wgs = up(R, 16 if R <= 16 else 32) * sum(up(c, 128) for c in C)
    even = up(up(T, up(512 if R > 16 else 256, wgs)), 256) * 256
    chunk = min(max(256, even), 1024) if ids else max(256 * math.ceil(8 * math.sqrt(T) / 256), even)
    return chunk, up(T, chunk)


def forward(T, n, R, K, N, f32):
    """Kernel forms of moe_adapter: (kernel, template arguments)."""
    rt, plan = rank_tiles(R), planned(T)
    workgroups = up(min(T, min(n, T) + T // 16), 8) * up(N, 1024)          # of an XCD
    if not plan and R <= 32 and R * K <= 32768 and K < (2176 if T > n else 4096) and workgroups * (K + 512) <= 64 * 2048:
        return [("expand", rt, f32, False, True)]
    return [("shrink", rt, False, plan), ("expand", rt, f32, plan, False)]


def backward(T, n, R, K, N, f32):
    """Kernel forms of moe_adapter_grad with all of its results."""
    rt, plan = rank_tiles(R), planned(T)
    groups, blocks = up(R, 16 if R <= 16 else 32), up(K, 128) + up(N, 128)
    few = T <= 64 * n and blocks * groups * n > 512
    rtw = 1 if R <= 16 else 2
    return [("shrink", rt, f32, plan), ("expand", rt, False, plan, False),
            ("weight", rtw, "plan" if plan else "scan", 1 if few else 8 // rtw, f32)]


BUILT = ({("shrink", rt, f, p) for rt in (1, 2, 4, 8) for f in (False, True) for p in (False, True)}
         | {("expand", rt, f, p, False) for rt in (1, 2, 4, 8) for f in (False, True) for p in (False, True)}
         | {("expand", rt, f, False, True) for rt in (1, 2) for f in (False, True)}
         | {("weight", rtw, kind, wt, f) for rtw in (1, 2) for kind in ("scan", "plan") for wt in (1, 8 // rtw) for f in (False, True)})


# ------------------------------------------------------- operands and results

def cut(v, parts):
    """float32 values of which only the first `parts` bf16 parts are kept (three keep all)."""
    v = np.asarray(v, np.float32)
    out, left = np.zeros(v.shape), v.copy()
    for _ in range(parts):
        part = (left.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out += part
        left = left - part
    return out


def long_values(rng, shape):
    """Normal float32 values of which two bf16 parts leave more than 2^-16 of each."""
    return (rng.standard_normal(shape).astype(np.float32).view(np.uint32) | np.uint32(0x80FF)).view(np.float32)


class Sparse:
    """Adapters of rank 1 or 2 in a set of R; dy has one column a token that is not zero, of values
    that need all three parts (float32), or whose products with the scale and the factor do
    (bf16: the best of 64); of each adapter's tokens two at most have an x and an h that are not zero."""

    def __init__(self, T, n, R, K, N, f32):
        rng = np.random.default_rng(T + 7 * R + N)
        self.f = f = ref.Factors(rng, n, R, K, N)
        f.rank = rng.integers(1, min(R, 2) + 1, n).astype(np.int32)
        self.ids = ids = rng.integers(-1, n, T).astype(np.int32)
        self.f32, self.live = f32, np.zeros(T, bool)
        for t in ref.tokens_of(ids, n).values():
            self.live[rng.choice(t, min(2, len(t)), False)] = True
        whole = rng.standard_normal((T, K)).astype(np.float32)
        self.x_dense = bf16_round(whole)                                   # (the forward sums are checked from the h they had)
        self.x = self.x_dense * self.live[:, None]
        self.dy = np.zeros((T, N), np.float32)
        at, every = rng.integers(0, N, T), np.arange(T)
        if f32:
            self.dy[every, at] = long_values(rng, T)
        else:
            tries = bf16_round(rng.standard_normal((T, 64)).astype(np.float32))
            used = np.maximum(ids, 0)
            g = (f.scale[used] * f.b[used, 0, at].astype(np.float64))[:, None] * tries
            left = np.abs(g - cut(g, 2)) / np.abs(g)
            self.dy[every, at] = tries[every, np.argmax(left, 1)]
        self.h = long_values(rng, (T, R)) * self.live[:, None]
        # what the adapters' part nearly cancels, so that rounding to bf16 hides little of it
        self.base = bf16_round(-self.dx_part(self.g(3), 3).astype(np.float32))

    def g(self, parts):
        """The gradients of the sums h, dy as `parts` parts, exact but for their rounding to float32."""
        f, g = self.f, np.zeros((len(self.ids), self.f.R))
        dy = cut(self.dy, parts)
        for i, t in ref.tokens_of(self.ids, f.n).items():
            _, B = f.of(i)
            g[t, :len(B)] = float(f.scale[i]) * (dy[t] @ B.T)
        return g.astype(np.float32)

    def dx_part(self, g, parts):
        dx, gp = np.zeros((len(self.ids), self.f.K)), cut(g, parts)
        for i, t in ref.tokens_of(self.ids, self.f.n).items():
            A, _ = self.f.of(i)
            dx[t] = gp[t, :len(A)] @ A
        return dx

    def y(self, h, parts=3):
        """y without a base from the sums h that the GPU returned, and its bound."""
        f = self.f
        y, bound = np.zeros((len(self.ids), f.N)), np.zeros((len(self.ids), f.N))
        for i, t in ref.tokens_of(self.ids, f.n).items():
            _, B = f.of(i)
            r, s = len(B), np.float32(f.scale[i])
            hs = cut((h[t, :r].astype(np.float32) * s), parts) if parts < 3 else float(s) * h[t, :r].astype(np.float64)
            y[t] = hs @ B
            bound[t] = (3 * r + 8) * ref.SUM * (np.abs(hs) @ np.abs(B))
        return y, bound + ref.TINY

    def gradients(self, x, parts=3):
        """dx, da, db (x: the rows, or what a checkpoint of them restores) and the bounds (dx's before its rounding)."""
        f, h = self.f, cut(self.h, parts)
        g = self.g(parts)
        gp, dyp = (g.astype(np.float64), self.dy.astype(np.float64)) if parts == 3 else (cut(g, parts), cut(self.dy, parts))
        part = self.dx_part(g, parts)
        dx, dxb = self.base + part, np.zeros_like(part)
        da, db = np.zeros((f.n, f.R, f.K)), np.zeros((f.n, f.R, f.N))
        dab, dbb = np.zeros_like(da), np.zeros_like(db)
        for i, t in ref.tokens_of(self.ids, f.n).items():
            A, B = f.of(i)
            r, s, live = len(A), float(f.scale[i]), int(self.live[t].sum())
            size = np.abs(g[t, :r].astype(np.float64))
            dxb[t] = (3 + 3 * r + 8) * ref.SUM * (size @ np.abs(A))        # (3: g's own sum, one column of three parts)
            da[i, :r] = gp[t, :r].T @ x[t]
            dab[i, :r] = (3 + 3 * live + 8) * ref.SUM * (size.T @ np.abs(x[t]))
            db[i, :r] = s * (h[t, :r].T @ dyp[t])
            # six products of the parts of both for a float32 dy; what is left out is a step more of each term
            dbb[i, :r] = (6 * live + 1 + 8) * ref.SUM * s * (np.abs(h[t, :r]).T @ np.abs(dyp[t]))
        dxb += 2 * U32 * (np.abs(self.base) + np.abs(dx))
        return dx, da, db, ref.rounded(dx, dxb + ref.TINY, False), dab + ref.TINY, dbb + ref.TINY


def router_operands(T, E, H):
    """logits_grad [T, E] and x [T, H] of which four tokens are not zero, the first and the last among them, and the sums'
    bound."""
    rng = np.random.default_rng(T + E)
    live = np.zeros(T, bool)
    live[[0, T - 1, T // 2, T // 3]] = True
    x = bf16_round(rng.standard_normal((T, H)).astype(np.float32)) * live[:, None]
    return long_values(rng, (T, E)) * live[:, None], x.astype(np.float32), (3 * 4 + 8) * ref.SUM
