"""Sizes that take each form of the adapters' and the shared matrices' kernels, and the rules
by which a call takes them."""
# T, n, R, K, N, float32 y and dy
CASES = [(T, n, R, K, N, f32) for T, n, R, K, N in [
    (9, 2, 8, 256, 72), (9, 2, 24, 256, 1100),                     # one launch
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
ROUTER = [(4200, 128, 1024), (9000, 40, 4096), (2100, 1024, 2048), (5000, 8, 8192), (3000, 16, 128), (700, 130, 256), (65536, 3, 128)]


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
    chunk = max(256, min(even, 1024) if ids else even)
    return chunk, up(T, chunk)


def forward(T, n, R, K, N, f32):
    """Kernel forms of moe_adapter: (kernel, template arguments)."""
    rt, plan = rank_tiles(R), planned(T)
    if not plan and R <= 32 and R * K <= 32768:
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
