"""Sizes that take each form of the dense quantised products' kernels, on a GPU of 256
compute units, and the question which form a size takes (host-only)."""
import ctypes

import quantized_expert_ffn_gemv_amd as moe

FORMATS = [(4, 128), (4, 64), (4, 32), (2, 128), (2, 64), (2, 32)]

# Streamed forward products: 128-runs of K from one to more than a launch takes, every count of waves
# and of scale pieces among them; few weight rows and many, one token tile and two.
RUNS = (1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 16, 17, 23, 32, 33, 41, 48, 49, 61, 64)
TOKENS_ROWS = ((5, 47), (3, 6007), (16, 8171), (7, 9001), (33, 4099), (17, 17011))


def stream_forms(bits, group):
    """(token tiles, weight row tiles, runs a wave, tiles ahead) of every kernel built for the format."""
    rows = (1, 2) if (bits, group) == (2, 128) else (1,)
    return {(nt, rt, g, r) for nt in (1, 2) for rt in rows for g in ((1, 2, 4, 6, 8) if nt == 1 else (1, 2, 4))
            for r in ((1, 2) if g == 1 else (1,))}


# Laid-out products: (T, N, K, bits, group) and the tile, its blocks a stage and whether the sum is split.
TILES = [(64, 64, 2), (64, 64, 4), (128, 128, 1), (256, 128, 1), (256, 256, 1)]
FORWARD = [(3000, 333, 128, 4, 128), (250, 333, 16384, 4, 32), (130, 4100, 128, 4, 32), (60, 16, 9088, 4, 32),
           (130, 30001, 128, 2, 128), (1000, 2100, 2944, 4, 32), (1500, 2100, 1920, 4, 32), (1500, 5300, 1152, 2, 64),
           (700, 2100, 9088, 4, 32), (440, 30001, 384, 4, 32), (3000, 700, 9088, 4, 32)]
GRAD_BF16 = [(440, 16, 2944, 4, 32), (1000, 2500, 384, 4, 32), (700, 333, 1152, 4, 32), (1000, 4100, 256, 4, 32),
             (1500, 16, 2944, 4, 128), (520, 2100, 4096, 4, 32), (440, 1500, 16384, 2, 128), (130, 14933, 4096, 4, 32),
             (2500, 333, 6400, 4, 128), (130, 9000, 9088, 2, 32)]
GRAD_F32 = [(520, 16, 2944, 4, 32), (440, 4100, 640, 4, 32), (1500, 333, 640, 4, 32), (440, 2100, 1152, 4, 32),
            (520, 16, 8192, 4, 32), (520, 1500, 4096, 4, 32), (440, 700, 16384, 4, 32), (130, 9000, 4096, 4, 32),
            (2500, 130, 6400, 2, 128), (130, 4100, 16384, 4, 32)]
LAID_OUT = (2500, 2500, 640, 4, 64)          # in both directions and types
# More laid-out tokens than are taken at once: forward, gradient with bf16 and with float32 dy.
TURNS = [(20000, 1200, 32768, 4, 128), (5600, 100001, 256, 4, 128), (2900, 100001, 384, 2, 32)]


def kernels(T, N, K, bits, group, f32=False, grad=False):
    w = moe.QMatrixC(None, None, None, N, K, group, bits)
    out = (ctypes.c_int32 * 8)()
    assert moe.lib().moe_linear_kernels(ctypes.byref(w), T, moe.F32 if f32 else moe.BF16, int(grad), out) == moe.OK
    return tuple(out)


def tile_of(k):
    """(rows, columns, blocks a stage, split) of a laid-out product's answer"""
    return k[1], k[2], k[4], k[3] > 1
