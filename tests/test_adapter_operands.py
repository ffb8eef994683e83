"""Where the adapters' operands may lie: column slices of wider buffers are taken, results
over memory that the call still reads are refused before anything is written."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import tuning_ref as ref
from weights_ref import bf16_round

BF = torch.bfloat16


@pytest.mark.parametrize("first,N,cols", [(8, 64, 72), (8, 59, 72), (16, 40, 72), (64, 8, 72), (8, 67, 80)])
def test_factor_rows_in_the_middle_of_a_buffer(first, N, cols):
    """b as columns first .. first + N - 1 of a wider buffer, up to its end."""
    a, wide, s = torch.zeros(3, 4, 256, dtype=BF), torch.zeros(3, 4, cols, dtype=BF), torch.zeros(3)
    b = wide[:, :, first:first + N]
    m = moe.Adapters(a, b, s)
    assert (m.N, m._c.ldb, m._c.b) == (N, cols, wide.data_ptr() + 2 * first)


def test_one_row_needs_no_stride():
    b = torch.zeros(1, 1, 67, dtype=BF)
    assert moe.Adapters(torch.zeros(1, 1, 128, dtype=BF), b, torch.zeros(1))._c.ldb == 72


def test_rows_between_16_byte_borders_are_refused():
    wide = torch.zeros(3, 4, 72, dtype=BF)
    with pytest.raises(ValueError, match="16-byte"):
        moe.Adapters(torch.zeros(3, 4, 256, dtype=BF), wide[:, :, 12:], torch.zeros(3))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("R,K", [(8, 256), (40, 1024)])
def test_results_from_the_middle_of_a_buffer(T, R, K):
    """The last columns of a buffer of NaNs, whose last row ends with it: the bits of a copy's results."""
    rng = np.random.default_rng(T + R)
    n, N, first = 3, 131, 24
    f = ref.Factors(rng, n, R, K, N)
    wide = torch.full((n, R, first + 136), float("nan"), dtype=BF, device="cuda")
    wide[:, :, first:first + N] = torch.from_numpy(f.b).to("cuda", BF)
    a, s = torch.from_numpy(f.a).to("cuda", BF), torch.from_numpy(f.scale).cuda()
    packed = torch.zeros(n, R, 136, dtype=BF, device="cuda")
    packed[:, :, :N] = wide[:, :, first:first + N]
    ids = torch.from_numpy(rng.integers(-1, n, T).astype(np.int32)).cuda()
    x, dy = (torch.from_numpy(bf16_round(rng.standard_normal((T, c)).astype(np.float32))).to("cuda", BF) for c in (K, N))
    got = []
    for b in (wide[:, :, first:first + N], packed[:, :, :N]):
        m = moe.Adapters(a, b, s)
        y, h, dx = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, R, device="cuda"), torch.empty(T, K, dtype=BF, device="cuda")
        da, db = torch.empty(n, R, K, device="cuda"), torch.empty(n, R, N, device="cuda")
        moe.adapter(m, ids, x, y, moe.AdapterBuffers.allocate(m, T), h=h)
        moe.adapter_grad(m, ids, dy, x, h, moe.AdapterBuffers.allocate(m, T, grad=True), dx=dx, da=da, db=db)
        got.append((y, h, dx, da, db))
    assert all(torch.equal(p, q) for p, q in zip(*got)) and all(bool(torch.isfinite(p).all()) for p in got[0])
    wy, wh, yb, _ = ref.adapter(f, ids.cpu().numpy(), x.float().cpu().numpy())
    assert np.all(np.abs(got[0][0].double().cpu().numpy() - wy) <= ref.rounded(wy, yb, False))


# ---------------------------------------------------------------- overlaps

A, FAR = 0x10000000, 0x7000000000


def _grad(dx, saved=None, x=None, h=FAR, da=FAR + (1 << 30), db=FAR + (1 << 31), T=4, lddx=256):
    m = moe.AdaptersC(FAR, FAR, 64, FAR, None, 4, 16, 256, 64)
    return moe.lib().moe_adapter_grad(ctypes.byref(m), T, FAR, FAR, 64, moe.BF16, x, 256, None if saved is None else ctypes.byref(saved), h,
                                      None, 0, dx, lddx, da, db, 0x100, 1 << 42, None)


@pytest.mark.parametrize("kw", [
    # 4 rows of 256 columns: dx 2048 bytes (512 apart: 2 (3 512 + 256) = 3584), the checkpoint 1024 of codes and 32 of scales, h 256
    dict(dx=A, saved=moe.CheckpointC(A, FAR, 4, 256)), dict(dx=A, saved=moe.CheckpointC(A + 2032, FAR, 4, 256)),
    dict(dx=A + 1022, saved=moe.CheckpointC(A, FAR, 4, 256)), dict(dx=A, saved=moe.CheckpointC(FAR, A + 2044, 4, 256)),
    dict(dx=A + 30, saved=moe.CheckpointC(FAR, A, 4, 256)), dict(dx=A, saved=moe.CheckpointC(A + 3568, FAR, 4, 256), lddx=512),
    dict(dx=A, x=FAR, h=A + 2044), dict(dx=A + 254, x=FAR, h=A), dict(dx=A, da=None, h=A),
])
def test_dx_over_what_the_factors_gradients_read_is_refused(kw):
    assert _grad(**kw) == moe.ERR_INVALID_ARG
    assert "dx overlaps" in moe.last_error()


def _projection(N=64, K=256):
    return moe.QMatrix(4, 128, torch.zeros(K // 128, N, 64, dtype=torch.uint8), *(torch.zeros(N, K // 128, dtype=torch.float16) for _ in range(2)))


def test_adapted_backward_refuses_before_it_writes(monkeypatch):
    """dx over what adapter_grad() would read: refused before linear_grad() has written it."""
    from quantized_expert_ffn_gemv_amd import layer

    called = []
    monkeypatch.setattr(layer, "linear_grad", lambda *a, **k: called.append("linear_grad"))
    monkeypatch.setattr(layer, "adapter_grad", lambda *a, **k: called.append("adapter_grad"))
    w, n, R, T, K, N = _projection(), 3, 4, 5, 256, 64
    m = moe.Adapters(torch.zeros(n, R, K, dtype=BF), torch.zeros(n, R, N, dtype=BF), torch.zeros(n))
    buf = layer.AdaptedBuffers(None, None, None, moe.AdapterBuffers.allocate(m, T, grad=True))
    ids, dy, h = torch.zeros(T, dtype=torch.int32), torch.zeros(T, N, dtype=BF), torch.zeros(T, R)
    da, db = torch.zeros(n, R, K), torch.zeros(n, R, N)
    x, wide = torch.zeros(T, K, dtype=BF), torch.zeros(T, 2 * K, dtype=BF)
    kept = moe.Checkpoint.allocate(2 * T, K, device="cpu")
    over_codes = kept.q.view(-1).view(BF)[:T * K].view(T, K)
    five = moe.Checkpoint(kept.q[:T], kept.scale[:T])
    over_h = torch.zeros(T * K, dtype=BF)
    for kw in (dict(dx=x, x=x, da=da), dict(dx=wide[:, 8:K + 8], x=wide[:, :K], da=da), dict(dx=over_codes, x=five, da=da),
               dict(dx=over_h.view(T, K), x=x, h=over_h.view(torch.float32)[:T * R].view(T, R), db=db)):
        args = dict(dict(h=h, da=None, db=None), **kw)
        with pytest.raises(ValueError, match="dx overlaps"):
            moe.adapted_linear_backward(w, m, ids, dy, args["x"], args["h"], buf, dx=args["dx"], da=args["da"], db=args["db"])
    assert not called
    # x is not read without da, and column slices of one buffer share nothing
    moe.adapted_linear_backward(w, m, ids, dy, x, h, buf, dx=x, db=db)
    moe.adapted_linear_backward(w, m, ids, dy, wide[:, :K], h, buf, dx=wide[:, K:], da=da, db=db)
    assert called == ["linear_grad", "adapter_grad"] * 2


def test_adapted_linear_refuses_before_it_writes(monkeypatch):
    """A residual in place is lost once linear() has run: what adapter() refuses is refused before."""
    from quantized_expert_ffn_gemv_amd import layer

    called = []
    monkeypatch.setattr(layer, "linear", lambda *a, **k: called.append("linear"))
    w, n, R, T, K, N = _projection(), 3, 4, 5, 256, 64
    m = moe.Adapters(torch.zeros(n, R, K, dtype=BF), torch.zeros(n, R, N, dtype=BF), torch.zeros(n))
    buf = layer.AdaptedBuffers(None, moe.AdapterBuffers.allocate(m, T))
    ids, x, y, h = torch.zeros(T, dtype=torch.int32), torch.zeros(T, K, dtype=BF), torch.zeros(T, N, dtype=BF), torch.zeros(T, R)
    small = layer.AdaptedBuffers(None, moe.AdapterBuffers(torch.zeros(256, dtype=torch.uint8)))
    for kw, word in ((dict(ids=ids.long()), "ids holds"), (dict(ids=ids[:4]), "ids has shape"), (dict(h=h[:4]), "h has shape"),
                     (dict(x=x.float()), "x holds"), (dict(y=y.half()), "y holds"), (dict(buf=small), "workspace")):
        a = dict(dict(ids=ids, x=x, y=y, h=h, buf=buf), **kw)
        with pytest.raises(ValueError, match=word):
            moe.adapted_linear(w, m, a["ids"], a["x"], a["y"], a["buf"], residual=a["y"], h=a["h"])
    assert not called
