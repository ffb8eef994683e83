"""Host-side refusals of the operators around frozen quantised weights: nothing
is launched, every call below fails (or is a no-op) on the host."""
import ctypes

import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe

FAKE = 0x10000000
MISALIGNED = FAKE + 1


def _w(N=64, K=256, group=128, bits=4, q=FAKE, scale=FAKE, bias=FAKE):
    return moe.QMatrixC(q, scale, bias, N, K, group, bits)


def _ws(w, T=4, t=moe.BF16, grad=0):
    out = ctypes.c_size_t(0)
    return moe.lib().moe_linear_workspace_bytes(ctypes.byref(w), T, t, grad, ctypes.byref(out)), out.value


@pytest.mark.parametrize("kw,T,t,status", [
    (dict(N=0), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(N=1 << 21), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(K=0), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(K=200), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(K=65536), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(bits=3), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(bits=8), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(group=96), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(group=256), 4, 0, moe.ERR_UNSUPPORTED),
    (dict(), -1, 0, moe.ERR_INVALID_ARG),
    (dict(), 65537, 0, moe.ERR_UNSUPPORTED),
    (dict(), 4, 2, moe.ERR_UNSUPPORTED),
])
def test_matrix_limits(kw, T, t, status):
    for grad in (0, 1):
        assert _ws(_w(**kw), T, t, grad)[0] == status
        assert moe.last_error()


def test_workspace_sizes():
    for grad in (0, 1):
        assert _ws(_w(), 0, 0, grad) == (moe.OK, 0)
        for T in (1, 64, 4096, 65536):
            st, n = _ws(_w(N=4099, K=2048), T, moe.F32, grad)
            assert st == moe.OK and 0 <= n < 1 << 32
    L = moe.lib()
    assert L.moe_linear_workspace_bytes(ctypes.byref(_w()), 1, 0, 0, None) == moe.ERR_INVALID_ARG
    assert L.moe_linear_workspace_bytes(None, 1, 0, 0, ctypes.byref(ctypes.c_size_t(0))) == moe.ERR_INVALID_ARG


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("kw", [dict(), dict(N=4099, K=16384), dict(N=20000, K=1024, group=32), dict(N=5000, K=8320, bits=2)])
def test_workspace_serves_fewer_tokens(kw, grad):
    for t in (moe.BF16, moe.F32):
        sizes = [_ws(_w(**kw), T, t, grad)[1] for T in range(1, 800)] + [_ws(_w(**kw), T, t, grad)[1] for T in (4096, 65536)]
        assert sizes == sorted(sizes)


def _linear(w=None, T=4, x=FAKE, ldx=256, rb=None, res=None, ldr=64, y=FAKE, ldy=64, t=moe.BF16, ws=FAKE, n=1 << 40):
    return moe.lib().moe_linear(ctypes.byref(w or _w()), T, x, ldx, rb, res, ldr, y, ldy, t, ws, n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(x=None), "x is NULL"),
    (dict(x=FAKE + 8), "x is not 16-byte"),
    (dict(ldx=248), "ldx"),
    (dict(ldx=260), "ldx"),
    (dict(y=None), "y is NULL"),
    (dict(y=MISALIGNED), "y is not"),
    (dict(y=FAKE + 2, t=moe.F32), "y is not 4-byte"),
    (dict(ldy=63), "ldy"),
    (dict(rb=FAKE + 2), "row_bias"),
    (dict(res=MISALIGNED), "residual"),
    (dict(res=FAKE, ldr=60), "ldr"),
    (dict(res=FAKE, y=FAKE, ldy=128), "residual"),
    (dict(res=FAKE, y=FAKE, t=moe.F32), "residual"),
    (dict(w=_w(q=None)), "q is NULL"),
    (dict(w=_w(scale=FAKE + 2)), "scale is not"),
    (dict(w=_w(bias=None)), "bias is NULL"),
])
def test_linear_refusals(kw, word):
    assert _linear(**kw) == moe.ERR_INVALID_ARG
    assert word in moe.last_error()


def _grad(w=None, T=4, dy=FAKE, lddy=64, t=moe.BF16, dx=FAKE, lddx=256, ws=FAKE, n=1 << 40, sync=FAKE):
    return moe.lib().moe_linear_grad(ctypes.byref(w or _w()), T, dy, lddy, t, dx, lddx, ws, n, sync, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dy=None), "dy is NULL"),
    (dict(dy=MISALIGNED), "dy is not"),
    (dict(dy=FAKE + 2, t=moe.F32), "dy is not"),
    (dict(lddy=63), "lddy"),
    (dict(dx=None), "dx is NULL"),
    (dict(dx=FAKE + 4), "dx is not"),
    (dict(lddx=128), "lddx"),
    (dict(lddx=257), "lddx"),
    (dict(sync=None), "sync is NULL"),
    (dict(sync=FAKE + 64), "sync is not"),
])
def test_linear_grad_refusals(kw, word):
    assert _grad(**kw) == moe.ERR_INVALID_ARG
    assert word in moe.last_error()


def test_workspace_refusals():
    """Where a workspace is needed, a missing, short or misaligned one is refused."""
    for grad in (0, 1):
        w = _w(N=4096, K=2048)
        st, need = _ws(w, 4096, moe.BF16, grad)
        assert st == moe.OK
        if need == 0:
            continue
        call = lambda ws, n: _grad(w, 4096, lddy=4096, lddx=2048, ws=ws, n=n) if grad else \
            _linear(w, 4096, ldx=2048, ldy=4096, ws=ws, n=n)
        assert call(None, need) == moe.ERR_WORKSPACE
        assert call(FAKE, need - 1) == moe.ERR_WORKSPACE
        assert "workspace" in moe.last_error()
        assert call(FAKE + 128, need) == moe.ERR_INVALID_ARG


def test_zero_tokens_are_no_ops():
    L = moe.lib()
    w = _w(q=None, scale=None, bias=None)
    assert L.moe_linear(ctypes.byref(w), 0, None, 0, None, None, 0, None, 0, 0, None, 0, None) == moe.OK
    assert L.moe_linear_grad(ctypes.byref(w), 0, None, 0, 0, None, 0, None, 0, None, None) == moe.OK
    d = moe.dims(0, 256, 512, 8, 2)
    assert L.moe_route_backward(ctypes.byref(d), *[None] * 3, 1, *[None] * 7) == moe.OK
    assert L.moe_combine_backward(ctypes.byref(d), *[None] * 7) == moe.OK


def test_balance_refusals():
    L = moe.lib()
    d = moe.dims(4, 256, 512, 8, 2)
    need = moe.balance_workspace_bytes(d)
    assert need > 0
    base = dict(logits=FAKE, ids=FAKE, valid=None, counts=FAKE, prob=FAKE, n=FAKE, losses=FAKE, ws=FAKE, nbytes=need,
                sync=FAKE)

    def call(**kw):
        a = dict(base, **kw)
        return L.moe_balance_loss(ctypes.byref(d), a["logits"], a["ids"], a["valid"], a["counts"], a["prob"], a["n"],
                                  a["losses"], a["ws"], a["nbytes"], a["sync"], None)

    for name in ("logits", "ids", "counts", "prob", "n", "losses", "sync"):
        assert call(**{name: None}) == moe.ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 2}) == moe.ERR_INVALID_ARG, name
    assert call(ws=None) == moe.ERR_WORKSPACE
    assert call(nbytes=need - 1) == moe.ERR_WORKSPACE
    assert call(ws=FAKE + 128) == moe.ERR_INVALID_ARG
    assert L.moe_balance_workspace_bytes(ctypes.byref(d), None) == moe.ERR_INVALID_ARG
    with pytest.raises(moe.MoeError):
        moe.balance_workspace_bytes(moe.dims(4, 256, 512, 2000, 2))


def test_route_backward_refusals():
    L = moe.lib()
    d = moe.dims(4, 256, 512, 8, 2)
    base = dict(logits=FAKE, ids=FAKE, g=FAKE, dg=FAKE, dl=FAKE, counts=FAKE, n=FAKE, valid=None, out=FAKE + 4096)

    def call(**kw):
        a = dict(base, **kw)
        return L.moe_route_backward(ctypes.byref(d), a["logits"], a["ids"], a["g"], 1, a["dg"], a["dl"], a["counts"],
                                    a["n"], a["valid"], a["out"], None)

    for name in ("logits", "ids", "g", "counts", "n", "out"):
        assert call(**{name: None}) == moe.ERR_INVALID_ARG, name
    for name in ("logits", "ids", "g", "dg", "dl", "counts", "n", "out"):
        assert call(**{name: FAKE + 2}) == moe.ERR_INVALID_ARG, name
    assert call(out=FAKE) == moe.ERR_INVALID_ARG
    assert "logits_grad" in moe.last_error()


def test_combine_backward_refusals():
    L = moe.lib()
    d = moe.dims(4, 256, 512, 8, 2)
    args = [FAKE, FAKE + 4096, FAKE, FAKE, FAKE, FAKE + 8192]
    for i in range(5):
        bad = list(args)
        bad[i] = None
        assert L.moe_combine_backward(ctypes.byref(d), *bad, None) == moe.ERR_INVALID_ARG, i
    for i in range(6):
        bad = list(args)
        bad[i] += 2
        assert L.moe_combine_backward(ctypes.byref(d), *bad, None) == moe.ERR_INVALID_ARG, i
    for same in (0, 1):
        bad = list(args)
        bad[5] = bad[same]
        assert L.moe_combine_backward(ctypes.byref(d), *bad, None) == moe.ERR_INVALID_ARG
        assert "y_rows_grad" in moe.last_error()
    bad_h = moe.Dims(4, 250, 512, 8, 2, 128)
    assert L.moe_combine_backward(ctypes.byref(bad_h), *args, None) == moe.ERR_UNSUPPORTED


def _qm(N=64, K=256, bits=4, group=128):
    return moe.QMatrix(bits, group, torch.zeros(K // 128, N, 16 * bits, dtype=torch.uint8),
                       torch.zeros(N, K // group, dtype=torch.float16), torch.zeros(N, K // group, dtype=torch.int16))


def test_binding_refuses_wrong_tensors():
    w = _qm()
    assert (w.N, w.K) == (64, 256)
    with pytest.raises(ValueError, match="bits 4 or 2"):
        moe.QMatrix(3, 128, w.q, w.scale, w.bias)
    with pytest.raises(ValueError, match="q has shape"):
        moe.QMatrix(2, 128, w.q, w.scale, w.bias)
    with pytest.raises(ValueError, match="scale has shape"):
        moe.QMatrix(4, 64, w.q, w.scale, w.bias)
    with pytest.raises(ValueError, match="bias holds"):
        moe.QMatrix(4, 128, w.q, w.scale, w.scale.float())
    with pytest.raises(ValueError, match="not contiguous"):
        moe.QMatrix(4, 128, w.q, torch.zeros(2, 64, dtype=torch.float16).t(), w.bias)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    y = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.linear(w, x, y)
    with pytest.raises(ValueError, match="x holds"):
        moe.linear(w, x.float(), y)
    with pytest.raises(ValueError, match="x has shape"):
        moe.linear(w, x[:, :128], y)
    with pytest.raises(ValueError, match="y has shape"):
        moe.linear(w, x, y[:3])
    with pytest.raises(ValueError, match="y holds"):
        moe.linear(w, x, y.half())
    with pytest.raises(ValueError, match="rows are not contiguous"):
        moe.linear(w, torch.zeros(256, 4, dtype=torch.bfloat16).t(), y)
    with pytest.raises(ValueError, match="row_bias has shape"):
        moe.linear(w, x, y, row_bias=torch.zeros(63))
    with pytest.raises(ValueError, match="residual holds"):
        moe.linear(w, x, y, residual=y.float())
    buf = moe.LinearBuffers(torch.zeros(256, dtype=torch.uint8), torch.zeros(moe.LINEAR_SYNC_INTS, dtype=torch.int32))
    with pytest.raises(ValueError, match="sync has shape"):
        moe.linear_grad(w, y, x, moe.LinearBuffers(buf.workspace, buf.sync[:8]))
    with pytest.raises(ValueError, match="dx has shape"):
        moe.linear_grad(w, y, x[:, :128], buf)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.linear_grad(w, y, x, buf)
    with pytest.raises(ValueError, match="elements of type"):
        moe.linear_workspace_bytes(w, 4, torch.float16)


def test_binding_refuses_wrong_router_tensors():
    d = moe.dims(4, 256, 512, 8, 2)
    L, ids, g = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    c, P, n, loss = torch.zeros(8, dtype=torch.int32), torch.zeros(8), torch.zeros(1, dtype=torch.int32), torch.zeros(2)
    buf = moe.BalanceBuffers.allocate(d, device="cpu")
    with pytest.raises(ValueError, match="on the GPU"):
        moe.balance_loss(d, L, ids, c, P, n, loss, buf)
    with pytest.raises(ValueError, match="logits has shape"):
        moe.balance_loss(d, L[:3], ids, c, P, n, loss, buf)
    with pytest.raises(ValueError, match="topk_ids holds"):
        moe.balance_loss(d, L, ids.long(), c, P, n, loss, buf)
    with pytest.raises(ValueError, match="valid has shape"):
        moe.balance_loss(d, L, ids, c, P, n, loss, buf, valid=torch.ones(5, dtype=torch.bool))
    with pytest.raises(ValueError, match="losses has shape"):
        moe.balance_loss(d, L, ids, c, P, n, torch.zeros(1), buf)
    with pytest.raises(ValueError, match="needs expert_counts"):
        moe.route_backward(d, L, ids, g, True, torch.zeros(4, 8), losses_grad=loss)
    with pytest.raises(ValueError, match="topk_w_grad has shape"):
        moe.route_backward(d, L, ids, g, True, torch.zeros(4, 8), topk_w_grad=torch.zeros(4, 3))
    out, y = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(8, 256, dtype=torch.bfloat16)
    p2r = torch.arange(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="y_rows has shape"):
        moe.combine_backward(d, out, y[:7], p2r, g, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="pair_to_row has"):
        moe.combine_backward(d, out, y, p2r[:5], g, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="on the GPU"):
        moe.combine_backward(d, out, y, p2r, g, torch.zeros(4, 2))
