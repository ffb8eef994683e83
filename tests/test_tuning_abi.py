"""Host-side refusals of the adapters, token probabilities and checkpoints: nothing is
launched, every call below fails (or is a no-op) on the host."""
import ctypes

import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe

FAKE = 0x10000000
FAR = 0x7000000000
BIG = 1 << 42


def lib():
    return moe.lib()


def by(s):
    return None if s is None else ctypes.byref(s)


def adapters(a=FAKE, b=FAKE, ldb=64, scale=FAKE, rank=None, n=4, R=16, K=256, N=64):
    return moe.AdaptersC(a, b, ldb, scale, rank, n, R, K, N)


@pytest.mark.parametrize("kw,T,status", [
    (dict(n=0), 4, moe.ERR_UNSUPPORTED), (dict(n=1025), 4, moe.ERR_UNSUPPORTED),
    (dict(R=0), 4, moe.ERR_UNSUPPORTED), (dict(R=129), 4, moe.ERR_UNSUPPORTED),
    (dict(K=0), 4, moe.ERR_UNSUPPORTED), (dict(K=200), 4, moe.ERR_UNSUPPORTED), (dict(K=32896), 4, moe.ERR_UNSUPPORTED),
    (dict(N=7), 4, moe.ERR_UNSUPPORTED), (dict(N=1 << 21, ldb=1 << 21), 4, moe.ERR_UNSUPPORTED),
    (dict(ldb=56), 4, moe.ERR_INVALID_ARG), (dict(N=60, ldb=60), 4, moe.ERR_INVALID_ARG),
    (dict(), -1, moe.ERR_INVALID_ARG), (dict(), 65537, moe.ERR_UNSUPPORTED),
])
def test_adapter_limits(kw, T, status):
    out = ctypes.c_size_t(0)
    for grad in (0, 1):
        assert lib().moe_adapter_workspace_bytes(by(adapters(**kw)), T, grad, by(out)) == status
        assert moe.last_error()


def test_adapter_workspace_grows_with_the_tokens():
    for kw in (dict(), dict(n=1, R=128, K=8192, N=5000, ldb=5000), dict(n=1024, R=3)):
        for grad in (0, 1):
            sizes = []
            for T in [0, 1, 2, 15, 16, 17, 255, 256, 257, 511, 512, 513, 600, 1024, 1025, 2048, 4096, 5000, 65535, 65536]:
                out = ctypes.c_size_t(0)
                assert lib().moe_adapter_workspace_bytes(by(adapters(**kw)), T, grad, by(out)) == moe.OK
                sizes.append(out.value)
            assert sizes == sorted(sizes) and sizes[-1] < 1 << 33
    assert lib().moe_adapter_workspace_bytes(None, 4, 0, by(ctypes.c_size_t(0))) == moe.ERR_INVALID_ARG
    assert lib().moe_adapter_workspace_bytes(by(adapters()), 4, 0, None) == moe.ERR_INVALID_ARG


def _adapter(m=None, T=4, ids=FAKE, x=FAKE, ldx=256, base=None, ldbase=64, y=FAR, ldy=64, t=moe.BF16, h=None, ws=FAKE, n=BIG):
    return lib().moe_adapter(by(m or adapters()), T, ids, x, ldx, base, ldbase, y, ldy, t, h, ws, n, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(m=adapters(a=None)), 1, "a is NULL"), (dict(m=adapters(a=FAKE + 8)), 1, "a is not 16"),
    (dict(m=adapters(b=FAKE + 2)), 1, "b is not 16"), (dict(m=adapters(scale=None)), 1, "scale is NULL"),
    (dict(m=adapters(rank=FAKE + 2)), 1, "rank"), (dict(ids=None), 1, "ids is NULL"), (dict(ids=FAKE + 1), 1, "ids"),
    (dict(x=None), 1, "x is NULL"), (dict(x=FAKE + 1), 1, "x is not"), (dict(ldx=255), 1, "rows of x"),
    (dict(y=None), 1, "y is NULL"), (dict(y=FAR + 2, t=moe.F32), 1, "y is not"), (dict(ldy=63), 1, "rows of y"),
    (dict(base=FAKE + 1), 1, "base"), (dict(base=FAKE, ldbase=60), 1, "rows of base"),
    (dict(base=FAR, ldbase=72), 1, "differs from it"), (dict(h=FAKE + 2), 1, "h is not"),
    (dict(t=2), 2, "element type"), (dict(ws=None), 3, "workspace"), (dict(n=16), 3, "workspace"),
    (dict(ws=FAKE + 16), 1, "workspace"), (dict(y=FAKE + 512), 1, "overlaps"), (dict(base=FAR + 64, ldbase=64), 1, "overlaps"),
])
def test_adapter_refusals(kw, status, word):
    assert _adapter(**kw) == status
    assert word in moe.last_error()


def test_no_tokens():
    assert _adapter(T=0, ids=None, x=None, y=None, ws=None, n=0) == moe.OK
    assert lib().moe_logprobs(0, 8, None, 8, 0, None, None, None, None, 0, None, None, None, 0, None, None) == moe.OK
    assert lib().moe_logprobs_grad(0, 8, None, 8, 0, None, None, None, None, None, None, 8, 0, None) == moe.OK
    assert lib().moe_checkpoint_save(by(moe.CheckpointC(None, None, 0, 256)), None, 256, None) == moe.OK
    d = moe.dims(0, 256, 128, 8, 2)
    assert lib().moe_combine_backward_saved(by(d), None, by(moe.CheckpointC(None, None, 0, 256)), None, None, None, None, None) == moe.OK


def checkpoint(q=FAKE, scale=FAKE, rows=4, K=256):
    return moe.CheckpointC(q, scale, rows, K)


def _grad(m=None, T=4, ids=FAKE, dy=FAKE, lddy=64, t=moe.BF16, x=FAKE, ldx=256, saved=None, h=FAKE, base=None, ldbase=256,
          dx=FAR, lddx=256, da=FAR, db=FAR, ws=FAKE, n=BIG):
    return lib().moe_adapter_grad(by(m or adapters()), T, ids, dy, lddy, t, x, ldx, by(saved), h, base, ldbase, dx, lddx, da, db, ws, n, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(ids=None), 1, "ids"), (dict(dy=None), 1, "dy is NULL"), (dict(lddy=63), 1, "rows of dy"),
    (dict(dy=FAKE + 2, t=moe.F32), 1, "dy is not"), (dict(t=3), 2, "element type"), (dict(x=FAKE + 1), 1, "x is not"),
    (dict(ldx=128), 1, "rows of x"), (dict(x=None), 1, "either x or x_saved"), (dict(saved=checkpoint()), 1, "either x or x_saved"),
    (dict(x=None, saved=checkpoint(rows=3)), 1, "x_saved"), (dict(x=None, saved=checkpoint(K=128)), 1, "x_saved"),
    (dict(x=None, saved=checkpoint(q=None)), 1, "NULL"), (dict(x=None, saved=checkpoint(q=FAKE + 8)), 1, "16-byte"),
    (dict(h=None), 1, "h is NULL"), (dict(da=FAR + 2), 1, "da"), (dict(db=FAR + 1), 1, "db"), (dict(lddx=200), 1, "rows of dx"),
    (dict(base=FAKE, ldbase=128), 1, "dx_base"), (dict(base=FAR, ldbase=512), 1, "differs from it"),
    (dict(dx=FAKE), 1, "overlaps"), (dict(base=FAR + 512), 1, "overlaps"), (dict(ws=None), 3, "workspace"),
])
def test_adapter_grad_refusals(kw, status, word):
    assert _grad(**kw) == status
    assert word in moe.last_error()


def _logprobs(T=4, V=100, L=FAKE, ld=100, t=moe.F32, tokens=FAKE, logp=FAKE, stats=FAKE, ent=None, n=0, ids=None, top=None,
              ws=FAKE, nbytes=BIG, sync=FAKE):
    return lib().moe_logprobs(T, V, L, ld, t, tokens, logp, stats, ent, n, ids, top, ws, nbytes, sync, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(T=-1), 1, "T"), (dict(T=65537), 2, "T"), (dict(V=0), 2, "V"), (dict(V=1048577), 2, "V"), (dict(n=65), 2, "n_top"),
    (dict(n=-1), 2, "n_top"), (dict(t=2), 2, "element type"), (dict(L=None), 1, "logits is NULL"), (dict(L=FAKE + 2), 1, "logits"),
    (dict(ld=99), 1, "rows of logits"), (dict(tokens=None), 1, "tokens"), (dict(logp=None), 1, "logp"), (dict(stats=FAKE + 2), 1, "stats"),
    (dict(ent=FAKE + 1), 1, "entropy"), (dict(n=3, top=FAKE), 1, "top_ids"), (dict(n=3, ids=FAKE), 1, "top_logp"),
    (dict(sync=None), 1, "sync"), (dict(sync=FAKE + 64), 1, "sync"), (dict(V=50000, ld=50000, ws=None), 3, "workspace"),
    (dict(V=50000, ld=50000, ws=FAKE + 16), 1, "workspace"), (dict(V=50000, ld=50000, nbytes=64), 3, "workspace"),
])
def test_logprobs_refusals(kw, status, word):
    assert _logprobs(**kw) == status
    assert word in moe.last_error()


def test_logprobs_workspace_serves_fewer_tokens():
    def size(T, V, n):
        out = ctypes.c_size_t(0)
        assert lib().moe_logprobs_workspace_bytes(T, V, n, by(out)) == moe.OK
        return out.value
    for V in (1, 2048, 2049, 49999, 1048576):
        for n in (0, 1, 20, 64):
            sizes = [size(T, V, n) for T in range(0, 600, 7)] + [size(65536, V, n)]
            assert sizes == sorted(sizes)


def _lgrad(T=4, V=100, L=FAKE, ld=100, t=moe.F32, tokens=FAKE, stats=FAKE, w=FAKE, ent=None, u=None, g=FAR, ldg=100, tg=moe.F32):
    return lib().moe_logprobs_grad(T, V, L, ld, t, tokens, stats, w, ent, u, g, ldg, tg, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(T=65537), 2, "T"), (dict(V=0), 2, "V"), (dict(t=5), 2, "element type"), (dict(tg=5), 2, "element type"),
    (dict(L=None), 1, "logits"), (dict(g=None), 1, "logits_grad"), (dict(ldg=99), 1, "rows of logits_grad"), (dict(tokens=None), 1, "tokens"),
    (dict(stats=None), 1, "stats"), (dict(w=FAKE + 2), 1, "logp_grad"), (dict(u=FAKE), 1, "entropy"), (dict(u=FAKE + 1, ent=FAKE), 1, "entropy_grad"),
    (dict(g=FAKE, tg=moe.BF16), 1, "overlaps"), (dict(g=FAKE, ldg=104), 1, "overlaps"), (dict(g=FAKE + 8), 1, "overlaps"),
])
def test_logprobs_grad_refusals(kw, status, word):
    assert _lgrad(**kw) == status
    assert word in moe.last_error()


@pytest.mark.parametrize("kw,status", [(dict(K=100), 2), (dict(K=0), 2), (dict(K=65536), 2), (dict(rows=-1), 2), (dict(rows=4194305), 2), (dict(rows=4194304, K=32768), 2),
                                       (dict(q=None), 1), (dict(scale=None), 1), (dict(q=FAKE + 4), 1), (dict(scale=FAKE + 2), 1)])
def test_checkpoint_refusals(kw, status):
    c = checkpoint(**kw)
    assert lib().moe_checkpoint_save(by(c), FAR, 65536, None) == status
    assert lib().moe_checkpoint_restore(by(c), FAR, 65536, None) == status
    for x, ld in ((None, 256), (FAR + 1, 256), (FAR, 255)):
        assert lib().moe_checkpoint_save(by(checkpoint()), x, ld, None) == moe.ERR_INVALID_ARG
        assert lib().moe_checkpoint_restore(by(checkpoint()), x, ld, None) == moe.ERR_INVALID_ARG


def test_saved_gates_and_router_weight_refusals():
    d = moe.dims(4, 256, 128, 8, 2)

    def gates(d=d, out=FAKE, y=checkpoint(rows=8), p2r=FAKE, g=FAKE, dg=FAKE, dy=None):
        return lib().moe_combine_backward_saved(by(d), out, by(y), p2r, g, dg, dy, None)

    assert gates(y=None) == gates(y=checkpoint(rows=7)) == gates(y=checkpoint(rows=8, K=128)) == moe.ERR_INVALID_ARG
    assert gates(out=FAKE + 8) == gates(p2r=None) == gates(dg=None) == gates(dy=FAKE) == gates(dy=FAR, g=None) == moe.ERR_INVALID_ARG
    assert gates(d=moe.dims(4, 200, 128, 8, 2)) == moe.ERR_UNSUPPORTED

    def weight(d=d, dl=FAKE, x=FAKE, ldx=256, saved=None, dw=FAR, db=None, ws=FAKE, n=BIG):
        return lib().moe_router_weight_grad(by(d), dl, x, ldx, by(saved), dw, db, ws, n, None)

    bad = moe.ERR_INVALID_ARG
    assert weight(dl=None) == weight(x=None) == weight(saved=checkpoint()) == weight(dw=None) == weight(db=FAR + 1) == bad
    assert weight(ldx=255) == weight(x=FAKE + 1) == weight(x=None, saved=checkpoint(rows=3)) == weight(x=None, saved=checkpoint(K=128)) == bad
    assert weight(d=moe.dims(4096, 256, 128, 8, 2), ws=None, n=0) == moe.ERR_WORKSPACE
    assert weight(d=moe.dims(4, 8320, 128, 8, 2)) == moe.ERR_UNSUPPORTED


def test_checkpoints_in_the_rows_own_memory_are_refused():
    bad = moe.ERR_INVALID_ARG
    # 4 rows of 256: 1024 bytes of codes, 32 of scales; the rows span 2048 bytes (3 ld + 256 elements)
    for c, x, ld in ((checkpoint(q=FAKE, scale=FAR), FAKE, 256), (checkpoint(q=FAKE, scale=FAR), FAKE - 2046, 256),
                     (checkpoint(q=FAKE, scale=FAR), FAKE + 1022, 256), (checkpoint(q=FAKE, scale=FAR), FAKE - 2560, 512),
                     (checkpoint(q=FAR, scale=FAKE), FAKE + 30, 256), (checkpoint(q=FAR, scale=FAKE), FAKE - 2046, 256)):
        assert lib().moe_checkpoint_save(by(c), x, ld, None) == bad
        assert lib().moe_checkpoint_restore(by(c), x, ld, None) == bad
        assert b"overlaps" in lib().moe_last_error()
    d = moe.dims(4, 256, 128, 8, 2)
    y = checkpoint(q=FAKE, scale=FAKE + 65536, rows=8)
    for dy in (FAKE - 4080, FAKE + 2032, FAKE + 65536 + 48, FAKE + 65536 - 4080, FAR + 2032, FAR - 4080):
        assert lib().moe_combine_backward_saved(by(d), FAR, by(y), FAR, FAR, FAR, dy, None) == bad
        assert b"one of the inputs" in lib().moe_last_error()


def test_binding_refuses_wrong_tensors():
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    a, b, s = torch.zeros(3, 4, 256, dtype=bf), torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3)
    m = moe.Adapters(a, b, s)
    assert (m.n, m.R, m.K, m.N, m._c.ldb) == (3, 4, 256, 64, 64)
    wide = torch.zeros(3, 4, 72, dtype=bf)
    assert moe.Adapters(a, wide[:, :, :67], s)._c.ldb == 72
    for wrong, word in ((torch.zeros(3, 4, 67, dtype=bf), "one stride"), (torch.zeros(3, 5, 64, dtype=bf), "b is"), (b.float(), "b is"),
                        (torch.zeros(3, 64, 4, dtype=bf).transpose(1, 2), "one stride"), (wide[:, :, 5:], "ends before")):
        with pytest.raises(ValueError, match=word):
            moe.Adapters(a, wrong, s)
    with pytest.raises(ValueError, match="scale has shape"):
        moe.Adapters(a, b, torch.zeros(2))
    with pytest.raises(ValueError, match="rank holds"):
        moe.Adapters(a, b, s, torch.zeros(3))
    packed = moe.Adapters.pack([torch.ones(2, 128), torch.ones(3, 128)], [torch.ones(9, 2), torch.full((9, 3), 2.0)], [1, 0.5], device="cpu")
    assert packed.R == 3 and packed.N == 9 and packed.rank.tolist() == [2, 3] and float(packed.b[1].sum()) == 54 and float(packed.a[0].sum()) == 256
    ids, x, y = torch.zeros(5, dtype=i32), torch.zeros(5, 256, dtype=bf), torch.zeros(5, 64, dtype=bf)
    buf = moe.AdapterBuffers.allocate(m, 5, grad=True)
    h = torch.zeros(5, 4)
    for kw, word in ((dict(), "on the GPU"), (dict(ids=ids.long()), "ids holds"), (dict(x=x[:4]), "has shape"), (dict(y=y.half()), "y holds"),
                     (dict(base=y.float()), "base holds"), (dict(h=h[:4]), "h has shape")):
        args = dict(dict(ids=ids, x=x, y=y, base=None, h=None), **kw)
        with pytest.raises(ValueError, match=word):
            moe.adapter(m, args["ids"], args["x"], args["y"], buf, base=args["base"], h=args["h"])
    with pytest.raises(ValueError, match="da needs x"):
        moe.adapter_grad(m, ids, y, None, h, buf, da=torch.zeros(3, 4, 256))
    with pytest.raises(ValueError, match="db has shape"):
        moe.adapter_grad(m, ids, y, x, h, buf, db=torch.zeros(3, 4, 63))
    with pytest.raises(ValueError, match="dx_base without"):
        moe.adapter_grad(m, ids, y, x, h, buf, dx_base=x)
    c = moe.Checkpoint.allocate(4, 256, device="cpu")
    with pytest.raises(ValueError, match="x keeps"):
        moe.adapter_grad(m, ids, y, c, h, buf, da=torch.zeros(3, 4, 256))
    with pytest.raises(ValueError, match="multiple of 128"):
        moe.Checkpoint(torch.zeros(4, 200, dtype=torch.int8), torch.zeros(4, 1))
    with pytest.raises(ValueError, match="scale has shape"):
        moe.Checkpoint(torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4, 1))
    with pytest.raises(ValueError, match="x has shape"):
        moe.checkpoint_save(x, c)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.checkpoint_restore(c, x[:4])
    L, tok, stats = torch.zeros(5, 9), torch.zeros(5, dtype=i32), torch.zeros(5, 2)
    lb = moe.LogprobBuffers.allocate(5, 9, 2, device="cpu")
    with pytest.raises(ValueError, match="go together"):
        moe.logprobs(L, tok, torch.zeros(5), stats, lb, top_ids=torch.zeros(5, 2, dtype=i32))
    with pytest.raises(ValueError, match="top_logp has shape"):
        moe.logprobs(L, tok, torch.zeros(5), stats, lb, top_ids=torch.zeros(5, 2, dtype=i32), top_logp=torch.zeros(5, 3))
    with pytest.raises(ValueError, match="tokens holds"):
        moe.logprobs(L, tok.long(), torch.zeros(5), stats, lb)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.logprobs(L, tok, torch.zeros(5), stats, lb)
    with pytest.raises(ValueError, match="needs entropy"):
        moe.logprobs_grad(L, tok, stats, L, entropy_grad=torch.zeros(5))
    d = moe.dims(5, 256, 128, 8, 2)
    with pytest.raises(ValueError, match="y_rows keeps"):
        moe.combine_backward(d, x, c, torch.zeros(10, dtype=i32), torch.zeros(5, 2), torch.zeros(5, 2))
    with pytest.raises(ValueError, match="w_router_grad has shape"):
        moe.router_weight_grad(d, torch.zeros(5, 8), x, torch.zeros(8, 128), moe.RouterWeightBuffers.allocate(d, device="cpu"))


def test_orchestration_refuses():
    d = moe.dims(4, 256, 128, 8, 2)
    buf = moe.LayerBuffers.allocate(d, device="cpu")
    grads = moe.RouterGradBuffers.allocate(d, device="cpu")
    out = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="goes with w_router_grad"):
        moe.router_backward(buf, grads, out, router_bias_grad=torch.zeros(8))
    with pytest.raises(ValueError, match="needs the step's x"):
        moe.router_backward(buf, grads, out, w_router_grad=torch.zeros(8, 256))
    w = moe.QMatrix(4, 128, torch.zeros(2, 64, 64, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.float16), torch.zeros(64, 2, dtype=torch.float16))
    m = moe.Adapters(torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3))
    with pytest.raises(ValueError, match="beside a projection"):
        moe.adapted_linear(w, m, None, None, None, None)
    with pytest.raises(ValueError, match="beside a projection"):
        moe.adapted_linear_backward(w, m, None, None, None, None, None)
