"""The router's backward pass where padded tokens hold anything, and the bits of its
softmax: against the 64-bit forms of weights_ref.py."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(seed, T, E, k):
    rng = np.random.default_rng(seed)
    L = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, L, ids


def route(L, ids, g, renorm, dg, counts, n, valid):
    T, E = L.shape
    out = torch.full((T, E), 7.0, device=DEV)
    moe.route_backward(moe.dims(T, 128, 128, E, ids.shape[1]), dev(L), dev(ids), dev(g), renorm, out,
                       None if dg is None else dev(dg), torch.tensor([0.5, 0.02], device=DEV), dev(counts.astype(np.int32)),
                       torch.tensor([n], dtype=torch.int32, device=DEV), dev(valid))
    return out.cpu().numpy()


@pytest.mark.parametrize("T,E,k", [(9, 5, 2), (40, 64, 4), (70, 128, 3), (33, 200, 8), (20, 500, 2), (300, 1024, 5)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_padded_tokens_may_hold_anything(T, E, k, bad):
    """Tokens that are not valid get the gates' part alone, whatever their logits are."""
    rng, L, ids = make(T, T, E, k)
    valid = np.ones(T, np.uint8)
    valid[::3] = 0
    clean = L.copy()
    L[::3] = bad
    L[3, 1:] = 0.0
    counts, _, n, _, _ = ref.balance(clean, ids, k, valid)
    g = np.full((T, k), 1.0 / k, np.float32)
    dg = rng.standard_normal((T, k)).astype(np.float32)
    for grads in (None, dg):
        got = route(L, ids, g, True, grads, counts, n, valid)
        want, mag = ref.route_backward(clean, ids, g, True, grads, (0.5, np.float32(0.02)), counts, n, valid)
        assert np.all(np.abs(got - want) <= (64 + 4 * ref.spread(clean)) * U * mag + 1e-37)
    # gates from the softmax over all experts, without their gradient: the losses' part alone
    got = route(L, ids, g, False, None, counts, n, valid)
    assert not got[::3].any() and np.isfinite(got).all()


@pytest.mark.parametrize("E", [3, 60, 128, 256, 512, 1000])
def test_softmax_keeps_small_probabilities(E):
    """Logits whose differences are exact: a probability is off by a few roundings, however small it is.

    p = exp(d) / S: the exponential's 2 U (hardware's 1 ulp) and its argument's correction, the
    product with 1 / S (2 U) and S's own relative error (at most 16 values a lane, then 6
    levels: 22 U, of sums whose small terms count nothing): 32 U in all."""
    rng = np.random.default_rng(E)
    T, k = 8, 2
    L = (-rng.integers(0, 80 * 1024, (T, E)) / 1024.0).astype(np.float32)
    L[:, 0] = 0.0
    ids = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    d = moe.dims(1, 128, 128, E, k)
    buf = moe.BalanceBuffers.allocate(d)
    for t in range(T):
        c, P = torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV)
        n, loss = torch.empty(1, dtype=torch.int32, device=DEV), torch.empty(2, device=DEV)
        moe.balance_loss(d, dev(L[t:t + 1]), dev(ids[t:t + 1]), c, P, n, loss, buf)
        want = ref.softmax(L[t:t + 1])[0][0]
        off = np.abs(P.double().cpu().numpy() - want) / (32 * U * want)
        assert off.max() <= 1.0, f"{off.max():.3g} times the bound"
