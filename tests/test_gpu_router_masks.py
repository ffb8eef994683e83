"""The router's backward pass where padded tokens hold anything, against the 64-bit
forms of weights_ref.py."""
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
