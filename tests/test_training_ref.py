"""The plain 64-bit forms that the GPU operators are compared with, checked on the
CPU against independent definitions: autograd in float64 and central differences."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import oracle
import quantized_expert_ffn_gemv_amd as moe
import weights_ref as ref


@pytest.mark.parametrize("bits", [4, 2])
@pytest.mark.parametrize("group", [128, 64, 32])
def test_weights_match_the_oracle_and_the_layout(bits, group):
    rng = np.random.default_rng(bits + group)
    N, K = 24, 384
    row_major = rng.integers(0, 256, (N, K * bits // 8), dtype=np.uint8)
    _, s, b = ref.make_matrix(rng, N, K, bits, group)
    W, mag = ref.weights(moe.group_major(row_major, bits), s, b, bits, group)
    want = oracle.dequant_matrix(row_major, s.view(np.uint16), b.view(np.uint16), bits)
    np.testing.assert_allclose(W, want, rtol=1e-15, atol=1e-15)
    assert np.all(mag >= np.abs(W) - 1e-12)


def _case(E, k, renorm, seed):
    rng = np.random.default_rng(seed)
    T = 6
    L = rng.normal(size=(T, E)) * 2
    ids = np.argsort(-L, axis=1, kind="stable")[:, :k]
    valid = np.array([1, 1, 0, 1, 1, 0], dtype=np.uint8)
    return rng, T, L, ids, valid


def _loss(L, ids, k, renorm, dgates, a, z, f, valid):
    """a balance + z z-loss + <dgates, gates> of torch logits, the counts constant."""
    V = valid.sum()
    E = L.shape[1]
    p = torch.softmax(L, 1)
    m = torch.from_numpy(valid.astype(np.float64))
    bal = E * (f * (p * m[:, None]).sum(0) / V).sum()
    zl = (torch.logsumexp(L, 1) ** 2 * m).sum() / V
    picked = torch.gather(L, 1, torch.from_numpy(ids))
    g = torch.softmax(picked, 1) if renorm else torch.gather(p, 1, torch.from_numpy(ids))
    return a * bal + z * zl + (g * dgates).sum(), g


@pytest.mark.parametrize("E,k", [(1, 1), (5, 2), (8, 8), (33, 4)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_formula(E, k, renorm):
    rng, T, L, ids, valid = _case(E, k, renorm, 7 * E + k)
    dg = rng.normal(size=(T, k))
    a, z = 0.7, 0.03
    counts, _, n, _, _ = ref.balance(L, ids, k, valid)
    f = torch.from_numpy(counts / (n * k))
    Lt = torch.from_numpy(L.copy()).requires_grad_(True)
    loss, g = _loss(Lt, ids, k, renorm, torch.from_numpy(dg), a, z, f, valid)
    loss.backward()
    d, mag = ref.route_backward(L, ids, g.detach().numpy(), renorm, dg, (a, z), counts, n, valid)
    np.testing.assert_allclose(d, Lt.grad.numpy(), rtol=0, atol=1e-12 * (1 + mag.max()))
    assert np.all(mag >= np.abs(d) - 1e-12)
    # central differences: error h^2 of the third derivative plus eps / h
    h = 1e-5
    for t, e in [(0, 0), (2, E - 1), (5, E // 2)]:
        step = np.zeros_like(L)
        step[t, e] = h
        hi, lo = (float(_loss(torch.from_numpy(L + s * step), ids, k, renorm, torch.from_numpy(dg), a, z, f, valid)[0])
                  for s in (1, -1))
        assert abs((hi - lo) / (2 * h) - d[t, e]) < 1e-8


def test_balance_against_loops():
    rng, T, L, ids, valid = _case(9, 3, True, 3)
    L[1, 4] = -np.inf
    L[3] = -np.inf
    counts, P, n, bal, z = ref.balance(L, ids, 3, valid)
    want_c, want_P, want_n, want_z = np.zeros(9, int), np.zeros(9), 0, 0.0
    for t in range(T):
        if not valid[t] or t == 3:
            continue
        want_n += 1
        total = sum(np.exp(v) for v in L[t])
        for e in range(9):
            want_P[e] += np.exp(L[t, e]) / total
        want_z += np.log(total) ** 2
        for j in range(3):
            want_c[ids[t, j]] += 1
    assert n == want_n and np.array_equal(counts, want_c)
    np.testing.assert_allclose(P, want_P / want_n, rtol=1e-12)
    np.testing.assert_allclose(z, want_z / want_n, rtol=1e-12)
    np.testing.assert_allclose(bal, 9 * sum(want_c[e] / (want_n * 3) * want_P[e] / want_n for e in range(9)), rtol=1e-12)
    assert ref.balance(L, ids, 3, np.zeros(T, np.uint8))[2:] == (0, 0.0, 0.0)


def test_uniform_routing_has_balance_loss_one():
    L = np.zeros((8, 4))
    ids = np.stack([np.arange(8) % 4, (np.arange(8) + 1) % 4], axis=1)
    _, P, n, bal, z = ref.balance(L, ids, 2)
    assert n == 8 and np.allclose(P, 0.25) and abs(bal - 1) < 1e-15 and abs(z - np.log(4) ** 2) < 1e-15


def test_bf16_round_matches_the_input_generator():
    a = np.random.default_rng(0).normal(size=1000).astype(np.float32)
    bits = mi.f32_to_bf16_bits(a)
    assert np.array_equal(ref.bf16_round(a).view(np.uint32) >> 16, bits)
