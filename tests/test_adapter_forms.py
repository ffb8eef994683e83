"""Host-only: the sizes of adapter_forms.py reach every kernel form of the adapters, and
their bounds show a form that has lost a part of its float32 operands."""
import ctypes

import numpy as np
import pytest

import adapter_forms as forms
import quantized_expert_ffn_gemv_amd as moe
import tuning_ref as ref


def test_every_form_is_reached():
    seen = set()
    for case in forms.CASES:
        seen |= set(forms.forward(*case)) | set(forms.backward(*case))
    assert seen == forms.BUILT


def test_splits_rounds_and_chunks_are_reached():
    scans = [c for c in forms.CASES if not forms.planned(c[0])]
    plans = [c for c in forms.CASES if forms.planned(c[0])]
    two = [c for c in scans if len(forms.forward(*c)) == 2]
    # more than four splits joined at once (ranks to 32) and four at a time, both factors' sums
    for tiles in (1, 2):
        assert any(forms.rank_tiles(R) == tiles and forms.splits(T, n, K) > 4 for T, n, R, K, N, _ in two)
    assert {forms.rank_tiles(R) for T, n, R, K, N, _ in plans if forms.splits(T, n, K) > 1} == {1, 2, 4, 8}
    assert {forms.rank_tiles(R) for T, n, R, K, N, _ in plans if forms.splits(T, n, N) > 1} == {1, 2, 4, 8}
    assert {T > 4096 for T, *_ in plans} == {False, True} and max(T for T, *_ in plans) == 65536
    chunks = {(1 if R <= 16 else 2, forms.grad_chunk(T, R, (K, N))[0]) for T, n, R, K, N, _ in plans}
    assert {c for _, c in chunks} == {256, 512, 768, 1024} and {(1, 1024), (2, 1024)} <= chunks
    assert {forms.grad_chunk(T, E, (H,), False) for T, E, H in forms.ROUTER} == {
        (768, 6), (1280, 8), (2304, 1), (1280, 4), (512, 6), (256, 3), (2048, 32), (512, 3)}


@pytest.mark.parametrize("case", forms.CASES, ids=str)
def test_workspaces_hold_what_the_rules_take(case):
    T, n, R, K, N, f32 = case
    for grad, C in ((0, (K,)), (1, (K, N))):
        out = ctypes.c_size_t(0)
        m = moe.AdaptersC(None, None, (N + 7) // 8 * 8, None, None, n, R, K, N)
        assert moe.lib().moe_adapter_workspace_bytes(ctypes.byref(m), T, grad, ctypes.byref(out)) == moe.OK
        need = forms.splits(T, n, C[-1]) * T * 16 * forms.rank_tiles(R) * 4
        if grad:
            chunk, chunks = forms.grad_chunk(T, R, C)
            need += 4 * T * R + (4 * R * (K + N) * (chunks if n == 1 else 2 * T // chunk) if forms.planned(T) and T > chunk else 0)
        assert out.value >= need


def test_three_parts_are_all_of_a_float32():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(10000) * np.exp(12 * rng.standard_normal(10000))).astype(np.float32)
    assert np.array_equal(forms.cut(v, 3), v.astype(np.float64))
    off = np.abs(forms.cut(v, 2) - v) / np.abs(v)
    assert 2.0 ** -17 < off.max() < 2.0 ** -15


@pytest.mark.parametrize("case", forms.CASES, ids=str)
def test_the_bounds_show_a_lost_part(case):
    """The mistake is planted here, in the reference: two parts instead of three of h, of g and of dy."""
    s = forms.Sparse(*case)
    _, h, *_ = ref.adapter(s.f, s.ids, s.x_dense)
    h = h.astype(np.float32)
    want, bound = s.y(h)
    assert np.max(np.abs(s.y(h, 2)[0] - want) / bound) > 1.5
    full, lost = s.gradients(s.x), s.gradients(s.x, 2)
    for k, name in enumerate(("dx", "da", "db")):
        assert np.max(np.abs(lost[k] - full[k]) / full[3 + k]) > 1.5, name


def test_the_router_bound_shows_a_lost_part():
    for T, E, H in forms.ROUTER[:1]:
        dl, x, steps = forms.router_operands(T, E, H)
        want, size = dl.astype(np.float64).T @ x, np.abs(dl).astype(np.float64).T @ np.abs(x)
        assert np.max(np.abs(forms.cut(dl, 2).T @ x - want) / (steps * size + ref.TINY)) > 1.5
