"""Host-only: the sizes of adapter_forms.py reach every kernel form of the adapters."""
import ctypes

import pytest

import adapter_forms as forms
import quantized_expert_ffn_gemv_amd as moe


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
        (512, 9), (1280, 8), (2304, 1), (1280, 4), (256, 12), (256, 3), (256, 256)}


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
