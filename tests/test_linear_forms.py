"""Host-only: the sizes of linear_forms.py reach every kernel form that the library
builds, and what moe_linear_kernels says agrees with the workspaces."""
import ctypes

import pytest

import linear_forms as forms
import quantized_expert_ffn_gemv_amd as moe


@pytest.mark.parametrize("bits,group", forms.FORMATS)
def test_every_streamed_form_is_reached(bits, group):
    seen = set()
    for runs in forms.RUNS:
        for T, N in forms.TOKENS_ROWS:
            k = forms.kernels(T, N, 128 * runs, bits, group)
            assert k[0] == moe.LINEAR_STREAMED and k[5] == 1
            seen.add(k[1:5])
    assert seen == forms.stream_forms(bits, group)


@pytest.mark.parametrize("table,f32,grad", [(forms.FORWARD, False, False), (forms.FORWARD, True, False),
                                            (forms.GRAD_BF16, False, True), (forms.GRAD_F32, True, True)])
def test_every_tile_is_reached_with_and_without_splits(table, f32, grad):
    seen = set()
    for size in table:
        k = forms.kernels(*size, f32, grad)
        assert k[0] == moe.LINEAR_LAID_OUT and k[6] == (2 if f32 and grad else 1)
        seen.add(forms.tile_of(k))
    assert seen == {t + (s,) for t in forms.TILES for s in (False, True)}


def test_splits_of_the_streamed_gradient():
    assert [forms.kernels(T, N, K, 4, 128, grad=True)[:2] for T, N, K in
            ((1, 4096, 4096), (8, 49999, 4096), (1, 200, 128), (5000, 300, 256))] == [(1, 8), (1, 8), (1, 1), (1, 1)]


def test_no_workspace_for_few_tokens():
    for bits, group in forms.FORMATS:
        for N in (1, 15, 100, 3000, 50000, 1 << 20):
            for K in (128, 640, 2048, 5120, 8192):
                for f32 in (False, True):
                    assert forms.kernels(16, N, K, bits, group, f32)[0] == moe.LINEAR_STREAMED
                    w = moe.QMatrixC(None, None, None, N, K, group, bits)
                    out = ctypes.c_size_t(1)
                    assert moe.lib().moe_linear_workspace_bytes(ctypes.byref(w), 16, int(f32), 0, ctypes.byref(out)) == moe.OK
                    assert out.value == 0


def test_kernels_refusals():
    L, out = moe.lib(), (ctypes.c_int32 * 8)(*[7] * 8)
    w = moe.QMatrixC(None, None, None, 64, 256, 128, 4)
    assert L.moe_linear_kernels(ctypes.byref(w), 4, 0, 0, None) == moe.ERR_INVALID_ARG
    assert L.moe_linear_kernels(None, 4, 0, 0, out) == moe.ERR_INVALID_ARG
    assert L.moe_linear_kernels(ctypes.byref(w), -1, 0, 0, out) == moe.ERR_INVALID_ARG
    assert L.moe_linear_kernels(ctypes.byref(w), 4, 2, 0, out) == moe.ERR_UNSUPPORTED
    assert list(out) == [7] * 8
    assert L.moe_linear_kernels(ctypes.byref(w), 0, 0, 0, out) == moe.OK and not any(out)


def test_the_size_that_is_laid_out_whatever_its_types():
    for f32 in (False, True):
        for grad in (False, True):
            assert forms.kernels(*forms.LAID_OUT, f32, grad)[0] == moe.LINEAR_LAID_OUT


def test_workspaces_are_bounded_and_quickly_told():
    """2.3 GB for any sizes, never less for more tokens, and no call's own need is more."""
    for N in (1, 1000, 49999, 1 << 20):
        for K in (128, 4096, 8320, 32768):
            for f32 in (False, True):
                for grad in (False, True):
                    w, sizes = moe.QMatrixC(None, None, None, N, K, 32, 4), []
                    for T in (1, 16, 17, 255, 300, 5000, 20000, 65536):
                        out = ctypes.c_size_t(0)
                        L = moe.lib()
                        assert L.moe_linear_workspace_bytes(ctypes.byref(w), T, int(f32), int(grad), ctypes.byref(out)) == moe.OK
                        sizes.append(out.value)
                    assert sizes == sorted(sizes) and sizes[-1] <= 2.3e9


def test_tokens_in_turns():
    for size, grad, turns in ((forms.LAID_OUT, False, 1), (forms.LAID_OUT, True, 1), (forms.TURNS[0], False, 2),
                              (forms.TURNS[1], True, 2), (forms.TURNS[2], True, 2)):
        assert forms.kernels(*size, size == forms.TURNS[2], grad)[7] == turns
