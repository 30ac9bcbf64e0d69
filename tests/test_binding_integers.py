"""Integers that a call's 32-bit arguments do not hold are refused, by way of the extension module and of ctypes: cut to
their low bits they would be other, valid numbers."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from test_long_context_cpu import BF, PLAN, FakeTensor, T

LARGE = (2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 63, 2 ** 64 + 7, 10 ** 30, -2 ** 31 - 1, -2 ** 32 + 7, -2 ** 63 - 1)


@pytest.fixture(params=["module", "ctypes"])
def way(request, monkeypatch):
    if request.param == "ctypes":
        monkeypatch.setattr(tp, "_entries", {})
        monkeypatch.setattr(tp, "_load_describe", lambda: None)
    elif tp._describe is None:
        pytest.skip("the extension module is not built")


def calls():
    q, k, n = [T(BF, 4, 256)] * 2, [T(BF, 40, 128)] * 2, FakeTensor(4)
    f = FakeTensor(64, dtype=torch.float32)
    return [lambda x: tp.tp_window_attn(PLAN, q, k, k, x, 0, q, stream=1), lambda x: tp.tp_window_attn(PLAN, q, k, k, 1, x, q, stream=1),
            lambda x: tp.tp_cache4_attn(PLAN, q, k, k, k, k, n, x, 0, q, stream=1),
            lambda x: tp.tp_cache4_attn(PLAN, q, k, k, k, k, n, 1, x, q, stream=1),
            lambda x: tp.tp_rotary(PLAN, n, f, q, None, q, None, layout=x, stream=1),
            lambda x: tp.tp_rotary(PLAN, n, f, q, None, q, None, inverse=x, stream=1)]


@pytest.mark.parametrize("large", LARGE)
def test_large_numbers_are_refused(way, large):
    for call in calls():
        with pytest.raises((ValueError, ctypes.ArgumentError), match="out of range"):
            call(large)
    for size in (tp.tp_window_attn_workspace_size, tp.tp_cache4_attn_workspace_size):
        for numbers in ((large, 0), (1, large)):
            with pytest.raises(ctypes.ArgumentError, match="out of range"):
                size(PLAN, 4, 40, *numbers)


def test_numbers_within(way):
    """The bounds themselves reach the library: its own refusals (a negative number, a layout that is not there), or the
    next check, of k's type or of the workspace."""
    for call in calls()[:5]:
        for x in (2 ** 31 - 1, -2 ** 31, -1):
            with pytest.raises(tp.TPError):
                call(x)
    for bad in (1.0, "1", None, b"1"):
        for call in calls()[:5]:
            with pytest.raises((TypeError, ctypes.ArgumentError)):
                call(bad)
    assert tp.tp_window_attn_workspace_size(PLAN, 4, 40, 2 ** 31 - 1, 2 ** 31 - 1) == tp.tp_window_attn_workspace_size(PLAN, 4, 40, 40, 0)
    assert tp.raw_status("tp_window_attn", None, None, None, None, ctypes.c_int32(3), 0, None, None, 0, None) == tp.TP_ERR_INVALID_ARG


def test_axes_of_a_list(way):
    q, n, f = [T(BF, 5, 256)] * 2, FakeTensor(2, 4), FakeTensor(3, dtype=torch.float32)
    for axis in ([0, 1, 2], [0, 2 ** 32, 1], (0, -1, 1), [2 ** 70] * 3):
        with pytest.raises(ValueError, match="axis"):
            tp.tp_rotary(PLAN, n, f, q, None, q, None, axis=axis, stream=1)
    with pytest.raises(tp.TPError):  # q has another number of tokens
        tp.tp_rotary(PLAN, n, f, q, None, q, None, axis=(0, 1, 0), stream=1)


@pytest.mark.skipif(tp._describe is None, reason="the extension module is not built")
def test_addresses_up_to_two_to_the_64():
    d = tp._load_describe()
    at = ctypes.cast(tp._lib.tp_window_attn, ctypes.c_void_p).value
    q = tp.arr([T(BF, 4, 256)] * 2)
    args = [PLAN.handle, q, q, q, 0, 0, q, 2 ** 64 - 16, 2 ** 64 - 1, 2 ** 64 - 1]
    assert d.window_attn(at, *args) == tp.TP_ERR_INVALID_ARG  # a window of 0
    for i, x in ((7, 2 ** 64), (8, -2 ** 63 - 1), (9, 2 ** 64), (4, 2 ** 31)):
        with pytest.raises(ValueError, match=f"argument {i + 1} is out of range: {x}"):
            d.window_attn(at, *args[:i], x, *args[i + 1:])
