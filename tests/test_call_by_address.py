"""The extension module's way to the library's long calls against ctypes': refusals, which need no GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp

d = tp._describe
pytestmark = pytest.mark.skipif(d is None, reason="the extension module is not built")


def test_calls_by_address():
    """The long calls' statuses are those of the same call through ctypes, whatever form an argument has."""
    plan = tp.tp_plan_create(2, 512, 4, 2, 128, 64)
    desc = tp.TpTensor(ptr=1 << 40, dtype=tp.TP_BF16, rows=4, cols=256, ld=256)
    two = tp.arr([desc, desc])
    at = lambda name: ctypes.cast(getattr(tp._lib, "tp_" + name), ctypes.c_void_p).value  # noqa: E731
    for window, sinks, q in ((0, 0, two), (-1, 0, two), (8, -1, two), (8, 0, None), (8, 0, two)):
        args = (plan.handle, q, two, two, window, sinks, two, None, 0, 1)
        want = tp.raw_status("tp_window_attn", *args)
        assert want != tp.TP_OK
        assert d.window_attn(at("window_attn"), *args) == want
        if q is not None:
            assert d.window_attn(at("window_attn"), plan.handle, ctypes.addressof(q), *args[2:]) == want

    class Three:
        def __index__(self):
            return 3

    axis = (ctypes.c_int32 * 3)(0, 0, 1)  # an axis that is not there
    args = [plan.handle, 4, 1 << 40, 1, 1 << 40, 3, axis, 0, 0, two, None, two, None, 1]
    assert d.rotary(at("rotary"), *args) == tp.raw_status("tp_rotary", *args) == tp.TP_ERR_INVALID_ARG
    args[3] = Three()
    args[1] = 5  # q has four tokens
    assert d.rotary(at("rotary"), *args) == tp.TP_ERR_INVALID_ARG
    for i, bad in ((1, None), (1, 2.0), (1, axis), (5, b"abc"), (9, 1.5), (9, torch.zeros(2)), (6, "x")):
        with pytest.raises((TypeError, BufferError)):
            d.rotary(at("rotary"), *args[:i], bad, *args[i + 1:])
    with pytest.raises(TypeError):
        d.rotary(at("rotary"), *args[:-1])
    with pytest.raises(ValueError):
        d.rotary(0, *args)
    for name, count in (("cache4_store", 11), ("cache4_load", 10), ("cache4_attn", 14)):
        none = [0] * count
        assert getattr(d, name)(at(name), *none) == tp.raw_status("tp_" + name, *none) == tp.TP_ERR_INVALID_ARG


def test_calls_without_the_module(monkeypatch):
    monkeypatch.setattr(tp, "_entries", {})
    monkeypatch.setattr(tp, "_load_describe", lambda: None)
    assert tp._entry("rotary") is tp._lib.tp_rotary
