"""The binding's descriptors written in C against those that its interpreted code packs."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp

d = tp._describe
pytestmark = pytest.mark.skipif(d is None, reason="the extension module is not built")


class Fake:
    """What the module reads of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, stride, dtype=torch.bfloat16, ptr=4096):
        self.shape, self._stride, self.dtype, self._ptr = torch.Size(shape), stride, dtype, ptr

    def stride(self):
        return self._stride

    def data_ptr(self):
        return self._ptr


@pytest.fixture(autouse=True)
def known_types():
    tp._dtypes()


def described(f, t):
    out = tp.TpTensor(ptr=1, dtype=7, reserved=7, rows=7, cols=7, ld=7)
    ok = f(t, ctypes.addressof(out))
    return (out.ptr, out.dtype, out.reserved, out.rows, out.cols, out.ld) if ok else None


@pytest.mark.parametrize("shape, stride", [((3, 8), (8, 1)), ((3, 8), (24, 1)), ((1, 8), (8, 1)), ((1, 8), (0, 1)),
                                           ((1, 8), (99, 1)), ((5, 1), (7, 1)), ((1, 1), (1, 1)), ((4, 6), (0, 1)),
                                           ((1 << 33, 2), (1 << 40, 1))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float8_e4m3fn])
def test_plain_matrices(shape, stride, dtype):
    t = Fake(shape, stride, dtype, ptr=(1 << 47) + 16)
    assert described(d.matrix, t) == tp._fields(t)


def test_rows():
    assert described(d.row, Fake((12,), (1,), torch.float32)) == (4096, tp.TP_F32, 0, 1, 12, 12)
    for t in (Fake((12,), (2,)), Fake((0,), (1,)), Fake((1, 12), (12, 1)), Fake((), ())):
        assert described(d.row, t) is None


class Raises(Fake):
    def data_ptr(self):
        raise RuntimeError("no storage")


class NotCuda(Fake):
    is_cuda = False


@pytest.mark.parametrize("t", [None, 5, object(), torch.zeros(2, 3), Fake((3, 8), (8, 2)), Fake((0, 8), (8, 1)),
                               Fake((8, 0), (1, 1)), Fake((2, 2, 2), (4, 2, 1)), Fake((3, 8), (8, 1), torch.float16),
                               Fake((3, 8), (8, 1), ptr=0), Fake((3, 8), (8, 1), ptr=-1), Fake((3, 8), (8, 1), ptr="x"),
                               Fake((3, 8), (8,)), Fake((3, 8), [8, 1]), Raises((3, 8), (8, 1)), NotCuda((3, 8), (8, 1)),
                               tp.TpTensor(ptr=16, dtype=tp.TP_BF16, rows=1, cols=8, ld=8)])
def test_the_rest_is_left_to_the_caller(t):
    assert described(d.matrix, t) is None and described(d.row, t) is None  # and nothing is raised


def test_a_vector_is_no_matrix():
    assert described(d.matrix, Fake((3,), (1,))) is None


def test_sequences():
    ts = [Fake((2, 8), (8, 1), ptr=4096 * i) for i in range(1, 5)]
    out = (tp.TpTensor * 4)()
    for seq in (ts, tuple(ts)):
        assert d.matrices(seq, 3, ctypes.addressof(out)) == 3
        assert [t.ptr for t in out] == [4096, 8192, 12288, None]
    assert d.matrices(ts, 9, ctypes.addressof((tp.TpTensor * 9)())) == 4
    assert d.matrices(ts[:2] + [None] + ts[2:], 4, ctypes.addressof(out)) == 2
    assert d.matrices(iter(ts), 3, ctypes.addressof(out)) == 0
    assert d.matrices([], 0, ctypes.addressof(out)) == 0


def test_a_sequence_that_shrinks_while_it_is_read():
    ts = []

    class Clears(Fake):
        def data_ptr(self):
            ts.clear()
            return 64

    ts.extend([Clears((2, 8), (8, 1)) for _ in range(3)])
    assert d.matrices(ts, 3, ctypes.addressof((tp.TpTensor * 3)())) == 1


@pytest.mark.parametrize("call", [lambda: d.matrix(1), lambda: d.matrix(Fake((1, 8), (8, 1)), 0), lambda: d.row(1, "x"),
                                  lambda: d.matrices([], "x", 16), lambda: d.matrices([], 1), lambda: d.dtypes(1)])
def test_wrong_calls(call):
    with pytest.raises((TypeError, ValueError)):
        call()


def test_scratch_mixes_both(monkeypatch):
    descriptor = tp.TpTensor(ptr=16, dtype=tp.TP_F32, rows=2, cols=8, ld=8)
    ts = [Fake((2, 8), (8, 1)), descriptor, Fake((2, 8), (16, 1), torch.float32)]

    def packed():
        s = tp._Scratch(8)
        assert s.one(None) is None and s.row(None) is None
        first = s.many(ts, 3)
        assert first == s.base
        s.one(ts[2])
        s.row(descriptor)
        return bytes(s.buf[:s.used])

    want = packed()
    assert len(want) == 5 * ctypes.sizeof(tp.TpTensor)
    monkeypatch.setattr(tp, "_matrix", lambda t, to: False)
    monkeypatch.setattr(tp, "_row", lambda t, to: False)
    monkeypatch.setattr(tp, "_matrices", lambda seq, n, to: 0)
    assert packed() == want


@pytest.mark.gpu
def test_cuda_tensors():
    from gpu_util import need_gpu
    need_gpu()
    x = torch.zeros(6, 64, device="cuda")
    for t in (x, x[1:, 8:40], x[:1], x[2:3].expand(4, 64), x.to(torch.bfloat16)[:, 3:], x.to(torch.float8_e4m3fn), x.t(), x[:0],
              x.cpu()):
        got = described(d.matrix, t)
        try:
            want = tp._fields(t)
        except (TypeError, ValueError):
            want = None
        assert got == want or (got is None and want[0] == 0), t.shape
    assert described(d.row, x[2]) == (x[2].data_ptr(), tp.TP_F32, 0, 1, 64, 64)


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
