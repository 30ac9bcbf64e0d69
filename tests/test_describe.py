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
