"""The long-context calls with several GPUs (pretended where there is one): every tensor lies on the current one, descriptors that
were packed before among them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from test_long_context_cpu import BF, PLAN, FakeTensor, T

FAKE = 1 << 40


class Matrix:
    """What the binding reads of a 2-D CUDA tensor."""
    is_cuda, dtype = True, torch.bfloat16

    def __init__(self, rows, cols, index):
        self.shape, self.device = torch.Size((rows, cols)), torch.device("cuda", index)

    def stride(self):
        return self.shape[1], 1

    def data_ptr(self):
        return FAKE


def pretend(monkeypatch, now=0):
    monkeypatch.setattr(tp, "_devices", 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now)


def test_packed_descriptors_remember_their_gpu(monkeypatch):
    pretend(monkeypatch)
    q, k = [T(BF, 4, 256)] * 2, [T(BF, 40, 128)] * 2
    window = lambda k: tp.tp_window_attn(PLAN, q, k, k, 0, 0, q, None, stream=1)  # noqa: E731  a window of 0 is refused by the library
    here, there = Matrix(40, 128, 0), Matrix(40, 128, 1)
    for bad in (tp.arr([there, there]), tp.arr(x for x in (here, there)), [here, tp.tensor(there)], tp.arr([tp.tensor(there)] * 2),
                [there, there], (here, there), tp.arr(tp.arr([here, there]))):
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            window(bad)
    for good in (tp.arr([here, here]), [tp.tensor(here)] * 2, k, tp.arr(k), (tp.TpTensor * 2)(*k), [here, here]):
        with pytest.raises(tp.TPError):
            window(good)
    pretend(monkeypatch, 1)
    with pytest.raises(tp.TPError):
        window(tp.arr([there, there]))
    monkeypatch.setattr(tp, "_devices", 1)  # one GPU: nothing is asked
    with pytest.raises(tp.TPError):
        window(tp.arr([here, there]))


def test_packing_is_as_before():
    m = Matrix(3, 8, 1)
    assert bytes(tp.arr([m])) == bytes(tp.tensor(m)) == bytes(tp.TpTensor(FAKE, BF, 0, 3, 8, 8))
    assert tp.tensor(m).device == 1 and tp.arr([m, T(BF, 1, 8)]).devices == {1} and tp.arr([T(BF, 1, 8)]).devices == frozenset()
    t = T(BF, 1, 8)
    assert tp.tensor(t) is t and len(tp.arr([])) == 1  # an array of nothing has an entry that is not read


@pytest.mark.skipif(tp._describe is None, reason="the extension module is not built")
def test_devices_that_are_no_numbers():
    d = tp._load_describe()
    out = tp.TpTensor()
    at = ctypes.addressof(out)
    f = FakeTensor(3)
    for call in (lambda: d.matrix(f, at, "x"), lambda: d.matrices([f], 1, at, None), lambda: d.vector(f, 4, 3, 0.5), lambda: d.bytes(f, "x"),
                 lambda: d.matrix(f, at, 0, 0), lambda: d.matrices([], 0, at, 0, 0), lambda: d.vector(f, 4, 3, 0, 0), lambda: d.bytes(f, 0, 0)):
        with pytest.raises(TypeError):
            call()
    # a stand-in is left to interpreted code where a device is asked for
    m = Matrix(3, 8, 0)
    assert d.matrix(m, at) and not d.matrix(m, at, 0) and d.matrices([m], 1, at, 0) == 0 and d.matrices([m], 1, at) == 1


@pytest.mark.gpu
def test_cuda_tensors(monkeypatch):
    """Real tensors of the current GPU pass; with another one pretended to be current each is refused."""
    from gpu_util import need_gpu
    need_gpu()
    now = torch.cuda.current_device()
    plan = tp.tp_plan_create(1, 512, 4, 2, 128, 1)
    new = lambda rows, cols, dtype=torch.bfloat16: torch.zeros(rows, cols, dtype=dtype, device="cuda")  # noqa: E731
    q, k, a, out = new(4, 512), new(9, 256), new(4, 512), new(4, 256)
    cache = [new(4 * 2 * 9, 64, torch.uint8), new(4 * 2 * 9, 4), new(4 * 2 * 9, 64, torch.uint8), new(4 * 2 * 9, 4)]
    ints, ws = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    freq, odd = torch.ones(64, device="cuda"), "cuda:%d" % now
    kv = new(4, 256)

    def calls(pack):
        c = [pack([t]) for t in cache]
        return [lambda: tp.tp_rotary(plan, ints, freq, pack([q]), pack([kv]), pack([a]), pack([out])),
                lambda: tp.tp_window_attn(plan, pack([q]), pack([k]), pack([k]), 3, 1, pack([a]), ws),
                lambda: tp.tp_cache4_store(plan, ints, pack([kv]), pack([kv]), *c, counts=ints),
                lambda: tp.tp_cache4_load(plan, ints, *c, pack([out]), pack([kv])),
                lambda: tp.tp_cache4_attn(plan, pack([q]), *c, ints, 3, 1, pack([a]), ws)]

    monkeypatch.setattr(tp, "_devices", 2)
    for pack in (list, tp.arr, lambda ts: [tp.tensor(t) for t in ts]):
        for call in calls(pack):
            call()
    torch.cuda.synchronize()
    assert tp.tp_device_status()[0] == tp.TP_OK
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now + 1)
    for pack in (list, tp.arr, lambda ts: [tp.tensor(t) for t in ts]):
        for call in calls(pack):
            with pytest.raises(ValueError, match=odd):
                call()
    # one tensor of a call alone
    for call in (lambda: tp._dev_ptr(ints, "torch.int32", device=now + 1), lambda: tp._workspace(ws, now + 1),
                 lambda: tp._args(1, now + 1).one(q), lambda: tp._args(2, now + 1).many([q, a], 2)):
        with pytest.raises(ValueError, match=odd):
            call()
    assert tp._dev_ptr(ints, "torch.int32", device=now) == ints.data_ptr() and tp._workspace(ws, now) == (ws.data_ptr(), 1 << 20)
