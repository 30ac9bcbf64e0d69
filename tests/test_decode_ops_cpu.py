"""Refusals of the operators between the projections: every case below returns its status
before any CUDA call, so it runs without a GPU."""
import ctypes

import pytest

import tensor_sharded_linear_gqa_gb300 as tp

FAKE = 1 << 40  # never dereferenced: every case fails validation first
BF, F32, E4 = tp.TP_BF16, tp.TP_F32, tp.TP_E4M3


def T(dtype, rows, cols, ld=None, ptr=FAKE):
    return tp.TpTensor(ptr, dtype, 0, rows, cols, ld if ld is not None else max(cols, 1))


def arr(*ts):
    a = (tp.TpTensor * len(ts))()
    for i, t in enumerate(ts):
        a[i] = t
    return a


def ref(t):
    return None if t is None else ctypes.byref(t)


# ---- tp_add_rmsnorm --------------------------------------------------------------
def norm_status(n=1, x=None, res=None, w=T(F32, 1, 64), eps=1e-5, res_out=None, y=T(BF, 4, 64), scale=None):
    x = x if x is not None else [T(F32, 4, 64)] * n
    return tp.raw_status("tp_add_rmsnorm", n, arr(*x), ref(res), ref(w), eps, ref(res_out), ref(y), scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0, x=[T(F32, 4, 64)]), "INVALID_ARG"),
    (dict(n=65, x=[T(F32, 4, 64)]), "INVALID_ARG"),
    (dict(eps=0.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(w=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"),
    (dict(w=T(F32, 1, 63)), "INVALID_ARG"), (dict(w=T(F32, 2, 64)), "INVALID_ARG"), (dict(w=T(E4, 1, 64)), "DTYPE"),
    (dict(y=T(BF, 5, 64)), "INVALID_ARG"), (dict(y=T(F32, 4, 64)), "DTYPE"), (dict(y=T(BF, 4, 64, ptr=None)), "INVALID_ARG"),
    (dict(y=T(E4, 4, 64)), "INVALID_ARG"),                     # 8-bit output without scales
    (dict(scale=FAKE), "INVALID_ARG"),                         # scales without an 8-bit output
    (dict(y=T(E4, 4, 64), scale=FAKE + 2), "ALIGNMENT"),
    (dict(res_out=T(F32, 4, 64)), "INVALID_ARG"),              # nothing to write it from
    (dict(res=T(F32, 4, 64), res_out=T(BF, 4, 64)), "DTYPE"),
    (dict(res=T(E4, 4, 64)), "DTYPE"), (dict(res=T(F32, 3, 64)), "INVALID_ARG"),
    (dict(n=2, x=[T(F32, 4, 64), T(BF, 4, 64)]), "DTYPE"),
    (dict(n=2, x=[T(F32, 4, 64), T(F32, 4, 65)]), "INVALID_ARG"),
    (dict(x=[T(E4, 4, 64)]), "DTYPE"), (dict(x=[T(F32, 4, 64, ld=63)]), "INVALID_ARG"),
    (dict(x=[T(F32, 4, 64, ptr=FAKE + 2)]), "ALIGNMENT"), (dict(x=[T(7, 4, 64)]), "INVALID_ARG"),
    (dict(x=[T(F32, -1, 64)]), "INVALID_ARG"),
])
def test_norm_refusals(kw, status):
    assert norm_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_norm_empty_and_failed_rank():
    assert norm_status(x=[T(F32, 0, 64, ptr=None)], y=T(BF, 0, 64, ptr=None)) == tp.TP_OK
    tp.tp_set_rank_health(1, False)
    try:
        assert norm_status(n=2) == tp.TP_ERR_RANK_FAILED
    finally:
        tp.tp_set_rank_health(1, True)


def test_other_calls_do_not_take_8_bit_operands():
    a = arr(T(E4, 4, 64))
    assert tp.raw_status("tp_column_linear", 1, a, arr(T(E4, 8, 64)), arr(T(BF, 4, 8)), 0, None) == tp.TP_ERR_INVALID_ARG
    assert tp.raw_status("tp_row_linear", 1, a, arr(T(E4, 8, 64)), arr(T(F32, 4, 8)), 0, None) == tp.TP_ERR_INVALID_ARG


# ---- tp_cache_evict ----------------------------------------------------------------
PLAN = tp.tp_plan_create(2, 512, 4, 2, 128, 64)  # two ranks, one kv head of 128 each


def evict_status(plan=PLAN, batch=2, lengths=FAKE, rows=40, rows_out=20, cols=128, kd=BF, wd=F32, w_cols=20, wo_cols=10,
                 budget=10, first=1, recent=2, lengths_out=FAKE, kept=FAKE, ld=None, k_out_ptr=2 * FAKE, v_out_ptr=3 * FAKE,
                 k_ptr=FAKE, v_ptr=FAKE, w_rows=2):
    k, v = [T(kd, rows, cols, ld, k_ptr)] * 2, [T(kd, rows, cols, ld, v_ptr)] * 2
    ko, vo = [T(kd, rows_out, cols, ld, k_out_ptr)] * 2, [T(kd, rows_out, cols, ld, v_out_ptr)] * 2
    w, wo = [T(wd, w_rows, w_cols)] * 2, [T(wd, w_rows, wo_cols, None, 4 * FAKE)] * 2
    return tp.raw_status("tp_cache_evict", plan.handle if plan else None, batch, lengths, arr(*k), arr(*v), arr(*w), budget,
                         first, recent, arr(*ko), arr(*vo), arr(*wo), lengths_out, kept, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(lengths=None), "INVALID_ARG"),
    (dict(lengths_out=None), "INVALID_ARG"), (dict(kept=None), "INVALID_ARG"), (dict(kept=FAKE + 2), "ALIGNMENT"),
    (dict(lengths=FAKE + 1), "ALIGNMENT"), (dict(budget=0), "INVALID_ARG"), (dict(first=-1), "INVALID_ARG"),
    (dict(recent=-1), "INVALID_ARG"), (dict(first=9, recent=2), "INVALID_ARG"), (dict(rows=41), "INVALID_ARG"),
    (dict(rows_out=18), "INVALID_ARG"),                   # nine rows a sequence for a budget of ten
    (dict(cols=64), "INVALID_ARG"), (dict(kd=F32), "DTYPE"), (dict(wd=BF), "DTYPE"), (dict(w_cols=19), "INVALID_ARG"),
    (dict(wo_cols=9), "INVALID_ARG"), (dict(ld=132), "ALIGNMENT"), (dict(w_rows=3), "INVALID_ARG"),
    (dict(k_out_ptr=FAKE), "INVALID_ARG"),                # K onto itself with another capacity
    (dict(k_out_ptr=FAKE, rows_out=40), "INVALID_ARG"),   # K in place, V not
    (dict(k_ptr=FAKE + 8), "ALIGNMENT"),
])
def test_evict_refusals(kw, status):
    assert evict_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_evict_unsupported_and_empty():
    odd = tp.tp_plan_create(1, 60, 1, 1, 60, 4)  # a head of 120 bytes
    assert evict_status(plan=odd, cols=60) == tp.TP_ERR_UNSUPPORTED
    assert evict_status(batch=0, rows=0, rows_out=0, w_rows=0, w_cols=0, wo_cols=0) == tp.TP_OK


def test_binding_counts_its_per_rank_arguments():
    with pytest.raises(ValueError):
        tp.tp_linear_epilogue(2, tp.TP_SHARD_COLUMN, [T(BF, 4, 64)], [T(BF, 8, 64)], T(BF, 4, 16))
    with pytest.raises(ValueError):
        tp.tp_linear_epilogue(2, tp.TP_SHARD_ROW, arr(T(BF, 4, 64)), arr(*[T(BF, 8, 64)] * 2), T(BF, 4, 8), stream=1)
    with pytest.raises(tp.TPError):  # enough of them, and the library refuses the shapes
        tp.tp_linear_epilogue(2, tp.TP_SHARD_COLUMN, [T(BF, 4, 64)], [T(BF, 8, 64)] * 2, T(BF, 4, 17), stream=1)
    many = [T(BF, 4, 64)] * 400  # more than the scratch holds at first
    with pytest.raises(tp.TPError):
        tp.tp_add_rmsnorm(many, None, T(BF, 1, 64), 1e-5, None, T(BF, 4, 64), stream=1)


# ---- tp_linear_epilogue ------------------------------------------------------------
def linear_status(n=1, shard=tp.TP_SHARD_COLUMN, x=None, xs=None, w=None, ws=None, bias=None, act=0, res=None, y=T(BF, 4, 96)):
    x = x or [T(BF, 4, 64)]
    w = w or [T(BF, 96 // n, 64)] * n
    return tp.raw_status("tp_linear_epilogue", n, shard, arr(*x), xs, arr(*w), ws, ref(bias), act, ref(res), ref(y), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=3), "TP_SIZE_NOT_POW2"), (dict(n=0, w=[T(BF, 96, 64)]), "INVALID_ARG"), (dict(shard=tp.TP_SHARD_VOCAB), "INVALID_ARG"),
    (dict(act=4), "INVALID_ARG"), (dict(act=-1), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"),
    (dict(y=T(BF, 4, 95)), "INVALID_ARG"), (dict(y=T(BF, 5, 96)), "INVALID_ARG"), (dict(y=T(E4, 4, 96)), "DTYPE"),
    (dict(x=[T(F32, 4, 64)], w=[T(F32, 96, 64)]), "DTYPE"), (dict(x=[T(E4, 4, 64)], xs=FAKE, ws=FAKE), "DTYPE"),
    (dict(w=[T(BF, 96, 63)]), "INVALID_ARG"), (dict(x=[T(BF, 4, 64, ptr=FAKE + 2)]), "ALIGNMENT"),
    (dict(x=[T(BF, 4, 60)], w=[T(BF, 96, 60, 64)]), "ALIGNMENT"), (dict(y=T(BF, 4, 96, 97)), "ALIGNMENT"),
    (dict(x=[T(E4, 4, 64)], w=[T(E4, 96, 64)]), "INVALID_ARG"),                    # 8 bits without scales
    (dict(x=[T(E4, 4, 64)], w=[T(E4, 96, 64)], xs=FAKE), "INVALID_ARG"),
    (dict(xs=FAKE), "INVALID_ARG"), (dict(ws=FAKE), "INVALID_ARG"),                # scales without 8 bits
    (dict(x=[T(E4, 4, 64)], w=[T(E4, 96, 64)], xs=FAKE + 2, ws=FAKE), "ALIGNMENT"),
    (dict(bias=T(F32, 1, 95)), "INVALID_ARG"), (dict(bias=T(E4, 1, 96)), "DTYPE"), (dict(bias=T(F32, 1, 96, ptr=FAKE + 1)), "ALIGNMENT"),
    (dict(res=T(F32, 4, 95)), "INVALID_ARG"), (dict(res=T(E4, 4, 96)), "DTYPE"), (dict(res=T(F32, 4, 96, ptr=FAKE + 4)), "ALIGNMENT"),
    (dict(n=2, w=[T(BF, 44, 64), T(BF, 52, 64)]), "ALIGNMENT"),                    # the second shard's columns at 88 bytes
    (dict(n=2, shard=tp.TP_SHARD_ROW, x=[T(BF, 4, 64), T(BF, 4, 64)], w=[T(BF, 96, 64), T(BF, 95, 64)]), "INVALID_ARG"),
    (dict(n=2, shard=tp.TP_SHARD_ROW, x=[T(BF, 4, 64), T(BF, 3, 64)], w=[T(BF, 96, 64)] * 2), "INVALID_ARG"),
    (dict(x=[T(BF, 4, 0)], w=[T(BF, 96, 0)]), "UNSUPPORTED"),                      # no input features
    (dict(n=32, x=[T(BF, 4, 64)], w=[T(BF, 8, 64)] * 32, y=T(BF, 4, 256)), "UNSUPPORTED"),  # 32 weights lying apart
])
def test_linear_refusals(kw, status):
    assert linear_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_linear_empty():
    assert linear_status(x=[T(BF, 0, 64, ptr=None)], y=T(BF, 0, 96, ptr=None)) == tp.TP_OK
    assert linear_status(w=[T(BF, 0, 64, ptr=None)], y=T(BF, 4, 0, ptr=None)) == tp.TP_OK


# ---- tp_prefix_attn ------------------------------------------------------------------
def attn_status(plan=PLAN, batch=3, q=None, kp=None, ko=None, vp=None, vo=None, lengths=FAKE, wi=None, wo=None, a=None, ws=FAKE,
                ws_bytes=1 << 40):
    q, a = q or T(BF, 3, 256), a or T(BF, 3, 256)
    kp, ko = kp or T(BF, 50, 128), ko or T(BF, 30, 128)
    vp, vo = vp or kp, vo or ko
    two = lambda t: None if t is None else arr(t, t)  # noqa: E731
    return tp.raw_status("tp_prefix_attn", plan.handle if plan else None, batch, two(q), two(kp), two(vp), two(ko), two(vo),
                         lengths, two(wi), two(wo), two(a), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(lengths=None), "INVALID_ARG"),
    (dict(lengths=FAKE + 1), "ALIGNMENT"), (dict(q=T(BF, 4, 256)), "INVALID_ARG"), (dict(q=T(BF, 3, 128)), "INVALID_ARG"),
    (dict(q=T(F32, 3, 256)), "DTYPE"), (dict(a=T(F32, 3, 256)), "DTYPE"), (dict(a=T(BF, 3, 256, 257)), "ALIGNMENT"),
    (dict(q=T(BF, 3, 256, ptr=FAKE + 2)), "ALIGNMENT"), (dict(kp=T(BF, 50, 64)), "INVALID_ARG"),
    (dict(vp=T(BF, 49, 128)), "INVALID_ARG"), (dict(ko=T(BF, 31, 128)), "INVALID_ARG"), (dict(vo=T(BF, 33, 128)), "INVALID_ARG"),
    (dict(kp=T(E4, 50, 128)), "DTYPE"), (dict(ko=T(BF, 30, 128, 130)), "ALIGNMENT"),
    (dict(wo=T(F32, 3, 9)), "INVALID_ARG"), (dict(wo=T(F32, 4, 10)), "INVALID_ARG"), (dict(wo=T(BF, 3, 10)), "DTYPE"),
    (dict(wi=T(F32, 3, 10)), "INVALID_ARG"),                       # weights in, none out
    (dict(wi=T(F32, 3, 10, ptr=FAKE + 2), wo=T(F32, 3, 10)), "ALIGNMENT"),
    (dict(ws=None), "WORKSPACE"), (dict(ws_bytes=1000), "WORKSPACE"), (dict(ws=FAKE + 8), "ALIGNMENT"),
])
def test_attn_refusals(kw, status):
    assert attn_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_attn_unsupported_empty_and_workspace():
    odd = tp.tp_plan_create(2, 512, 4, 2, 96, 64)
    assert attn_status(plan=odd, q=T(BF, 3, 192), a=T(BF, 3, 192), kp=T(BF, 50, 96), ko=T(BF, 30, 96)) == tp.TP_ERR_UNSUPPORTED
    assert attn_status(batch=0, q=T(BF, 0, 256), a=T(BF, 0, 256), ko=T(BF, 0, 128)) == tp.TP_OK
    size = tp.tp_prefix_attn_workspace_size
    assert size(PLAN, 0, 100, 100, True) == 0 and size(PLAN, 4, -1, 0, False) == 0 and size(PLAN, 4, 0, 0, True) == 0
    assert size(PLAN, 4, 0, 100, True) - size(PLAN, 4, 0, 100, False) == 4 * 4 * 100 * 4  # four q heads' scores, a multiple of 256
    assert attn_status(ws_bytes=size(PLAN, 3, 50, 10, False) - 1) == tp.TP_ERR_WORKSPACE
    assert size(PLAN, 1 << 40, 1, 1, False) == 0
    assert attn_status(batch=1 << 40, q=T(BF, 1 << 30, 256)) == tp.TP_ERR_INVALID_ARG


# ---- the binding's own checks: what the library sees as bare addresses ------------------
class FakeTensor:
    """What the binding reads of a torch tensor on the GPU."""

    def __init__(self, n, dtype="float32", cuda=True, contiguous=True):
        import torch
        self.n, self.dtype, self.is_cuda, self.contiguous = n, getattr(torch, dtype), cuda, contiguous

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return FAKE


@pytest.fixture
def no_library(monkeypatch):
    class Unreachable:
        def __getattr__(self, name):
            def entry(*args):
                raise AssertionError(f"{name} was called")
            return entry

    monkeypatch.setattr(tp, "_lib", Unreachable())
    return PLAN


def e4m3_norm(scale):
    tp.tp_add_rmsnorm(T(F32, 4, 64), None, T(F32, 1, 64), 1e-5, None, T(E4, 4, 64), scale, stream=1)


def e4m3_linear(xs, ws):
    tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, [T(E4, 4, 64)], [T(E4, 96, 64)], T(BF, 4, 96), x_scale=xs, w_scale=ws, stream=1)


@pytest.mark.parametrize("n", [0, 1, 3, 5])
def test_scales_have_one_entry_a_token_or_feature(no_library, n):
    pytest.importorskip("torch")
    with pytest.raises(ValueError, match="y_scale"):
        e4m3_norm(FakeTensor(n))
    with pytest.raises(ValueError, match="x_scale"):
        e4m3_linear(FakeTensor(n), FakeTensor(96))
    with pytest.raises(ValueError, match="w_scale"):
        e4m3_linear(FakeTensor(4), FakeTensor(n))


def attn(plan, lengths, ws):
    q, kp, ko = [T(BF, 3, 256)] * 2, [T(BF, 50, 128)] * 2, [T(BF, 30, 128)] * 2
    tp.tp_prefix_attn(plan, q, kp, kp, ko, ko, lengths, q, ws, stream=1)


def evict(plan, lengths, lengths_out, kept):
    k, w = [T(BF, 30, 128)] * 2, [T(F32, 3, 10)] * 2
    tp.tp_cache_evict(plan, lengths, k, k, w, 5, 1, 1, k, k, w, lengths_out, kept, stream=1)


def test_addresses_must_be_the_gpus(no_library):
    pytest.importorskip("torch")
    f, i = lambda n: FakeTensor(n), lambda n: FakeTensor(n, "int32")  # noqa: E731
    host = {"float32": lambda n: FakeTensor(n, cuda=False), "int32": lambda n: FakeTensor(n, "int32", cuda=False)}
    calls = [lambda: e4m3_norm(host["float32"](4)), lambda: e4m3_linear(host["float32"](4), f(96)),
             lambda: e4m3_linear(f(4), host["float32"](96)),
             lambda: attn(no_library, host["int32"](3), FakeTensor(1 << 30, "uint8")),
             lambda: attn(no_library, i(3), FakeTensor(1 << 30, "uint8", cuda=False)),
             lambda: attn(no_library, i(3), FakeTensor(1 << 30, "uint8", contiguous=False)),  # an expanded byte, say
             lambda: evict(no_library, host["int32"](3), i(3), i(30)), lambda: evict(no_library, i(3), host["int32"](3), i(30)),
             lambda: evict(no_library, i(3), i(3), host["int32"](30))]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_right_sizes_reach_the_library(no_library):
    pytest.importorskip("torch")
    i = lambda n: FakeTensor(n, "int32")  # noqa: E731
    for call in (lambda: e4m3_norm(FakeTensor(4)), lambda: e4m3_linear(FakeTensor(4), FakeTensor(96)),
                 lambda: attn(no_library, i(3), FakeTensor(1 << 30, "uint8")), lambda: evict(no_library, i(3), i(3), i(30))):
        with pytest.raises(AssertionError, match="was called"):
            call()


def test_attn_workspace_size_of_unsupported_sizes():
    size = tp.tp_prefix_attn_workspace_size
    plans = {"d 96": tp.tp_plan_create(2, 512, 4, 2, 96, 64), "64 ranks": tp.tp_plan_create(64, 64, 64, 64, 64, 64),
             "257 heads a group": tp.tp_plan_create(1, 64, 257, 1, 64, 64)}
    for name, plan in plans.items():
        assert size(plan, 2, 100, 10, False) == 0, name
    assert size(PLAN, 1, 100, 4194240, False) > 0 and size(PLAN, 1, 100, 4194241, False) == 0
    assert size(PLAN, 1, (1 << 31) - 257, 0, False) > 0 and size(PLAN, 1, (1 << 31) - 256, 0, False) == 0
    assert size(PLAN, 8388607 // 4, 100, 0, False) > 0 and size(PLAN, 8388607 // 4 + 1, 100, 0, False) == 0


def test_the_example_refuses_a_step_on_full_caches():
    pytest.importorskip("torch")
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step_cpu", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layer = m.Layer.__new__(m.Layer)  # no weights: the refusal comes first
    layer.longest = layer.capacity = 12
    with pytest.raises(RuntimeError, match="full"):
        layer.step(None)
