"""Refusals of the calls for long contexts: every case below returns its status before any CUDA
call, so it runs without a GPU."""
import ctypes

import pytest

import tensor_sharded_linear_gqa_gb300 as tp

FAKE = 1 << 40  # never dereferenced: every case fails validation first
BF, F32, E4, U8 = tp.TP_BF16, tp.TP_F32, tp.TP_E4M3, tp.TP_U8
PLAN = tp.tp_plan_create(2, 512, 4, 2, 128, 64)      # two ranks, two q heads and one kv head of 128 each
SHARED = tp.tp_plan_create(4, 512, 8, 2, 64, 64)     # K/V replicated: one source of two heads of 64


def T(dtype, rows, cols, ld=None, ptr=FAKE):
    return tp.TpTensor(ptr, dtype, 0, rows, cols, ld if ld is not None else max(cols, 1))


def arr(*ts):
    a = (tp.TpTensor * len(ts))()
    for i, t in enumerate(ts):
        a[i] = t
    return a


def many(t, n):
    return None if t is None else arr(*[t] * n)


# ---- tp_rotary ---------------------------------------------------------------------
def rotary_status(plan=PLAN, tokens=4, pos=FAKE, axes=1, freq=FAKE, pairs=64, axis=None, layout=0, inverse=0,
                  q=T(BF, 4, 256), k=T(BF, 4, 128), qo=T(BF, 4, 256, ptr=2 * FAKE), ko=T(BF, 4, 128, ptr=3 * FAKE)):
    axis = None if axis is None else (ctypes.c_int32 * len(axis))(*axis)
    return tp.raw_status("tp_rotary", plan.handle if plan else None, tokens, pos, axes, freq, pairs, axis, layout, inverse,
                         many(q, 2), many(k, 2), many(qo, 2), many(ko, 2), None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), "INVALID_ARG"), (dict(tokens=-1), "INVALID_ARG"), (dict(tokens=5), "INVALID_ARG"),
    (dict(pos=None), "INVALID_ARG"), (dict(freq=None), "INVALID_ARG"), (dict(pos=FAKE + 2), "ALIGNMENT"),
    (dict(freq=FAKE + 1), "ALIGNMENT"), (dict(axes=0), "INVALID_ARG"), (dict(axes=9), "UNSUPPORTED"),
    (dict(pairs=0), "INVALID_ARG"), (dict(pairs=65), "INVALID_ARG"), (dict(layout=2), "INVALID_ARG"),
    (dict(pairs=3, axis=[0, 0, 1]), "INVALID_ARG"), (dict(pairs=3, axes=2, axis=[0, -1, 1]), "INVALID_ARG"),
    (dict(q=None, k=None, qo=None, ko=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(ko=None), "INVALID_ARG"),
    (dict(k=T(F32, 4, 128)), "DTYPE"), (dict(qo=T(F32, 4, 256)), "DTYPE"),
    (dict(q=T(E4, 4, 256), k=None, qo=T(E4, 4, 256), ko=None), "DTYPE"), (dict(q=T(U8, 4, 256)), "INVALID_ARG"),
    (dict(q=T(BF, 4, 255)), "INVALID_ARG"), (dict(ko=T(BF, 3, 128)), "INVALID_ARG"), (dict(q=T(BF, 4, 256, ld=255)), "INVALID_ARG"),
    (dict(q=T(BF, 4, 256, ptr=FAKE + 1)), "ALIGNMENT"), (dict(q=T(BF, 4, 256, ptr=None)), "INVALID_ARG"),
])
def test_rotary_refusals(kw, status):
    assert rotary_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_rotary_sizes_and_none():
    wide = tp.tp_plan_create(1, 1024, 1, 1, 1024, 1)
    big = T(BF, 4, 1024)
    assert rotary_status(plan=wide, pairs=257, q=big, qo=big, k=big, ko=big) == tp.TP_ERR_UNSUPPORTED
    # in place with another pitch: a row would meet others
    assert rotary_status(q=T(BF, 4, 256, ld=512), qo=T(BF, 4, 256)) == tp.TP_ERR_INVALID_ARG
    none = T(BF, 0, 256, ptr=None)
    assert rotary_status(tokens=0, pos=None, freq=None, q=none, qo=none, k=None, ko=None) == tp.TP_OK


# ---- tp_window_attn ------------------------------------------------------------------
def window_status(plan=PLAN, t=4, s=40, window=8, sinks=1, q=None, k=None, a=None, v=None, ws=FAKE, size=1 << 40):
    q, a = q or T(BF, t, 256), a or T(BF, t, 256, ptr=2 * FAKE)
    k, v = k or T(BF, s, 128), v or T(BF, s, 128)
    return tp.raw_status("tp_window_attn", plan.handle if plan else None, arr(q, q), arr(k, k), arr(v, v), window, sinks, arr(a, a),
                         ws, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), "INVALID_ARG"), (dict(window=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(sinks=-1), "INVALID_ARG"), (dict(t=5, s=4), "INVALID_ARG"), (dict(q=T(BF, 4, 128)), "INVALID_ARG"),
    (dict(q=T(F32, 4, 256)), "DTYPE"), (dict(a=T(F32, 4, 256)), "DTYPE"), (dict(k=T(E4, 40, 128)), "DTYPE"),
    (dict(v=T(BF, 39, 128)), "INVALID_ARG"), (dict(a=T(BF, 5, 256)), "INVALID_ARG"),
    (dict(k=T(BF, 40, 128, ptr=FAKE + 8)), "ALIGNMENT"), (dict(v=T(BF, 40, 128, ld=132)), "ALIGNMENT"),
    (dict(a=T(BF, 4, 256, ptr=FAKE + 2)), "ALIGNMENT"), (dict(q=T(BF, 4, 256, ptr=None)), "INVALID_ARG"),
    (dict(s=2 ** 31 - 1), "UNSUPPORTED"), (dict(t=2 ** 27, s=2 ** 27), "UNSUPPORTED"),
])
def test_window_refusals(kw, status):
    assert window_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_window_head_sizes_and_no_tokens():
    for hd in (32, 96, 256):
        plan = tp.tp_plan_create(1, hd, 1, 1, hd, 1)
        assert window_status(plan=plan, q=T(BF, 4, hd), a=T(BF, 4, hd), k=T(BF, 4, hd), v=T(BF, 4, hd)) == tp.TP_ERR_UNSUPPORTED
        assert tp.tp_window_attn_workspace_size(plan, 4, 4, 8, 0) == 0
    none = T(BF, 0, 256, ptr=None)
    assert window_status(t=0, q=none, a=none, ws=None, size=0) == tp.TP_OK
    for sizes in ((0, 4, 8, 0), (5, 4, 8, 0), (4, 4, 0, 0), (4, 4, 8, -1), (4, 2 ** 31 - 1, 8, 0)):
        assert tp.tp_window_attn_workspace_size(PLAN, *sizes) == 0


# ---- the 4-bit caches ------------------------------------------------------------------
def cache(plan, batch, cap, kc=None, ks=None, vc=None, vs=None):
    src = 1 if plan.dims.num_kv_heads < plan.dims.tp_size else plan.dims.tp_size
    rows, d = batch * plan.dims.num_kv_heads // src * cap, plan.dims.head_dim
    return [many(x or y, src) for x, y in zip((kc, ks, vc, vs), [T(U8, rows, d // 2), T(BF, rows, d // 32)] * 2)]


def store_status(plan=PLAN, batch=3, cap=10, n=2, lengths=FAKE, counts=None, k=None, v=None, load=False, **kw):
    k, v = k or T(BF, batch * n, 128), v or T(BF, batch * n, 128)
    c = cache(plan or PLAN, batch, cap, **kw)
    h = plan.handle if plan else None
    if load:
        return tp.raw_status("tp_cache4_load", h, batch, lengths, *c, arr(k, k), arr(v, v), None)
    return tp.raw_status("tp_cache4_store", h, batch, lengths, counts, arr(k, k), arr(v, v), *c, None)


@pytest.mark.parametrize("load", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(batch=2 ** 31), "INVALID_ARG"),
    (dict(lengths=None), "INVALID_ARG"), (dict(lengths=FAKE + 2), "ALIGNMENT"),
    (dict(k=T(BF, 7, 128)), "INVALID_ARG"), (dict(v=T(BF, 3, 128)), "INVALID_ARG"), (dict(k=T(BF, 6, 64)), "INVALID_ARG"),
    (dict(k=T(E4, 6, 128)), "DTYPE"), (dict(v=T(F32, 6, 128)), "DTYPE"), (dict(v=T(BF, 6, 128, ld=129)), "ALIGNMENT"),
    (dict(k=T(BF, 6, 128, ptr=FAKE + 4)), "ALIGNMENT"), (dict(k=T(BF, 6, 128, ptr=None)), "INVALID_ARG"),
    (dict(kc=T(U8, 31, 64)), "INVALID_ARG"), (dict(kc=T(U8, 30, 64, ld=80)), "INVALID_ARG"), (dict(kc=T(BF, 30, 64)), "DTYPE"),
    (dict(ks=T(F32, 30, 4)), "DTYPE"), (dict(ks=T(BF, 30, 8)), "INVALID_ARG"), (dict(vc=T(U8, 30, 128)), "INVALID_ARG"),
    (dict(vs=T(BF, 27, 4)), "INVALID_ARG"), (dict(vc=T(U8, 30, 64, ptr=FAKE + 8)), "ALIGNMENT"),
    (dict(vs=T(BF, 30, 4, ptr=FAKE + 4)), "ALIGNMENT"), (dict(ks=T(BF, 30, 4, ptr=None)), "INVALID_ARG"),
])
def test_store_and_load_refusals(kw, status, load):
    assert store_status(load=load, **kw) == getattr(tp, "TP_ERR_" + status)


def test_store_takes_bf16_and_aligned_counts():
    f = T(F32, 6, 128)
    assert store_status(k=f, v=f) == tp.TP_ERR_DTYPE
    assert store_status(counts=FAKE + 2) == tp.TP_ERR_ALIGNMENT
    none = T(BF, 0, 128, ptr=None)
    assert store_status(n=0, k=none, v=none, lengths=None) == tp.TP_OK and store_status(n=0, k=none, v=none, load=True) == tp.TP_OK
    assert store_status(batch=0, k=none, v=none, kc=T(U8, 0, 64, ptr=None)) == tp.TP_OK


def attn_status(plan=PLAN, batch=3, cap=10, q=None, a=None, lengths=FAKE, window=4, sinks=1, ws=FAKE, size=1 << 40, **kw):
    q, a = q or T(BF, batch, 256), a or T(BF, batch, 256, ptr=2 * FAKE)
    return tp.raw_status("tp_cache4_attn", plan.handle if plan else None, batch, many(q, 4), *cache(plan or PLAN, batch, cap, **kw),
                         lengths, window, sinks, many(a, 4), ws, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(lengths=None), "INVALID_ARG"),
    (dict(lengths=FAKE + 2), "ALIGNMENT"), (dict(window=0), "INVALID_ARG"), (dict(sinks=-2), "INVALID_ARG"),
    (dict(q=T(BF, 3, 128)), "INVALID_ARG"), (dict(q=T(F32, 3, 256)), "DTYPE"), (dict(a=T(BF, 4, 256)), "INVALID_ARG"),
    (dict(a=T(F32, 3, 256)), "DTYPE"), (dict(a=T(BF, 3, 256, ptr=FAKE + 8)), "ALIGNMENT"), (dict(q=T(BF, 3, 256, ld=260)), "ALIGNMENT"),
    (dict(kc=T(U8, 29, 64)), "INVALID_ARG"), (dict(vs=T(BF, 30, 2)), "INVALID_ARG"), (dict(vc=T(E4, 30, 64)), "DTYPE"),
    (dict(plan=SHARED), "INVALID_ARG"), (dict(batch=2 ** 23, cap=1), "UNSUPPORTED"),
])
def test_attn_refusals(kw, status):
    assert attn_status(**kw) == getattr(tp, "TP_ERR_" + status)


def test_attn_replicated_heads_sizes_and_no_sequences():
    q = T(BF, 3, 128)
    assert attn_status(plan=SHARED, q=q, a=T(BF, 3, 128, ld=132)) == tp.TP_ERR_ALIGNMENT  # its caches are taken
    odd = tp.tp_plan_create(1, 96, 1, 1, 96, 1)
    assert attn_status(plan=odd) == tp.TP_ERR_UNSUPPORTED and tp.tp_cache4_attn_workspace_size(odd, 1, 4, 8, 0) == 0
    none = T(BF, 0, 256, ptr=None)
    assert attn_status(batch=0, q=none, a=none, lengths=None, ws=None, size=0) == tp.TP_OK
    for sizes in ((0, 4, 8, 0), (4, 0, 8, 0), (4, 4, 0, 0), (4, 4, 8, -1), (-1, 4, 8, 0)):
        assert tp.tp_cache4_attn_workspace_size(PLAN, *sizes) == 0


def test_a_failed_rank_stops_every_call():
    tp.tp_set_rank_health(1, False)
    try:
        assert rotary_status() == window_status() == store_status() == store_status(load=True) == attn_status() == tp.TP_ERR_RANK_FAILED
    finally:
        tp.tp_set_rank_health(1, True)


# ---- the binding's own checks ------------------------------------------------------------
torch = pytest.importorskip("torch")


class FakeTensor:
    """What the binding reads of a CUDA vector."""

    def __init__(self, *shape, dtype=torch.int32, cuda=True, contiguous=True):
        self.shape, self.dtype, self.is_cuda, self._contiguous = shape, dtype, cuda, contiguous

    def is_contiguous(self):
        return self._contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def element_size(self):
        return 4

    def data_ptr(self):
        return FAKE


def test_binding_checks_bare_addresses():
    f = FakeTensor(64, dtype=torch.float32)
    q = [T(BF, 4, 256)] * 2

    def rotary(pos=FakeTensor(1, 4), freq=f, axis=None, q=q):
        tp.tp_rotary(PLAN, pos, freq, q, None, q, None, axis=axis, stream=1)

    for bad in (lambda: rotary(pos=FakeTensor(1, 1, 4)), lambda: rotary(axis=[0] * 63), lambda: rotary(axis=tp.rotary_axes([1, 2])),
                lambda: rotary(axis=(ctypes.c_float * 64)()), lambda: rotary(q=q[:1]), lambda: rotary(pos=FakeTensor(4, cuda=False))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: rotary(pos=FakeTensor(4, dtype=torch.int64)), lambda: rotary(freq=FakeTensor(64, dtype=torch.float64)),
                lambda: rotary(pos=FakeTensor(4, contiguous=False))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(tp.TPError):
        rotary(pos=FakeTensor(2, 5), axis=tp.rotary_axes([32, 32]))  # q has four tokens
    assert list(tp.rotary_axes([2, 1, 3])) == [0, 0, 1, 2, 2, 2]

    k = [T(BF, 40, 128)] * 2
    for ws in (FakeTensor(9, cuda=False), FakeTensor(9, contiguous=False)):
        with pytest.raises(ValueError):
            tp.tp_window_attn(PLAN, q, k, k, 8, 0, q, ws, stream=1)
        with pytest.raises(ValueError):
            tp.tp_cache4_attn(PLAN, q, k, k, k, k, FakeTensor(3), 8, 0, q, ws, stream=1)
    with pytest.raises(tp.TPError):
        tp.tp_window_attn(PLAN, q, k, k, 0, 0, q, None, stream=1)
    with pytest.raises(ValueError):
        tp.tp_cache4_store(PLAN, FakeTensor(3), q, q, k, k, k, k, counts=FakeTensor(2), stream=1)
    with pytest.raises(TypeError):
        tp.tp_cache4_load(PLAN, FakeTensor(3, dtype=torch.int64), k, k, k, k, q, q, stream=1)


def test_binding_refuses_another_device(monkeypatch):
    """With several GPUs (pretended here) each tensor of a call lies on the current one."""
    monkeypatch.setattr(tp, "_devices", 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here, there = FakeTensor(3), FakeTensor(3)
    here.device, there.device = torch.device("cuda", 0), torch.device("cuda", 1)
    q, k = [T(BF, 3, 256)] * 2, [T(BF, 40, 128)] * 2
    cache = (k, k, k, k)
    calls = [lambda x: tp.tp_rotary(PLAN, x, FakeTensor(64, dtype=torch.float32), q, None, q, None, stream=1),
             lambda x: tp.tp_rotary(PLAN, FakeTensor(3), FakeTensor(64, dtype=torch.float32), [x, x], None, q, None, stream=1),
             lambda x: tp.tp_window_attn(PLAN, q, k, k, 8, 0, q, x, stream=1),
             lambda x: tp.tp_cache4_store(PLAN, x, k, k, *cache, stream=1),
             lambda x: tp.tp_cache4_store(PLAN, here, k, k, *cache, counts=x, stream=1),
             lambda x: tp.tp_cache4_load(PLAN, x, *cache, k, k, stream=1),
             lambda x: tp.tp_cache4_attn(PLAN, q, *cache, x, 8, 0, q, None, stream=1)]
    for call in calls:
        with pytest.raises(ValueError, match="cuda:1"):
            call(there)
    for call in calls[3:]:  # the current device: on to the library's own refusals (k has the wrong type)
        with pytest.raises(tp.TPError):
            call(here)
