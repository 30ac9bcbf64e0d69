"""tp_rotary against the rotation in float64.

Tolerance, from the roundings the call makes (u = 2^-24): the turn is a 64-bit fraction whose upper 32
bits are rounded to f32 (at most 2^-25 of half a turn: pi 2^-25 of angle, and pi 2^-31 from the bits below);
freq / (2 pi) is off by 2^-52 of itself, so a position's angle by 2^-52 of the whole angle; the sine and
cosine add at most 2^-23. A rotated value is two products and a sum in f32 (3u of |a| + |b|) and one rounding to the
output's type."""
import math

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def reference(x, pos, freq, axis, d, layout, inverse=False):
    """(rotated, tolerance) in float64 of x [T x heads*d]."""
    pairs = freq.numel()
    angle = pos.double()[torch.tensor(axis, device="cuda")].t() * freq.double()
    slack = math.pi * (2.0 ** -25 + 2.0 ** -31) + 2.0 ** -23 + 2.0 ** -52 * angle.abs() + 3 * 2.0 ** -24
    c, s = torch.cos(angle)[:, None], (-1 if inverse else 1) * torch.sin(angle)[:, None]
    y = x.double().view(x.shape[0], -1, d).clone()
    one = slice(0, pairs) if layout == tp.TP_ROTARY_HALVES else slice(0, 2 * pairs, 2)
    two = slice(pairs, 2 * pairs) if layout == tp.TP_ROTARY_HALVES else slice(1, 2 * pairs, 2)
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = a * c - b * s, a * s + b * c
    tol = torch.zeros_like(y)
    tol[..., one] = tol[..., two] = (a.abs() + b.abs()) * slack[:, None]
    tol += y.abs() * torch.finfo(x.dtype).eps / 2
    tol[..., 2 * pairs:] = 0
    return y.view_as(x), tol.view_as(x) * 1.01


def make(tp_size, hq, hkv, d, T, pairs, axes, dtype, seed=0, pad=0, top=4096):
    g = torch.Generator(device="cuda").manual_seed(seed + T * 131 + d)
    plan = tp.tp_plan_create(tp_size, hq * d, hq, hkv, d, tp_size)
    sources = tp_size if hkv >= tp_size else 1
    whole = {}
    for name, heads in (("q", hq), ("k", hkv)):
        t = torch.randn(T, heads * d + pad, generator=g, device="cuda").to(TYPES[dtype])
        whole[name] = t[:, :heads * d]
    pos = torch.randint(-top // 2, top, (axes, T), generator=g, device="cuda", dtype=torch.int32)
    freq = (10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).float()
    axis = [i * axes // pairs for i in range(pairs)]
    return plan, sources, whole, pos, freq, axis


def split(t, n):
    return list(t.split(t.shape[1] // n, dim=1))


SHAPES = [  # tp, Hq, Hkv, d, T, pairs, axes, padding of the rows
    (1, 1, 1, 64, 1, 32, 1, 0), (1, 4, 2, 128, 1, 64, 3, 0), (2, 8, 2, 128, 77, 64, 3, 0), (8, 16, 4, 128, 5, 64, 1, 0),
    (1, 3, 1, 64, 129, 16, 2, 0),      # a part of the head
    (1, 2, 2, 64, 33, 5, 2, 0),        # pairs that fill no 16 bytes
    (1, 2, 1, 6, 50, 3, 3, 0),         # heads that fill none
    (2, 4, 4, 128, 19, 24, 1, 3),      # odd pitches
    (1, 1, 1, 256, 600, 128, 8, 0), (1, 1, 1, 512, 9, 256, 4, 8), (4, 12, 3, 80, 40, 40, 1, 0),
    (1, 64, 8, 128, 1500, 64, 3, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [tp.TP_ROTARY_HALVES, tp.TP_ROTARY_NEIGHBOURS])
def test_against_float64(shape, dtype, layout):
    need_gpu()
    n, hq, hkv, d, T, pairs, axes, pad = shape
    if hkv >= n and hkv % n:
        pytest.skip("no such plan")
    plan, s, x, pos, freq, axis = make(n, hq, hkv, d, T, pairs, axes, dtype, pad=pad)
    out = {k: torch.full_like(v, float("nan")) for k, v in x.items()}
    tp.tp_rotary(plan, pos, freq, split(x["q"], n), split(x["k"], s), split(out["q"], n), split(out["k"], s), axis=axis, layout=layout)
    for name in ("q", "k"):
        want, tol = reference(x[name], pos, freq, axis, d, layout)
        assert ((out[name].double() - want).abs() <= tol).all(), name
    # in place, and each alone, give the same bits
    q, k = x["q"].clone(), x["k"].clone()
    tp.tp_rotary(plan, pos, freq, split(q, n), None, split(q, n), None, axis=axis, layout=layout)
    tp.tp_rotary(plan, pos, freq, None, split(k, s), None, split(k, s), axis=axis, layout=layout)
    assert torch.equal(q, out["q"]) and torch.equal(k, out["k"])


def test_far_positions():
    """Angles of 10^9 radians: f32 products of position and frequency would be off by whole turns."""
    need_gpu()
    plan, s, x, _, freq, axis = make(1, 2, 1, 128, 9, 64, 1, "f32")
    pos = torch.tensor([[0, 1, -1, 1 << 20, (1 << 24) + 1, -(1 << 30) - 7, 1000000007, (1 << 31) - 1, -(1 << 31)]], dtype=torch.int32,
                       device="cuda")
    out = [torch.empty_like(x["q"]), torch.empty_like(x["k"])]
    tp.tp_rotary(plan, pos, freq, [x["q"]], [x["k"]], [out[0]], [out[1]])
    for got, name in zip(out, ("q", "k")):
        want, tol = reference(x[name], pos, freq, [0] * 64, 128, tp.TP_ROTARY_HALVES)
        assert ((got.double() - want).abs() <= tol).all()
    assert torch.equal(out[0][0], x["q"][0])  # position 0 turns nothing


@pytest.mark.parametrize("layout", [tp.TP_ROTARY_HALVES, tp.TP_ROTARY_NEIGHBOURS])
def test_inverse_is_the_gradient(layout):
    """The gradient by autograd of the formula, and by differences of the call, is the inverse turn."""
    need_gpu()
    plan, s, x, pos, freq, axis = make(1, 2, 1, 64, 11, 24, 2, "f32")
    dy = torch.randn_like(x["q"])
    dx = torch.empty_like(dy)
    tp.tp_rotary(plan, pos, freq, [dy], None, [dx], None, axis=axis, layout=layout, inverse=True)
    leaf = x["q"].double().requires_grad_()
    y = leaf.view(11, -1, 64)
    angle = pos.double()[torch.tensor(axis, device="cuda")].t() * freq.double()
    c, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = (y[..., :24], y[..., 24:48]) if layout == tp.TP_ROTARY_HALVES else (y[..., 0:48:2], y[..., 1:48:2])
    ra, rb = a * c - b * sn, a * sn + b * c
    turned = torch.cat([ra, rb], -1) if layout == tp.TP_ROTARY_HALVES else torch.stack([ra, rb], -1).flatten(-2)
    torch.cat([turned, y[..., 48:]], -1).view_as(leaf).backward(dy.double())
    want, tol = reference(dy, pos, freq, axis, 64, layout, inverse=True)
    assert torch.allclose(leaf.grad, want, rtol=0, atol=1e-12)
    assert ((dx.double() - leaf.grad).abs() <= tol).all()
    # differences: the call is linear, so a step of 1 in one value gives the derivative itself
    base = torch.zeros_like(x["q"])
    for col in (0, 5, 30, 47, 50, 127):
        step = base.clone()
        step[:, col] = 1.0
        out = torch.empty_like(step)
        tp.tp_rotary(plan, pos, freq, [step], None, [out], None, axis=axis, layout=layout)
        assert torch.allclose((out.double() * dy.double()).sum(1), leaf.grad[:, col], rtol=0, atol=128 * 6 * 2.0 ** -22)


def test_rows_apart_and_special_values():
    need_gpu()
    plan, s, x, pos, freq, axis = make(1, 2, 1, 128, 40, 64, 1, "bf16")
    buf = torch.full((40, 2 * 128 + 24), 7.0, device="cuda").to(torch.bfloat16)
    out = buf[:, 8:8 + 256]
    x["q"][3, 5], x["q"][4, 200] = float("nan"), float("inf")
    tp.tp_rotary(plan, pos, freq, [x["q"]], None, [out], None, axis=axis)
    assert (buf[:, :8] == 7).all() and (buf[:, 264:] == 7).all()  # nothing beside the view is written
    assert out[3, 5].isnan() and out[3, 69].isnan() and not out[3, 6].isnan() and not out[3, 128 + 5].isnan()
    assert not torch.isfinite(out[4, 200].float()) and torch.isfinite(out[4, 72].float())


def test_other_stream_and_captured_graph():
    need_gpu()
    plan, s, x, pos, freq, axis = make(2, 4, 2, 128, 70, 64, 3, "bf16")
    want = torch.empty_like(x["q"])
    tp.tp_rotary(plan, pos, freq, split(x["q"], 2), None, split(want, 2), None, axis=axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    tp.tp_rotary(plan, pos, freq, split(x["q"], 2), None, split(got, 2), None, axis=axis, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_rotary(plan, pos, freq, split(x["q"], 2), None, split(got, 2), None, axis=axis)
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_no_tokens():
    need_gpu()
    plan = tp.tp_plan_create(1, 128, 1, 1, 128, 1)
    e = torch.empty(0, 128, device="cuda")
    tp.tp_rotary(plan, torch.empty(1, 0, dtype=torch.int32, device="cuda"), torch.ones(64, device="cuda"), [e], [e], [e], [e])
