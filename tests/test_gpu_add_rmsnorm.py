"""tp_add_rmsnorm against the definition in float64, row by row and element by element.

Tolerances, from the roundings the call makes: z is a sum of n_x + 1 terms in f32 (each
addition 2^-24 of a partial sum, bounded by the sum of the terms' sizes); the sum of squares
adds positive terms over at most 64 f32 roundings, so the factor rsqrt(mean + eps) is off by
at most 40 * 2^-24 with rsqrtf's own error; the output is rounded once, by half a step
(bf16 2^-8, e4m3 2^-4 relative, or half its smallest step 2^-10 in units of the scale)."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def padded(rows, cols, dtype, lead=0, pad=None):
    """An uninitialised [rows x cols] view; lead elements before it, pitch rounded to 16 bytes or cols + pad."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = -(-cols // per) * per if pad is None else cols + pad
    base = torch.zeros(rows * ld + lead + per, dtype=dtype, device="cuda")
    return base[lead:lead + rows * ld].view(rows, ld)[:, :cols]


def reference(xs, res, w):
    z = sum(x.double() for x in xs)
    size = sum(x.double().abs() for x in xs)
    if res is not None:
        z = z + res.double()
        size = size + res.double().abs()
    factor = 1.0 / (z.square().mean(1, keepdim=True) + EPS).sqrt()
    return z, size, z * factor * w.double(), factor


def check(xs, res, w, y_type, res_out, y, scale):
    z, size, v, factor = reference(xs, res, w)
    n = len(xs) + 1
    dz = n * U * size
    if res_out is not None:
        half = torch.finfo(res_out.dtype).eps / 2
        assert ((res_out.double() - z).abs() <= half * z.abs() + dz * 1.01 + 1e-38).all()
    # an error of z moves v by itself and through the factor
    rel_factor = 40 * U + (dz.square().mean(1, keepdim=True).sqrt() * factor)
    slack = dz * factor * w.double().abs() + (rel_factor + 6 * U) * v.abs()
    if y_type == "e4m3":
        top = v.abs().amax(1).clamp_min(2.0 ** -96)
        tol = (rel_factor[:, 0] + 8 * U) * top + (dz * factor * w.double().abs()).amax(1)
        assert ((scale.double() * 448.0 - top).abs() <= tol).all()
        got = y.double() * scale.double()[:, None]
        assert ((got - v).abs() <= 2.0 ** -4 * v.abs() + scale.double()[:, None] * 2.0 ** -10 + 1.07 * slack).all()
        # the largest element of a row of ordinary size has the largest code
        assert (y.double().abs().amax(1)[top > 2.0 ** -90] == 448.0).all()
    else:
        assert ((y.double() - v).abs() <= 2.0 ** -8 * v.abs() + 1.01 * slack + 1e-38).all()


def run(xs, res, w, y_type, in_place=False, **layout):
    T, D = xs[0].shape
    y = padded(T, D, TYPES[y_type], **layout)
    scale = torch.full((T,), float("nan"), device="cuda") if y_type == "e4m3" else None
    res_in = None if res is None else res.clone()
    res_out = None if res is None else (res if in_place else padded(T, D, res.dtype, **layout))
    tp.tp_add_rmsnorm(xs if len(xs) > 1 else xs[0], res, w, EPS, res_out, y, scale)
    torch.cuda.synchronize()
    check(xs, res_in, w, y_type, res_out, y, scale)


@pytest.mark.parametrize("y_type", ["bf16", "e4m3"])
@pytest.mark.parametrize("x_type,res_type,n", [("bf16", "bf16", 1), ("f32", "f32", 8), ("f32", "bf16", 3),
                                               ("bf16", "f32", 2), ("f32", None, 1), ("bf16", None, 5)])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (2, 8), (5, 129), (64, 4096), (7, 4104), (3, 8200), (2, 16384), (2, 16392)])
def test_against_definition(T, D, x_type, res_type, n, y_type):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(T * 131 + D)

    def draw(dtype, std):
        t = padded(T, D, dtype)
        t.copy_(torch.randn(T, D, generator=g, device="cuda") * std)
        return t

    xs = [draw(TYPES[x_type], 1.0) for _ in range(n)]
    res = draw(TYPES[res_type], 3.0) if res_type else None
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(TYPES["bf16" if D % 2 else "f32"])
    run(xs, res, w, y_type)


@pytest.mark.parametrize("D", [8, 250, 4096, 9000])
@pytest.mark.parametrize("res_type", ["f32", "bf16"])
def test_residual_in_place_and_odd_alignment(D, res_type):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(D)
    for lead, pad in ((0, None), (1, 3)):
        x = padded(6, D, torch.float32, lead, pad)
        x.copy_(torch.randn(6, D, generator=g, device="cuda"))
        res = padded(6, D, TYPES[res_type], lead, pad)
        res.copy_(torch.randn(6, D, generator=g, device="cuda"))
        w = torch.randn(D, generator=g, device="cuda")
        run([x], res, w, "bf16", in_place=True, lead=lead, pad=pad)
        run([x], res, w, "e4m3", in_place=True, lead=lead, pad=pad)


def test_rows_of_zeros_tiny_large_and_nan():
    need_gpu()
    D = 512
    x = torch.zeros(5, D, device="cuda")
    x[1] = 1e-30
    x[2] = 1e15
    x[3, 7] = float("nan")
    x[4, 9] = 1000.0  # one outlier: every other code is far below it
    x[4, 10] = 1.0
    w = torch.ones(D, device="cuda")
    y = torch.empty(5, D, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(5, device="cuda")
    tp.tp_add_rmsnorm(x, None, w, EPS, None, y, scale)
    assert (y[0].float() == 0).all() and scale[0].item() == pytest.approx(2.0 ** -96 / 448)
    assert torch.isfinite(y[1].float()).all() and torch.isfinite(scale[:3]).all()
    assert (y[2].float() == 448.0).all()
    assert torch.isnan(y[3].float()).all()
    assert y[4, 9].float().item() == 448.0 and y[4, 10].float().item() == 0.4375  # 0.448 on the e4m3 grid
    yb = torch.empty(5, D, dtype=torch.bfloat16, device="cuda")
    tp.tp_add_rmsnorm(x, None, w, EPS, None, yb)
    assert torch.isnan(yb[3].float()).all() and torch.isfinite(yb[[0, 1, 2, 4]].float()).all()


def test_partials_are_added_in_rank_order_and_runs_repeat():
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn(33, 1000, generator=g, device="cuda") * 10 ** r for r in range(4)]
    res = torch.randn(33, 1000, generator=g, device="cuda")
    out = torch.empty_like(res)
    y = torch.empty(33, 1000, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1000, device="cuda")
    tp.tp_add_rmsnorm(xs, res, w, EPS, out, y)
    assert torch.equal(out, (((xs[0] + xs[1]) + xs[2]) + xs[3]) + res)
    again = torch.empty_like(y)
    tp.tp_add_rmsnorm(xs, res, w, EPS, out, again)
    assert torch.equal(y, again)


def test_empty_and_other_stream():
    need_gpu()
    w = torch.ones(64, device="cuda")
    tp.tp_add_rmsnorm(torch.empty(0, 64, device="cuda"), None, w, EPS, None,
                      torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    side = torch.cuda.Stream()
    x = torch.randn(9, 64, device="cuda")
    y = torch.empty(9, 64, dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    tp.tp_add_rmsnorm(x, None, w, EPS, None, y, stream=side)
    side.synchronize()
    check([x], None, w, "bf16", None, y, None)


@pytest.mark.parametrize("D, n, lead, pad", [(512, 1, 0, None), (512, 3, 0, None), (16384, 1, 0, None), (250, 1, 1, 3),
                                             (20000, 1, 0, None)])
def test_nan_and_infinities_reach_the_scale(D, n, lead, pad):
    """The largest |y| of such a row is not a number, so its scale is none, and neither is any code."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(D + n)
    xs = []
    for _ in range(n):
        x = padded(6, D, torch.float32, lead, pad)
        x.copy_(torch.randn(6, D, generator=g, device="cuda"))
        xs.append(x)
    xs[-1][1, D - 3] = float("inf")
    xs[0][2, 4] = float("-inf")
    xs[0][4, D // 2] = float("nan")
    w = 1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")
    y, scale = padded(6, D, TYPES["e4m3"], lead, pad), torch.zeros(6, device="cuda")
    tp.tp_add_rmsnorm(xs if n > 1 else xs[0], None, w, EPS, None, y, scale)
    torch.cuda.synchronize()
    for row in (1, 2, 4):
        assert torch.isnan(scale[row]) and torch.isnan(y[row].float()).all()
    rest = [0, 3, 5]
    check([x[rest] for x in xs], None, w, "e4m3", None, y.view(torch.uint8)[rest].view(TYPES["e4m3"]), scale[rest])
    w[7] = float("nan")
    tp.tp_add_rmsnorm(xs if n > 1 else xs[0], None, w, EPS, None, y, scale)
    assert torch.isnan(scale).all() and torch.isnan(y.float()).all()
