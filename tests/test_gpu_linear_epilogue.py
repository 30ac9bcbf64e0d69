"""tp_linear_epilogue against the formula in float64.

Tolerances, from the roundings the call makes (u = 2^-24): the products of bf16 or e4m3 values
are exact in f32; the tensor core adds one step of 16 (bf16) or 32 (e4m3) products at a time
into the f32 accumulator and may truncate, so a sum is off by at most (K / 16 + 16) * 2u of the
sum of the products' sizes. Scales and bias add 4u of the value; the activations are
1.13-Lipschitz and off by (8 + 2 |v|) * 2u of their value (x Phi(x): of |v|); the residual's
addition adds u; the output is rounded once (f32 u, bf16 2^-8 of the value)."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def padded(rows, cols, dtype):
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.zeros(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def draw(rows, cols, dtype, g, std):
    t = padded(rows, cols, dtype)
    t.copy_((torch.randn(rows, cols, generator=g, device="cuda") * std).to(dtype))
    return t


def act64(v, name):
    if name == "relu":
        return v.clamp_min(0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def check(y, x, w, xs, ws, bias, act, res):
    K = x.shape[1]
    acc = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if xs is not None:
        f = xs.double()[:, None] * ws.double()
        acc, size = acc * f, size * f
    tol = (K / 16 + 16) * 2 * U * size + 4 * U * acc.abs()
    v = acc
    if bias is not None:
        v = v + bias.double()
        tol = tol + 2 * U * v.abs()
    out = act64(v, act)
    if act == "gelu":
        tol = 1.13 * tol + (8 + 2 * v.abs()) * 2 * U * v.abs()
    elif act == "silu":
        tol = 1.13 * tol + (8 + 2 * v.abs()) * 2 * U * out.abs() + 1e-36
    if res is not None:
        out = out + res.double()
        tol = tol + U * out.abs()
    half = U if y.dtype == F32 else 2.0 ** -8
    err = (y.double() - out).abs()
    assert torch.isfinite(y.float()).all()
    assert (err <= tol * 1.01 + half * (out.abs() + tol) + 1e-37).all(), float((err - tol - half * out.abs()).max())


class Problem:
    def __init__(self, T, K, N, dtype, seed, apart=False, tp_size=1, shard="column"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        e = dtype == E4M3
        self.x, self.w = draw(T, K, dtype, g, 40.0 if e else 1.0), draw(N, K, dtype, g, 40.0 if e else 0.05)
        self.xs = torch.rand(T, generator=g, device="cuda") * 0.05 + 0.01 if e else None
        self.ws = torch.rand(N, generator=g, device="cuda") * 0.002 + 0.001 if e else None
        self.bias = torch.randn(N, generator=g, device="cuda")
        self.res = {F32: draw(T, N, F32, g, 1.0), BF16: draw(T, N, BF16, g, 1.0), None: None}
        own = (lambda t: padded(*t.shape, t.dtype).copy_(t)) if apart else (lambda t: t)
        if shard == "row":
            self.xr = [own(t) for t in self.x.split(K // tp_size, dim=1)]
            self.wr = [own(t) for t in self.w.split(K // tp_size, dim=1)]
        else:
            self.xr, self.wr = [self.x], [own(t) for t in self.w.split(N // tp_size, dim=0)]
        self.n, self.shard = tp_size, tp.TP_SHARD_ROW if shard == "row" else tp.TP_SHARD_COLUMN

    def run(self, y_dtype=BF16, bias=True, act="none", res=None, in_place=False):
        r = self.res[res]
        y = padded(self.x.shape[0], self.w.shape[0], y_dtype)
        if in_place:
            y.copy_(r)
        b = (self.bias if bias is True else bias) if bias is not False else None
        tp.tp_linear_epilogue(self.n, self.shard, self.xr, self.wr, y, bias=b, activation=tp.ACTIVATIONS[act],
                              residual=y if in_place else r, x_scale=self.xs, w_scale=self.ws)
        torch.cuda.synchronize()
        assert tp.tp_device_status()[0] == tp.TP_OK
        check(y, self.x, self.w, self.xs, self.ws, b, act, r)
        return y


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 4096, 4096), (2, 17, 5), (16, 200, 130), (17, 1000, 300), (61, 4096, 1792),
          (64, 130, 4097), (128, 512, 512), (129, 333, 257), (255, 2048, 1000), (256, 256, 256), (257, 64, 513),
          (517, 1000, 2050), (1000, 520, 2560), (2047, 777, 1283), (4097, 96, 640)]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_shapes(T, K, N, dtype):
    need_gpu()
    p = Problem(T, K, N, dtype, T + K + N)
    p.run(y_dtype=BF16, bias=True, act="none", res=None)
    p.run(y_dtype=F32, bias=False, act="none", res=F32)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("T", [3, 200, 1024])
def test_epilogues(T, dtype):
    need_gpu()
    p = Problem(T, 384, 1544, dtype, T)
    for act, res, y_dtype, bias in itertools.product(("none", "relu", "gelu", "silu"), (None, BF16, F32), (BF16, F32),
                                                     (True, False)):
        p.run(y_dtype=y_dtype, bias=bias, act=act, res=res)
    p.run(bias=p.bias.to(BF16), act="silu")
    p.run(y_dtype=F32, res=F32, in_place=True)
    p.run(y_dtype=BF16, res=BF16, in_place=True, act="gelu")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("shard", ["column", "row"])
@pytest.mark.parametrize("T,tp_size", [(1, 8), (33, 4), (700, 2), (2100, 8)])
def test_shards(T, tp_size, shard, apart, dtype):
    need_gpu()
    p = Problem(T, 16 * 8 * 9, 8 * 8 * 17, dtype, T, apart, tp_size, shard)
    p.run(y_dtype=BF16, act="relu", res=BF16)
    y = p.run(y_dtype=F32, res=F32)
    assert torch.equal(y, p.run(y_dtype=F32, res=F32))  # sums in a fixed order


def test_empty_slices_and_rows():
    need_gpu()
    p = Problem(5, 64, 64, BF16, 1)
    y = padded(5, 64, F32)
    none = torch.empty(5, 0, dtype=BF16, device="cuda")
    tp.tp_linear_epilogue(2, tp.TP_SHARD_ROW, [p.x, none], [p.w, torch.empty(64, 0, dtype=BF16, device="cuda")], y)
    check(y, p.x, p.w, None, None, None, "none", None)
    y.zero_()
    tp.tp_linear_epilogue(2, tp.TP_SHARD_COLUMN, [p.x], [torch.empty(0, 64, dtype=BF16, device="cuda"), p.w], y)
    check(y, p.x, p.w, None, None, None, "none", None)
    tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, [torch.empty(0, 64, dtype=BF16, device="cuda")], [p.w],
                          torch.empty(0, 64, device="cuda"))
    torch.cuda.synchronize()


def test_infinities_and_nan_stay_in_their_rows():
    need_gpu()
    p = Problem(40, 128, 256, BF16, 2)
    p.x[3, 5] = float("inf")
    p.x[7, 0] = float("nan")
    y = padded(40, 256, F32)
    tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, [p.x], [p.w], y, activation=tp.TP_ACT_RELU)
    assert torch.isnan(y[7]).all()
    assert not torch.isfinite(y[3]).all()
    rest = [i for i in range(40) if i not in (3, 7)]
    check(y[rest], p.x[rest], p.w, None, None, None, "relu", None)


def test_norm_feeds_the_8_bit_product():
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(9)
    T, D, N = 37, 512, 384
    h = torch.randn(T, D, generator=g, device="cuda")
    gain = torch.ones(D, device="cuda")
    x, xs = torch.empty(T, D, dtype=E4M3, device="cuda"), torch.empty(T, device="cuda")
    tp.tp_add_rmsnorm(h, None, gain, 1e-5, None, x, xs)
    w = draw(N, D, E4M3, g, 30.0)
    ws = torch.full((N,), 1e-3, device="cuda")
    y = torch.empty(T, N, dtype=F32, device="cuda")
    tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, [x], [w], y, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    check(y, x, w, xs, ws, None, "none", None)


# Steps of the tensor core's f32 accumulation (32 bytes of K each) in one accumulator, by the launch rules:
# K / 16 (bf16) or K / 32 (e4m3) over the split and over the accumulators that fit in tensor memory, 64 at
# least as a bound. One accumulator of n steps is off by 1.6e-8 n of the result's norm (it truncates: 8e-6
# over 512 steps); the limit is one and a half times that plus the f32 output's 2^-24.
@pytest.mark.parametrize("T, K, N, dtype, steps", [
    (1, 8192, 8192, BF16, 64), (64, 8192, 8192, BF16, 64), (128, 8192, 8192, BF16, 64), (61, 5000, 14336, BF16, 64),
    (128, 16384, 2048, E4M3, 64), (64, 8192, 28672, E4M3, 64),
    (200, 8192, 8192, BF16, 128), (300, 8192, 4096, BF16, 128), (256, 8192, 4096, E4M3, 64),
    (1000, 8192, 4096, BF16, 64), (1030, 5000, 2560, BF16, 64), (1000, 16384, 4096, E4M3, 64),
])
def test_f32_sums_over_a_long_k(T, K, N, dtype, steps):
    need_gpu()
    p = Problem(T, K, N, dtype, K + T)
    y = padded(T, N, F32)
    tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, p.xr, p.wr, y, x_scale=p.xs, w_scale=p.ws)
    want = p.x.double() @ p.w.double().t()
    if dtype == E4M3:
        want = want * p.xs.double()[:, None] * p.ws.double()
    err = float((y.double() - want).norm() / want.norm())
    assert err <= 1.5 * 1.6e-8 * steps + U


def one_value_a_row(v, act):
    """act(v) for every element of a row, through a product that gives v exactly."""
    T = len(v)
    x, w, y = padded(T, 64, BF16), padded(1544, 64, BF16), padded(T, 1544, F32)
    x[:, 3] = v
    w[:, 3] = 1.0
    tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, [x], [w], y, activation=act)
    return y.double()


# x Phi(x) = x/2 erfc(-x / sqrt 2): the argument is off by 2u of itself, which moves erfc by at most
# x^2 + 1 times that, erfc by 8u, and two products by u.
@pytest.mark.parametrize("T", [40, 1200])
def test_gelu_far_in_its_tail(T):
    need_gpu()
    v = torch.linspace(-12.0, 12.0, T, device="cuda").to(BF16)
    y, f = one_value_a_row(v, tp.TP_ACT_GELU), v.double()
    want, rel = 0.5 * f * torch.erfc(-f / math.sqrt(2)), (2 * (f.square() + 1) + 10) * U
    assert ((y - want[:, None]).abs() <= (1.01 * rel * want.abs())[:, None]).all()


# x / (1 + e^-x): the exponential is off by 2u, the sum by u, the quotient by u; 2u are left for their forms.
@pytest.mark.parametrize("T", [40, 1200])
def test_silu_far_in_its_tail(T):
    need_gpu()
    v = torch.linspace(-80.0, 40.0, T, device="cuda").to(BF16)
    y, f = one_value_a_row(v, tp.TP_ACT_SILU), v.double()
    want = f / (1 + torch.exp(-f))
    assert ((y - want[:, None]).abs() <= (1.01 * 6 * U * want.abs())[:, None]).all()


# Few tokens and a K of more chunks of 64 steps than fit in tensor memory: they are added under the
# products, through every accumulator several times over. The limit is that of 64 steps above.
@pytest.mark.parametrize("T, K, N, dtype", [
    (128, 8192, 28672, BF16), (100, 28672, 8192, BF16), (200, 8192, 8192, BF16), (300, 20000, 4096, BF16),
    (17, 16384, 20480, BF16), (61, 20000, 14336, BF16), (1, 28672, 4096, BF16), (128, 16384, 28672, E4M3), (256, 28672, 8192, E4M3),
])
def test_f32_sums_that_outgrow_tensor_memory(T, K, N, dtype):
    need_gpu()
    p = Problem(T, K, N, dtype, K + T)
    y, again = padded(T, N, F32), padded(T, N, F32)
    for out in (y, again):
        tp.tp_linear_epilogue(1, tp.TP_SHARD_COLUMN, p.xr, p.wr, out, x_scale=p.xs, w_scale=p.ws)
    assert torch.equal(y, again)
    want = torch.cat([p.x.double() @ w.double().t() for w in p.w.split(4096)], 1)
    if dtype == E4M3:
        want = want * p.xs.double()[:, None] * p.ws.double()
    err = float((y.double() - want).norm() / want.norm())
    assert err <= 1.5 * 1.6e-8 * 64 + U
    assert tp.tp_device_status()[0] == tp.TP_OK
