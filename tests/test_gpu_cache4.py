"""The 4-bit caches: storing and reading back exactly, attention against the softmax in float64 over the
values that the codes stand for.

Tolerances of the attention, from the roundings it makes (u = 2^-24): products of q and whole codes are exact; a
group's sum of 32 of them starts at -8 sum(q) and is off by at most 18 * 2u of its parts' sizes, which
with codes of 0..15 are at most (|code - 8| + 16) |q|; scaling and adding the groups adds 8u of the same.
q enters in f16 scaled to its head's largest value: values below 2^-28 of it lose bits, at most 2^-34
of it each. A softmax weight is off by at most twice the largest score error, plus 2^-18 for the exponentials
and the joins. p times the scale is rounded to bf16 (2^-8) and the output once (2^-8)."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.bfloat16
ALL = 2 ** 31 - 1


def definition(x):
    """(codes, bf16 scales) of values [.., d], in float64."""
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    bad = ~torch.isfinite(g).all(-1)
    scale = torch.where(bad, float("nan"), top / 7).to(BF16)
    s = scale.double()[..., None]
    code = torch.where(s > 0, torch.clamp(torch.round(g / torch.where(s > 0, s, 1.0)), -8, 7), 0.0)
    return (code.nan_to_num(0.0) + 8).to(torch.uint8).flatten(-2), scale


def row_bytes(code, piece):
    """The documented order of a row's bytes: pieces of `piece` values, group by group."""
    d = code.shape[-1]
    out = torch.zeros(*code.shape[:-1], d // 2, dtype=torch.uint8, device=code.device)
    at = 0
    for first in range(0, 32, piece):
        for group in range(d // 32):
            for i in range(0, piece, 2):
                v = group * 32 + first + i
                out[..., at] = code[..., v] | code[..., v + 1] << 4
                at += 1
    return out


class Cache:
    """A cache of `batch` sequences on the GPU, and its values in float64."""

    def __init__(self, tp_size, hq, hkv, d, B, C, fill=0xAA):
        self.plan = tp.tp_plan_create(tp_size, hq * d, hq, hkv, d, tp_size)
        self.n, self.s = tp_size, tp_size if hkv >= tp_size else 1
        self.hq, self.hkv, self.d, self.B, self.C, self.hr = hq, hkv, d, B, C, hkv // self.s
        rows = B * self.hr * C
        self.codes = [torch.full((self.s, rows, d // 2), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scale = [torch.full((self.s, rows, d // 32), float("nan"), dtype=BF16, device="cuda") for _ in range(2)]

    def args(self):
        return list(self.codes[0]), list(self.scale[0]), list(self.codes[1]), list(self.scale[1])

    def store(self, k, v, lengths, counts=None, stream=None):
        tp.tp_cache4_store(self.plan, lengths, self.cols(k), self.cols(v), *self.args(), counts=counts, stream=stream)

    def load(self, first, n, dtype=torch.float32):
        k, v = (torch.full((self.B * n, self.hkv * self.d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        tp.tp_cache4_load(self.plan, first, *self.args(), self.cols(k), self.cols(v))
        return k, v

    def cols(self, t, n=None):
        n = n or self.s
        return list(t.split(t.shape[1] // n, dim=1))

    def view(self, which):
        """[source, B, heads, C, ..] views of the codes and the scales."""
        return (t.view(self.s, self.B, self.hr, self.C, t.shape[-1]) for t in (self.codes[which], self.scale[which]))


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(rows, cols, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std).to(BF16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tp_size, hkv", [(1, 1), (2, 2), (4, 2), (2, 4), (1, 3)])
@pytest.mark.parametrize("n", [1, 3, 37])
def test_store_and_load(d, tp_size, hkv, n):
    need_gpu()
    B, C = 5, 41
    c = Cache(tp_size, max(tp_size, hkv) if max(tp_size, hkv) % hkv == 0 else hkv, hkv, d, B, C)
    k, v = normal(B * n, hkv * d, n), normal(B * n, hkv * d, n + 1, 1e-3)
    k[0, :32] = 0                                   # a group of zeros
    k[1 % (B * n), 32:64] = k[1 % (B * n), 32:64] * 1e-38   # subnormal scales
    v[-1, -32:] = v[-1, -32:].sign() * 2.0 ** 100
    start = [0, C - n, 1, 2, 0]
    before = [t.clone() for t in c.codes + [x.view(torch.int16) for x in c.scale]]
    c.store(k, v, ints(*start))
    assert tp.tp_device_status()[0] == tp.TP_OK
    for which, (x, piece) in enumerate(((k, 8), (v, 4))):
        code, scale = definition(x.view(B, n, c.s, c.hr, d))
        codes, scales = c.view(which)
        old_c = before[which].view_as(codes)
        old_s = before[2 + which].view(*scales.shape)
        for b in range(B):
            at = slice(start[b], start[b] + n)
            want = row_bytes(code[b], piece).permute(1, 2, 0, 3)
            assert torch.equal(codes[:, b, :, at], want)
            assert torch.equal(scales[:, b, :, at].view(torch.int16), scale[b].permute(1, 2, 0, 3).contiguous().view(torch.int16))
            rest = torch.ones(C, dtype=torch.bool, device="cuda")
            rest[at] = False
            assert torch.equal(codes[:, b][:, :, rest], old_c[:, b][:, :, rest])  # other positions stay
            assert torch.equal(scales[:, b][:, :, rest].view(torch.int16), old_s[:, b][:, :, rest])
        value = (code.double() - 8) * scale.double().repeat_interleave(32, -1)
        got = c.load(ints(*start), n)[which]
        assert torch.equal(got.double(), value.view(B * n, -1))
        assert torch.equal(c.load(ints(*start), n, BF16)[which], value.view(B * n, -1).float().to(BF16))


def test_groups_that_are_not_finite():
    need_gpu()
    c = Cache(1, 1, 1, 64, 1, 4)
    k, v = normal(2, 64, 1), normal(2, 64, 2)
    k[0, 3], k[1, 40], v[0, 0], v[1, 63] = float("nan"), float("inf"), float("-inf"), float("nan")
    c.store(k, v, ints(1))
    gk, gv = c.load(ints(1), 2)
    assert gk[0, :32].isnan().all() and gk[1, 32:].isnan().all() and gv[0, :32].isnan().all() and gv[1, 32:].isnan().all()
    assert torch.isfinite(gk[0, 32:]).all() and torch.isfinite(gk[1, :32]).all() and torch.isfinite(gv[0, 32:]).all()


def test_counts_and_lengths_out_of_range():
    need_gpu()
    B, n, C = 6, 4, 10
    k, v = normal(B * n, 128, 3), normal(B * n, 128, 4)
    full = Cache(1, 1, 1, 128, B, C, fill=0x88)
    full.scale[0].zero_(), full.scale[1].zero_()
    full.store(k, v, ints(0, 3, 6, 0, 2, 5), counts=ints(4, 0, 2, 1, 4, 3))
    assert tp.tp_device_status()[0] == tp.TP_OK
    want = full.load(ints(*[0] * B), C)
    for b, (start, count) in enumerate(zip((0, 3, 6, 0, 2, 5), (4, 0, 2, 1, 4, 3))):
        rows = want[0][b * C:(b + 1) * C]
        filled = (rows != 0).any(1).nonzero().flatten().tolist()
        assert filled == list(range(start, start + count))
    for lengths, counts, kept in (([-1, 0, 0, 0, 0, 0], None, [0, 4, 4, 4, 4, 4]), ([11, 10, 8, 0, 0, 0], None, [0, 0, 2, 4, 4, 4]),
                                  ([0] * 6, [5, -1, 4, 4, 4, 4], [4, 0, 4, 4, 4, 4]),
                                  ([2 ** 31 - 1, -2 ** 31, 0, 0, 0, 0], None, [0, 0, 4, 4, 4, 4]),
                                  ([-1, 0, 0, 0, 0, 0], [0, 4, 4, 4, 4, 4], [0, 4, 4, 4, 4, 4])):
        c = Cache(1, 1, 1, 128, B, C, fill=0x88)
        c.scale[0].zero_(), c.scale[1].zero_()
        c.store(k, v, ints(*lengths), counts=None if counts is None else ints(*counts))
        assert tp.tp_device_status()[0] == tp.TP_ERR_BAD_LENGTH
        rows = c.load(ints(*[0] * B), C)[0].view(B, C, 128)
        assert [(rows[b] != 0).any(1).sum().item() for b in range(B)] == kept
    assert tp.tp_device_status()[0] == tp.TP_OK
    for first in (-1, 11, -2 ** 31):
        gk, _ = full.load(ints(first, 8, 0, 0, 0, 0), 4)
        assert tp.tp_device_status()[0] == tp.TP_ERR_BAD_LENGTH
        assert (gk[:4] == 0).all() and (gk[6:8] == 0).all()  # positions past the end


def test_a_batch_of_which_a_part_is_given():
    """A sequence's rows are neighbours: a prompt goes into one sequence of a batch's cache."""
    need_gpu()
    c = Cache(1, 2, 2, 128, 3, 20, fill=0)
    k, v = normal(7, 256, 5), normal(7, 256, 6)
    one = [t[0].view(3, 40, -1)[1] for t in (c.codes[0], c.scale[0], c.codes[1], c.scale[1])]
    tp.tp_cache4_store(c.plan, ints(2), [k], [v], *[[t] for t in one])
    codes, _ = c.view(0)
    assert (codes[:, 0] == 0).all() and (codes[:, 2] == 0).all()
    assert torch.equal(codes[0, 1, :, 2:9], row_bytes(definition(k.view(7, 2, 128))[0], 8).permute(1, 0, 2))


class Attention(Cache):
    def __init__(self, tp_size, hq, hkv, d, B, C, lens, window, sinks, seed=0, q_std=1.0, k_std=1.0):
        super().__init__(tp_size, hq, hkv, d, B, C)
        self.lens, self.window, self.sinks = ints(*lens), window, sinks
        if C > 0:
            channel = 1 + 3 * (normal(1, hkv * d, seed + 9).abs() > 1.7).to(BF16)
            self.store(normal(B * C, hkv * d, seed + 1, k_std) * channel, normal(B * C, hkv * d, seed + 2), ints(*[0] * B))
            self.kv = [t.double() for t in self.load(ints(*[0] * B), C)]
        self.q = normal(B, hq * d, seed + 3, q_std)
        # rows past the lengths hold anything
        for which in range(2):
            codes, scale = self.view(which)
            for b, n in enumerate(lens):
                scale[:, b, :, max(n, 0):] = float("nan")
                codes[:, b, :, max(n, 0):] = 0x5F

    def run(self, stream=None, views=True):
        whole = torch.full_like(self.q, float("nan"))
        q, a = (self.cols(t, self.n) for t in (self.q, whole))
        if not views:
            q, a = [x.contiguous() for x in q], [x.contiguous() for x in a]
        ws = torch.full((tp.tp_cache4_attn_workspace_size(self.plan, self.B, self.C, self.window, self.sinks),), 255, dtype=torch.uint8,
                        device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        tp.tp_cache4_attn(self.plan, q, *self.args(), self.lens, self.window, self.sinks, a, ws, stream=stream)
        torch.cuda.synchronize()
        return torch.cat(a, 1)

    def check(self, a, skip=()):
        d, G = self.d, self.hq // self.hkv
        for b in range(self.B):
            n = min(max(int(self.lens[b]), 0), self.C)
            j = torch.arange(n, device="cuda")
            j = j[(j >= n - self.window) | (j < self.sinks)] + b * self.C
            for h in range(self.hkv):
                if (b, h) in skip:
                    continue
                got = a[b].view(self.hq, d)[h * G:(h + 1) * G].double()
                if n == 0:
                    assert (got == 0).all()
                    continue
                cols = slice(h * d, (h + 1) * d)
                k, v = self.kv[0][j][:, cols], self.kv[1][j][:, cols]
                scale = definition_scale(self, b, h, j - b * self.C)
                q = self.q[b].view(self.hq, d)[h * G:(h + 1) * G].double()
                s = q @ k.t() / d ** 0.5
                size = q.abs() @ (k.abs() + 16 * scale).t() / d ** 0.5
                lost = 2.0 ** -34 * q.abs().amax(1, keepdim=True) * k.abs().sum(1) / d ** 0.5
                ds = ((18 * 2 + 8) * U * size + 4 * U * s.abs() + lost).amax(1, keepdim=True)
                p = torch.softmax(s, 1)
                out = p @ v
                tol = (2.0 ** -8 + 2 * ds + 2.0 ** -18) * (p @ v.abs()) + 2.0 ** -8 * out.abs()
                assert ((got - out).abs() <= 1.02 * tol + 1e-30).all(), (b, h, float(((got - out).abs() / tol).max()))


def definition_scale(c, b, h, j):
    """float64 scales of K at positions j, one for each value."""
    _, scale = c.view(0)
    return scale[h // c.hr, b, h % c.hr, j].double().repeat_interleave(32, -1)


SHAPES = [  # tp, Hq, Hkv, d, B, C, lengths, window, sinks
    (1, 1, 1, 128, 1, 1, [1], ALL, 0), (1, 1, 1, 64, 1, 1, [0], ALL, 0), (1, 2, 1, 64, 2, 3, [0, 3], 1, 0),
    (1, 8, 1, 128, 3, 0, [0, 0, 0], 7, 1), (1, 16, 4, 128, 1, 640, [577], ALL, 0), (2, 8, 2, 64, 5, 70, [0, 1, 69, 70, 16], 16, 1),
    (4, 8, 4, 128, 3, 200, [200, 63, 65], 48, 4), (8, 64, 8, 128, 9, 130, [0, 5, 64, 128, 129, 130, 17, 16, 15], 33, 17),
    (8, 32, 4, 128, 6, 1100, [1, 2, 3, 1098, 1099, 1100], 500, 100),      # K/V replicated, a group on two ranks
    (4, 12, 2, 64, 4, 333, [333, 0, 7, 32], ALL, 0),                       # six heads a group, replicated
    (1, 9, 1, 128, 2, 600, [600, 513], 512, 0), (1, 16, 1, 64, 2, 300, [300, 299], ALL, 0),   # two products of heads
    (1, 40, 2, 128, 2, 200, [200, 150], 100, 3), (1, 34, 2, 64, 1, 100, [99], 20, 90),        # three and two tiles of heads
    (1, 4, 2, 128, 2, 20000, [20000, 19985], ALL, 0), (1, 4, 2, 128, 2, 20000, [20000, 5000], 3000, 2000),
    (1, 8, 1, 64, 100, 45, [i % 46 for i in range(100)], 20, 2), (2, 16, 2, 128, 200, 90, [90 - i % 91 for i in range(200)], 64, 4),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6] + s[7:])))
def test_attention(shape):
    need_gpu()
    c = Attention(*shape)
    a = c.run()
    c.check(a)
    assert tp.tp_device_status()[0] == tp.TP_OK
    assert torch.equal(a, c.run(views=False))  # the same bits every time, whatever the pitch

MANY = [  # more CTAs than the SMs hold: up to 256 sequences start in the order of their length
    (1, 8, 8, 128, 61, 100, [i * 37 % 101 for i in range(61)], ALL, 0), (2, 16, 8, 64, 64, 50, [50] * 64, 20, 2),
    (1, 8, 4, 128, 130, 70, [i * 29 % 71 for i in range(130)], 40, 3), (4, 8, 4, 64, 256, 33, [(i * i) % 34 for i in range(256)], ALL, 0),
    (1, 4, 4, 128, 257, 40, [i * 7 % 41 for i in range(257)], 9, 9), (1, 8, 4, 128, 128, 40, [0] * 127 + [40], ALL, 0),
    (1, 16, 8, 64, 60, 40, [0] * 60, 5, 1), (1, 36, 2, 64, 129, 64, [64 - i % 65 for i in range(129)], 30, 0),
    (1, 2, 2, 64, 240, 300, [300 - (i * 17) % 301 for i in range(240)], ALL, 0),
    (1, 1, 1, 64, 33, 8300, [8300 - 251 * i for i in range(33)], ALL, 0),
]


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "-".join(map(str, s[:6] + s[7:])))
def test_many_sequences(shape):
    need_gpu()
    c = Attention(*shape, seed=3)
    a = c.run()
    c.check(a)
    assert tp.tp_device_status()[0] == tp.TP_OK
    assert torch.equal(a, c.run(views=False))


@pytest.mark.parametrize("q_std, k_std", [(4.0, 1.0), (30.0, 1.0), (1e-3, 1e3), (1e20, 1e-20), (1e-20, 1e20), (2.0 ** 90, 2.0 ** -90)])
def test_sharp_scores_and_sizes(q_std, k_std):
    need_gpu()
    c = Attention(2, 16, 2, 128, 4, 150, [150, 0, 77, 64], ALL, 0, seed=2, q_std=q_std, k_std=k_std)
    c.check(c.run())


def test_values_of_very_different_sizes():
    need_gpu()
    c = Attention(1, 8, 1, 128, 1, 300, [300], ALL, 0, seed=4)
    k, v = normal(300, 128, 14), normal(300, 128, 15) * torch.logspace(-12, 12, 300, device="cuda")[:, None].to(BF16)
    c.store(k, v, ints(0))
    c.kv = [t.double() for t in c.load(ints(0), 300)]
    c.check(c.run())


def test_q_of_very_different_sizes():
    """A head's values over 2^40: small ones lose bits in f16, which the tolerance counts."""
    need_gpu()
    c = Attention(1, 8, 1, 128, 1, 200, [200], ALL, 0, seed=5)
    c.q *= torch.logspace(-20, 0, 1024, base=2.0, device="cuda").to(BF16)[torch.randperm(1024, device="cuda")] ** 2
    c.check(c.run())
    c.q.zero_()
    c.check(c.run())


def test_bad_lengths_are_clamped_and_reported():
    need_gpu()
    c = Attention(1, 4, 2, 64, 3, 20, [20, 0, 9], 8, 1)
    c.lens = ints(21, -1, 9)
    c.check(c.run())
    assert tp.tp_device_status()[0] == tp.TP_ERR_BAD_LENGTH
    assert tp.tp_device_status()[0] == tp.TP_OK


def test_keys_out_of_sight_do_not_matter():
    need_gpu()
    c = Attention(1, 8, 2, 128, 2, 300, [300, 280], 50, 3, seed=6)
    want = c.run()
    for which in range(2):
        codes, scale = c.view(which)
        scale[:, 0, :, 3:250] = float("nan")
        scale[:, 1, :, 3:230] = float("inf")
    assert torch.equal(want, c.run())


def test_a_sequence_with_nan_spoils_only_itself():
    need_gpu()
    c = Attention(1, 8, 2, 128, 3, 50, [50, 50, 20], ALL, 0, seed=7)
    _, vs = c.view(1)
    vs[0, 1, 0, 3, 1] = float("nan")         # sequence 1, kv head 0, values 32..63
    a = c.run()
    assert a[1].view(8, 128)[:4, 32:64].isnan().all() and not a[1].view(8, 128)[:4, 64:].isnan().any()
    c.check(a, skip={(1, 0)})
    c.q[2, 5] = float("nan")
    a = c.run()
    assert a[2].view(8, 128)[0].isnan().all() and not a[2].view(8, 128)[1:].isnan().any()


def test_other_stream_and_captured_graph():
    need_gpu()
    c = Attention(2, 8, 2, 128, 6, 400, [0, 3, 400, 20, 170, 16], 300, 4, seed=9)
    want = c.run()
    assert torch.equal(want, c.run(stream=torch.cuda.Stream()))
    a = torch.zeros_like(c.q)
    ws = torch.empty(tp.tp_cache4_attn_workspace_size(c.plan, c.B, c.C, c.window, c.sinks), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_cache4_attn(c.plan, c.cols(c.q, 2), *c.args(), c.lens, c.window, c.sinks, c.cols(a, 2), ws)
    for _ in range(3):
        a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want)


def test_nothing_to_do():
    need_gpu()
    c = Cache(1, 1, 1, 64, 2, 4)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    c.store(e, e, ints(0, 0))
    tp.tp_cache4_load(c.plan, ints(0, 0), *c.args(), [e], [e])
    z = Cache(1, 1, 1, 64, 0, 4)
    tp.tp_cache4_attn(z.plan, [e], *z.args(), torch.empty(0, dtype=torch.int32, device="cuda"), 1, 0, [e])
