"""tp_window_attn against the softmax over the visible keys in float64.

Tolerances, from the roundings the call makes (u = 2^-24): a score is a sum of d exact products in f32,
off by at most (d / 16 + 16) * 2u of the sum of the products' sizes, and its scaling adds 4u of it; so a
softmax weight is off by at most twice the largest score error (its own and the normaliser's), plus 2^-18
for the exponentials and the joins of the splits. P is rounded to bf16 for P V (2^-8 of each p) and the
output is rounded once (2^-8)."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.bfloat16
ALL = 2 ** 31 - 1


class Case:
    def __init__(self, tp_size, hq, hkv, d, T, S, window, sinks, seed=0, q_std=1.0, views=False):
        g = torch.Generator(device="cuda").manual_seed(seed * 7919 + T * 31 + S)
        draw = lambda r, c, std=1.0: (torch.randn(r, c, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
        self.plan = tp.tp_plan_create(tp_size, hq * d, hq, hkv, d, tp_size)
        self.n, self.s = tp_size, tp_size if hkv >= tp_size else 1
        self.hq, self.hkv, self.d, self.T, self.S, self.window, self.sinks = hq, hkv, d, T, S, window, sinks
        self.q, self.k, self.v = draw(T, hq * d, q_std), draw(S, hkv * d), draw(S, hkv * d)
        self.views = views

    def parts(self, t, n):
        out = list(t.split(t.shape[1] // n, dim=1))
        return out if self.views else [x.contiguous() for x in out]

    def run(self, stream=None):
        q, k, v = self.parts(self.q, self.n), self.parts(self.k, self.s), self.parts(self.v, self.s)
        whole = torch.full_like(self.q, float("nan"))
        a = list(whole.split(whole.shape[1] // self.n, dim=1)) if self.views else [torch.full_like(x, float("nan")) for x in q]
        ws = torch.full((tp.tp_window_attn_workspace_size(self.plan, self.T, self.S, self.window, self.sinks),), 255,
                        dtype=torch.uint8, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        tp.tp_window_attn(self.plan, q, k, v, self.window, self.sinks, a, ws, stream=stream)
        torch.cuda.synchronize()
        return torch.cat(a, 1)

    def check(self, a, rows=None):
        d, G = self.d, self.hq // self.hkv
        j = torch.arange(self.S, device="cuda")
        step = 256
        for t0 in range(0, self.T, step):
            t1 = min(self.T, t0 + step)
            pos = torch.arange(self.S - self.T + t0, self.S - self.T + t1, device="cuda")[:, None]
            seen = ((j <= pos) & ((j > pos - self.window) | (j < self.sinks)))[:, None]
            for h in range(self.hkv):
                cols = slice(h * d, (h + 1) * d)
                k, v = self.k[:, cols].double(), self.v[:, cols].double()
                q = self.q[t0:t1, h * G * d:(h + 1) * G * d].reshape(-1, d).double()
                got = a[t0:t1, h * G * d:(h + 1) * G * d].reshape(-1, G, d).double()
                s = (q @ k.t() / d ** 0.5).view(t1 - t0, G, -1).masked_fill(~seen, float("-inf"))
                size = (q.abs() @ k.abs().t() / d ** 0.5).view(t1 - t0, G, -1).masked_fill(~seen, 0.0)
                ds = ((d / 16 + 16) * 2 * U * size + 4 * U * s.masked_fill(~seen, 0.0).abs()).amax(-1, keepdim=True)
                p = torch.softmax(s, -1)
                out, mag = p @ v, p @ v.abs()
                tol = (2.0 ** -8 + 2 * ds + 2.0 ** -18) * mag + 2.0 ** -8 * out.abs()
                assert ((got - out).abs() <= 1.02 * tol + 1e-30).all(), (t0, h, float(((got - out).abs() - tol).max()))


SHAPES = [  # tp, Hq, Hkv, d, T, S, window, sinks
    (1, 1, 1, 128, 1, 1, 1, 0), (1, 1, 1, 64, 1, 1, ALL, 5), (1, 8, 1, 128, 1, 700, 100, 4), (1, 2, 2, 64, 3, 3, 1, 0),
    (1, 4, 4, 128, 130, 130, ALL, 0), (2, 8, 2, 128, 257, 257, 128, 0), (2, 8, 2, 128, 257, 257, 129, 1), (1, 4, 2, 64, 300, 300, 17, 3),
    (8, 64, 8, 128, 129, 900, 256, 4), (8, 32, 4, 128, 70, 515, 64, 200),   # K/V replicated, a group on two ranks; many sinks
    (4, 12, 2, 64, 200, 333, 50, 130),                                      # six heads a group
    (1, 7, 1, 128, 111, 1000, 300, 2), (1, 20, 1, 64, 60, 61, 5, 5),        # groups that divide no tile
    (1, 2, 1, 128, 1500, 1500, 700, 140), (1, 300, 1, 64, 3, 5, 2, 1),      # a group of more than two tiles
    (1, 1, 1, 128, 1000, 1000, 1, 0), (1, 1, 1, 128, 1000, 1000, 2, 1),     # a window of one key: every row its own
    (2, 4, 2, 128, 2100, 2100, 384, 0), (1, 16, 2, 64, 2, 20000, ALL, 0), (1, 16, 2, 128, 1, 20000, 8000, 4000),
    (1, 1, 1, 64, 128, 4096, 128, 128), (1, 1, 1, 64, 128, 4095, 129, 129),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("views", [False, True])
def test_against_softmax(shape, views):
    need_gpu()
    c = Case(*shape, views=views)
    a = c.run()
    c.check(a)
    assert tp.tp_device_status()[0] == tp.TP_OK
    assert torch.equal(a, c.run())  # the same bits every time


@pytest.mark.parametrize("q_std", [4.0, 30.0])
def test_sharp_scores(q_std):
    need_gpu()
    c = Case(2, 16, 2, 128, 400, 700, 150, 3, seed=2, q_std=q_std)
    c.check(c.run())


def test_maxima_that_jump_behind_masked_blocks():
    """Rows whose first block is masked, and whose block maxima rise and fall by tens of log2 units."""
    need_gpu()
    c = Case(1, 4, 1, 128, 1200, 1200, 500, 4, seed=5)
    ramp = torch.arange(1200, device="cuda")[:, None] // 128 * 1.3
    c.k += (ramp * torch.sign(c.q[0, :128].float())).to(BF16)
    c.k[:4] -= (9 * torch.sign(c.q[0, :128].float())).to(BF16)
    c.check(c.run())


def test_a_wide_window_is_causal_attention():
    need_gpu()
    c = Case(2, 8, 2, 128, 777, 777, ALL, 0, seed=3)
    a = c.run()
    assert torch.equal(a, Case(2, 8, 2, 128, 777, 777, 777, 0, seed=3).run())
    want = [torch.empty_like(x) for x in c.parts(c.q, 2)]
    ws = torch.empty(tp.tp_attn_core_workspace_size(c.plan, 777), dtype=torch.uint8, device="cuda")
    tp.tp_attn_core(c.plan, c.parts(c.q, 2), c.parts(c.k, 2), c.parts(c.v, 2), want, True, ws)
    # both are within a rounding of P and one of A of the same softmax
    assert ((torch.cat(want, 1).float() - a.float()).abs() <= 4 * 2.0 ** -8 * c.v.float().abs().max()).all()


def test_keys_out_of_sight_do_not_matter():
    need_gpu()
    c = Case(1, 8, 2, 128, 100, 1500, 200, 4, seed=6)
    want = c.run()
    # blocks of 128 keys that no query sees: not read at all
    c.k[128:1100], c.v[128:1100] = float("nan"), float("inf")
    assert torch.equal(want, c.run())
    # keys beside seen ones in a block: any scores
    c.k[4:128], c.k[1100:1201] = float("nan"), float("inf")
    assert torch.equal(want, c.run())


def test_nan_of_a_row_spoils_only_itself():
    need_gpu()
    c = Case(1, 8, 2, 128, 300, 300, 64, 0, seed=7)
    want = c.run()
    c.q[5, 3] = float("nan")
    a = c.run()
    assert a[5, :128].isnan().all()
    a[5, :128] = want[5, :128]
    assert torch.equal(a, want)


def test_other_stream_and_captured_graph():
    need_gpu()
    for shape in ((2, 8, 2, 128, 6, 900, 300, 4), (2, 8, 2, 64, 900, 900, 300, 4)):  # joined splits, and none
        c = Case(*shape, seed=9)
        want = c.run()
        assert torch.equal(want, c.run(stream=torch.cuda.Stream()))
        q, k, v = c.parts(c.q, 2), c.parts(c.k, 2), c.parts(c.v, 2)
        a = [torch.zeros_like(x) for x in q]
        ws = torch.empty(tp.tp_window_attn_workspace_size(c.plan, c.T, c.S, c.window, c.sinks), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tp.tp_window_attn(c.plan, q, k, v, c.window, c.sinks, a, ws)
        for _ in range(3):
            for x in a:
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(torch.cat(a, 1), want)


def test_nothing_beside_the_output_is_written():
    need_gpu()
    c = Case(1, 4, 2, 128, 133, 200, 50, 1, seed=11)
    buf = torch.full((140, 4 * 128 + 16), 3.0, device="cuda", dtype=BF16)
    tp.tp_window_attn(c.plan, [c.q], [c.k], [c.v], 50, 1, [buf[:133, 8:520]],
                      torch.empty(tp.tp_window_attn_workspace_size(c.plan, 133, 200, 50, 1), dtype=torch.uint8, device="cuda"))
    c.check(buf[:133, 8:520])
    assert (buf[133:] == 3).all() and (buf[:, :8] == 3).all() and (buf[:, 520:] == 3).all()


def test_no_tokens():
    need_gpu()
    plan = tp.tp_plan_create(1, 128, 1, 1, 128, 1)
    e, k = torch.empty(0, 128, device="cuda", dtype=BF16), torch.ones(5, 128, device="cuda", dtype=BF16)
    tp.tp_window_attn(plan, [e], [k], [k], 4, 0, [e])


def test_sources_that_overlap():
    """Two sources' keys in one buffer, the second a row on: each has its own pitch of one source."""
    need_gpu()
    c = Case(2, 4, 2, 64, 30, 90, 20, 2)
    buf = torch.randn(91, 64, device="cuda").to(BF16)
    plan, q = c.plan, c.parts(c.q, 2)
    ws = torch.empty(tp.tp_window_attn_workspace_size(plan, 30, 90, 20, 2), dtype=torch.uint8, device="cuda")
    got, want = ([torch.zeros_like(x) for x in q] for _ in range(2))
    shared = [buf[:90], buf[1:]]
    tp.tp_window_attn(plan, q, shared, shared, 20, 2, got, ws)
    apart = [x.clone() for x in shared]
    tp.tp_window_attn(plan, q, apart, [x.clone() for x in apart], 20, 2, want, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


# As many items as fill the SMs, of two row tiles each, and items of two row tiles in splits
FULL = [(1, 64, 32, 64, 560, 700, 130, 20), (8, 64, 8, 128, 2450, 2600, 200, 4), (1, 32, 4, 64, 3000, 3000, 333, 0),
        (1, 32, 4, 128, 5000, 5000, ALL, 0), (2, 152, 152, 128, 40, 300, 70, 9), (1, 152, 152, 64, 255, 2000, 1500, 300),
        (1, 32, 8, 128, 512, 5000, 4096, 0), (1, 8, 8, 128, 600, 9000, ALL, 0), (4, 64, 2, 64, 700, 6000, 5000, 33)]


@pytest.mark.parametrize("shape", FULL, ids=lambda s: "-".join(map(str, s)))
def test_many_rows(shape):
    need_gpu()
    c = Case(*shape, seed=12)
    a = c.run()
    c.check(a)
    assert tp.tp_device_status()[0] == tp.TP_OK
    assert torch.equal(a, c.run())


@pytest.mark.parametrize("q_std", [4.0, 30.0])
def test_many_rows_with_sharp_scores(q_std):
    need_gpu()
    c = Case(2, 64, 16, 128, 1210, 1300, 150, 3, seed=13, q_std=q_std)
    c.check(c.run())


def test_many_rows_with_maxima_that_jump():
    need_gpu()
    c = Case(1, 64, 16, 128, 1200, 1200, 500, 4, seed=14)
    ramp = torch.arange(1200, device="cuda")[:, None] // 128 * 1.3
    c.k += (ramp * torch.sign(c.q[0, :128].float()).repeat(16)).to(BF16)
    c.k[:4] -= (9 * torch.sign(c.q[0, :128].float()).repeat(16)).to(BF16)
    c.check(c.run())


def test_many_rows_out_of_sight_and_nan():
    need_gpu()
    c = Case(1, 64, 16, 64, 1300, 3000, 200, 4, seed=15)
    want = c.run()
    c.k[128:1400], c.v[128:1400] = float("nan"), float("inf")  # blocks that no query sees
    c.k[4:128] = float("nan")
    assert torch.equal(want, c.run())
    c.q[700, 3] = float("nan")
    a = c.run()
    assert a[700, :64].isnan().all()
    a[700, :64] = want[700, :64]
    assert torch.equal(a, want)


def test_many_rows_in_a_graph():
    need_gpu()
    c = Case(2, 64, 16, 128, 900, 900, 300, 4, seed=16)
    want = c.run()
    assert torch.equal(want, c.run(stream=torch.cuda.Stream()))
    q, k, v = c.parts(c.q, 2), c.parts(c.k, 2), c.parts(c.v, 2)
    a = [torch.zeros_like(x) for x in q]
    assert tp.tp_window_attn_workspace_size(c.plan, 900, 900, 300, 4) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_window_attn(c.plan, q, k, v, 300, 4, a, None)
    for _ in range(3):
        for x in a:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(a, 1), want)
