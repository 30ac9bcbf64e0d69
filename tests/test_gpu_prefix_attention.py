"""tp_prefix_attn against the softmax over prefix and own keys in float64.

Tolerances, from the roundings the call makes (u = 2^-24): a score is a sum of d exact products
in f32, off by at most (d / 16 + 16) * 2u of the sum of the products' sizes, and its scaling adds
4u of it; so a softmax weight is off by at most twice the largest score error (its own and the
normaliser's), plus 2^-18 for the exponentials and the joins of the splits. P is rounded to bf16
for P V (2^-8 of each p) and the output is rounded once (2^-8). An accumulated weight adds its
group's weights in f32."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.bfloat16


class Case:
    def __init__(self, tp_size, hq, hkv, d, B, P, C, lens, seed=0, q_std=1.0, views=False):
        g = torch.Generator(device="cuda").manual_seed(seed * 7919 + B * 31 + P + C)
        draw = lambda r, c, std=1.0: (torch.randn(r, c, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
        self.plan = tp.tp_plan_create(tp_size, hq * d, hq, hkv, d, tp_size)
        self.n, self.s = tp_size, tp_size if hkv >= tp_size else 1
        self.hq, self.hkv, self.d, self.B, self.P, self.C = hq, hkv, d, B, P, C
        self.q = draw(B, hq * d, q_std)
        self.kp, self.vp, self.ko, self.vo = draw(P, hkv * d), draw(P, hkv * d), draw(B * C, hkv * d), draw(B * C, hkv * d)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.w = torch.rand(self.s, B * (hkv // self.s), C, generator=g, device="cuda")
        self.views = views

    def parts(self, t, n):
        out = list(t.split(t.shape[1] // n, dim=1))
        return out if self.views else [x.contiguous() for x in out]

    def run(self, weights=True, alias=False, stream=None, first=False):
        q = self.parts(self.q, self.n)
        kv = [self.parts(t, self.s) for t in (self.kp, self.vp, self.ko, self.vo)]
        whole = torch.full_like(self.q, float("nan"))
        a = list(whole.split(whole.shape[1] // self.n, dim=1)) if self.views else [torch.full_like(x, float("nan")) for x in q]
        ws = torch.empty(tp.tp_prefix_attn_workspace_size(self.plan, self.B, self.P, self.C, weights), dtype=torch.uint8,
                         device="cuda")
        wi = list(self.w.clone())
        wo = (wi if alias else [torch.full_like(x, float("nan")) for x in wi]) if weights else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        tp.tp_prefix_attn(self.plan, q, *kv, self.lens, a, ws, weight_in=wi if weights and not first else None, weight_out=wo,
                          stream=stream)
        torch.cuda.synchronize()
        return torch.cat(a, 1), None if wo is None else torch.stack(wo)

    def check(self, a, w, first=False, skip=()):
        d, G, hr = self.d, self.hq // self.hkv, self.hkv // self.s
        for b in range(self.B):
            n = min(max(int(self.lens[b]), 0), self.C)
            for h in range(self.hkv):
                if (b, h) in skip:
                    continue
                cols = slice(h * d, (h + 1) * d)
                own = slice(b * self.C, b * self.C + n)
                k = torch.cat([self.kp[:, cols], self.ko[own, cols]]).double()
                v = torch.cat([self.vp[:, cols], self.vo[own, cols]]).double()
                q = self.q[b].view(self.hq, d)[h * G:(h + 1) * G].double()
                got = a[b].view(self.hq, d)[h * G:(h + 1) * G].double()
                if self.P + n == 0:
                    assert (got == 0).all()
                    p = torch.zeros(G, 0, dtype=torch.float64, device="cuda")
                    rel = torch.zeros(G, 1, device="cuda")
                else:
                    s = q @ k.t() / d ** 0.5
                    ds = ((d / 16 + 16) * 2 * U * (q.abs() @ k.abs().t()) / d ** 0.5 + 4 * U * s.abs()).amax(1, keepdim=True)
                    p = torch.softmax(s, dim=1)
                    out = p @ v
                    rel = 2 * ds + 2.0 ** -18
                    tol = (2.0 ** -8 + rel) * (p @ v.abs()) + 2.0 ** -8 * out.abs()
                    assert ((got - out).abs() <= 1.02 * tol + 1e-30).all(), (b, h, float(((got - out).abs() - tol).max()))
                if w is not None:
                    row = w[h // hr, b * hr + h % hr].double()
                    ref = p[:, self.P:].sum(0)
                    tol = (p[:, self.P:] * rel).sum(0) + (G + 2) * U * ref
                    if not first:
                        ref = ref + self.w[h // hr, b * hr + h % hr, :n].double()
                        tol = tol + U * ref
                    assert ((row[:n] - ref).abs() <= 1.02 * tol + 1e-30).all()
                    assert (row[n:] == 0).all()


SHAPES = [  # tp, Hq, Hkv, d, B, P, C, lengths
    (1, 1, 1, 128, 1, 1, 1, [0]), (1, 1, 1, 128, 1, 0, 1, [1]), (1, 2, 1, 64, 2, 0, 3, [0, 3]),
    (1, 4, 4, 128, 3, 127, 0, [0, 0, 0]), (1, 16, 4, 128, 1, 100, 64, [33]), (2, 8, 2, 64, 5, 300, 70, [0, 1, 69, 70, 16]),
    (4, 8, 4, 128, 3, 129, 200, [200, 63, 65]), (8, 64, 8, 128, 9, 515, 130, [0, 5, 64, 128, 129, 130, 17, 16, 15]),
    (8, 32, 4, 128, 6, 1024, 40, [1, 2, 3, 38, 39, 40]),   # K/V replicated, a group on two ranks
    (4, 12, 2, 64, 4, 250, 33, [33, 0, 7, 32]),            # six heads a group, replicated
    (2, 6, 2, 128, 50, 384, 65, [i % 66 for i in range(50)]),  # three heads a group, two row tiles
    (1, 40, 2, 128, 2, 130, 600, [600, 513]),              # twenty heads a group: two 16-head tiles
    (1, 7, 1, 128, 40, 1000, 20, [20 - i % 21 for i in range(40)]),
    (1, 2, 2, 128, 2, 20000, 1100, [1100, 1023]),          # many splits of both parts
    (1, 8, 1, 64, 100, 2050, 5, [i % 6 for i in range(100)]),  # 800 rows: four tile pairs
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:7])))
@pytest.mark.parametrize("views", [False, True])
def test_against_softmax(shape, views):
    need_gpu()
    c = Case(*shape, views=views)
    a, w = c.run()
    c.check(a, w)
    assert tp.tp_device_status()[0] == tp.TP_OK
    a2, w2 = c.run(alias=True)  # weights accumulated in place; the same bits
    assert torch.equal(a, a2) and torch.equal(w, w2)
    a3, _ = c.run(weights=False)
    assert torch.equal(a, a3)
    a4, w4 = c.run(first=True)
    assert torch.equal(a, a4)
    c.check(a4, w4, first=True)


@pytest.mark.parametrize("q_std", [4.0, 30.0])
def test_sharp_scores(q_std):
    need_gpu()
    c = Case(2, 16, 2, 128, 4, 700, 150, [150, 0, 77, 64], seed=2, q_std=q_std)
    c.check(*c.run())


def test_block_maxima_that_jump():
    """Rows whose block maxima rise by tens of log2 units, so the reference maximum lags and then moves."""
    need_gpu()
    c = Case(1, 4, 1, 128, 70, 128 * 12, 300, [300 - i for i in range(70)], seed=5)
    ramp = torch.arange(12, device="cuda").repeat_interleave(128)[:, None] * 1.3
    c.kp += (ramp * torch.sign(c.q[0, :128].float())).to(BF16)
    c.ko += (torch.linspace(0, 8, c.B * c.C, device="cuda")[:, None] * torch.sign(c.q[1, :128].float())).to(BF16)
    c.check(*c.run())


def test_stale_rows_past_the_length_do_not_matter():
    need_gpu()
    c = Case(1, 8, 2, 128, 4, 60, 90, [0, 13, 64, 90], seed=6)
    want = c.run()
    for b, n in enumerate(c.lens.tolist()):
        c.ko[b * 90 + n:(b + 1) * 90] = float("nan")
        c.vo[b * 90 + n:(b + 1) * 90] = float("inf")
        c.w[:, b * 2:(b + 1) * 2, n:] = float("nan")
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_sequence_with_nan_spoils_only_itself():
    need_gpu()
    c = Case(1, 8, 2, 128, 3, 200, 50, [50, 50, 20], seed=7)
    c.vo[50 + 3, 5] = float("nan")          # sequence 1, kv head 0
    a, w = c.run()
    assert torch.isnan(a[1].view(8, 128)[:4, 5].float()).all()
    c.check(a, w, skip={(1, 0)})


def test_bad_lengths_are_clamped_and_reported():
    need_gpu()
    for C, lens in ((20, [21, -1]), (0, [0, 4])):
        c = Case(1, 4, 2, 64, 2, 40, C, lens)
        a, w = c.run()
        c.check(a, w)
        assert tp.tp_device_status()[0] == tp.TP_ERR_BAD_LENGTH
        assert tp.tp_device_status()[0] == tp.TP_OK


def test_other_stream_and_captured_graph():
    need_gpu()
    c = Case(2, 8, 2, 128, 6, 300, 40, [0, 3, 40, 20, 17, 16], seed=9)
    want = c.run()
    side = torch.cuda.Stream()
    got = c.run(stream=side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    q = c.parts(c.q, 2)
    kv = [c.parts(t, 2) for t in (c.kp, c.vp, c.ko, c.vo)]
    a = [torch.zeros_like(x) for x in q]
    ws = torch.empty(tp.tp_prefix_attn_workspace_size(c.plan, c.B, c.P, c.C, False), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_prefix_attn(c.plan, q, *kv, c.lens, a, ws)
    for _ in range(3):
        for x in a:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(a, 1), want[0])


# Which kernels a call takes goes by its sizes: one launch of clusters for few keys and sequences
# with at most 16 heads a group, else the prefix, own and joining kernels. Both sides of each limit.
EDGES = [
    (1, 16, 1, 128, 1, 8128, 64, [64]),                     # 128 tiles over eight CTAs: the most
    (1, 16, 1, 64, 1, 8129, 64, [64]),                      # one more
    (1, 4, 1, 128, 1, 0, 8192, [8191]), (1, 4, 1, 64, 2, 0, 8193, [8193, 0]),
    (1, 8, 1, 128, 150, 700, 270, [i * 9 % 271 for i in range(150)]),   # a CTA a sequence, 16 tiles
    (2, 16, 2, 64, 77, 960, 128, [i * 5 % 129 for i in range(77)]),     # more units than SMs
    (1, 17, 1, 128, 3, 200, 300, [0, 300, 65]),             # 17 heads
    (1, 8, 4, 128, 1, 65, 64 * 11 + 1, [64 * 11]),          # tiles that do not divide by the CTAs
    (8, 16, 4, 64, 3, 64, 64, [0, 64, 1]), (1, 3, 3, 128, 2, 128, 2048, [1, 2047]),
]


@pytest.mark.parametrize("shape", EDGES, ids=lambda s: "-".join(map(str, s[:7])))
def test_both_sides_of_the_kernels_limits(shape):
    need_gpu()
    c = Case(*shape, seed=21, views=True)
    a, w = c.run()
    c.check(a, w)
    a2, w2 = c.run(alias=True)
    assert torch.equal(a, a2) and torch.equal(w, w2)
    a3, _ = c.run(weights=False)
    assert torch.equal(a, a3)
    c.check(*c.run(first=True), first=True)
    assert tp.tp_device_status()[0] == tp.TP_OK


WAYS = [(1, 8, 2, 128, 5, 300, 130), (1, 34, 2, 128, 5, 300, 130), (1, 8, 2, 64, 5, 0, 130), (1, 34, 2, 64, 5, 0, 130)]


@pytest.mark.parametrize("shape", WAYS, ids=lambda s: "-".join(map(str, s)))
def test_stale_rows_bad_lengths_and_nan_in_both_ways(shape):
    need_gpu()
    c = Case(*shape, [0, 13, 64, 130, 99], seed=22)
    want = c.run()
    for b, n in enumerate(c.lens.tolist()):
        c.ko[b * 130 + n:(b + 1) * 130] = float("inf")
        c.vo[b * 130 + n:(b + 1) * 130] = float("nan")
        c.w[:, b * 2:(b + 1) * 2, n:] = float("nan")
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert tp.tp_device_status()[0] == tp.TP_OK
    c.lens[0] = -7
    c.lens[3] = 131
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])  # clamped to 0 and to the capacity
    assert tp.tp_device_status()[0] == tp.TP_ERR_BAD_LENGTH
    assert tp.tp_device_status()[0] == tp.TP_OK
    c.lens[0], c.lens[3] = 0, 130
    c.ko[2 * 130 + 63, 7] = float("nan")     # sequence 2, kv head 0
    a, w = c.run()
    group = c.hq // 2
    assert torch.isnan(a[2].view(c.hq, c.d)[:group].float()).all()
    keep = torch.ones(5, c.hq, dtype=torch.bool, device="cuda")
    keep[2, :group] = False
    assert torch.equal(a.view(5, c.hq, c.d)[keep], want[0].view(5, c.hq, c.d)[keep])


def test_long_scores_that_jump_in_both_ways():
    """The maxima rise from tile to tile by tens of log2 units, over the CTAs of a cluster and over splits."""
    need_gpu()
    for hq in (4, 17):
        c = Case(1, hq, 1, 128, 2, 64 * 9, 64 * 7, [64 * 7, 100], seed=23)
        ramp = torch.arange(9, device="cuda").repeat_interleave(64)[:, None] * 1.3
        c.kp += (ramp * torch.sign(c.q[0, :128].float())).to(BF16)
        c.ko += (torch.linspace(8, 0, c.B * c.C, device="cuda")[:, None] * torch.sign(c.q[1, :128].float())).to(BF16)
        c.check(*c.run())


def test_eviction_reads_the_accumulated_weights():
    need_gpu()
    c = Case(2, 8, 2, 128, 3, 100, 64, [64, 50, 10], seed=11)
    a, w = c.run()
    kv = [c.parts(t, 2) for t in (c.ko, c.vo)]
    kept = torch.empty(2, 3, 32, dtype=torch.int32, device="cuda")
    lens = c.lens.clone()
    before = [t.clone() for t in kv[0]]
    wl = list(w)
    tp.tp_cache_evict(c.plan, lens, kv[0], kv[1], wl, 32, 2, 8, kv[0], kv[1], wl, lens, kept)
    torch.cuda.synchronize()
    assert lens.tolist() == [32, 32, 10]
    for s in range(2):
        at = kept[s, 1].long()
        assert torch.equal(kv[0][s][64:96], before[s][64 + at])


# One prefix-free batch per kernel route: clusters of one launch (groups of at most 16 heads), and the
# three kernels (17 heads). The last own key is alone in its warp's share, with every count of keys.
@pytest.mark.parametrize("length", [1, 17, 33, 49, 65, 97, 129, 130])
@pytest.mark.parametrize("hq, P", [(8, 0), (34, 0), (8, 70), (34, 70)])
def test_a_nan_in_the_last_own_key_reaches_the_output(hq, P, length):
    need_gpu()
    c = Case(1, hq, 2, 128, 5, P, 130, [64, length, 130, length, 13], seed=31)
    want, w_want = c.run()
    c.ko[130 + length - 1, 5] = float("nan")   # sequence 1, kv head 0
    a, w = c.run()
    group = hq // 2
    assert torch.isnan(a[1].view(hq, 128)[:group].float()).all()
    assert torch.isnan(w[0, 2, :length]).all() and (w[0, 2, length:] == 0).all()
    keep = torch.ones(5, hq, dtype=torch.bool, device="cuda")
    keep[1, :group] = False
    assert torch.equal(a.view(5, hq, 128)[keep], want.view(5, hq, 128)[keep])
    rows = [i for i in range(10) if i != 2]
    assert torch.equal(w[0, rows], w_want[0, rows])


def check_hidden(c, hide_prefix, hide_own):
    """Keys that every q row scores with -inf (through channel 0) have weight 0, as in the definition;
    rows of such keys alone divide 0 by 0. hide_prefix: [P], hide_own: [B, C] truth values."""
    d, G, hr = c.d, c.hq // c.hkv, c.hkv // c.s
    c.q.view(c.B, c.hq, d)[:, :, 0] = 1.0
    finite = c.kp.clone(), c.ko.clone()
    c.kp.view(c.P, c.hkv, d)[hide_prefix, :, 0] = float("-inf")
    c.ko.view(c.B, c.C, c.hkv, d)[hide_own, :, 0] = float("-inf")
    a, w = c.run(first=True)
    for b in range(c.B):
        n = min(max(int(c.lens[b]), 0), c.C)
        hidden = torch.cat([hide_prefix, hide_own[b, :n]])
        for h in range(c.hkv):
            cols = slice(h * d, (h + 1) * d)
            own = slice(b * c.C, b * c.C + n)
            k = torch.cat([finite[0][:, cols], finite[1][own, cols]]).double()
            v = torch.cat([c.vp[:, cols], c.vo[own, cols]]).double()
            q = c.q[b].view(c.hq, d)[h * G:(h + 1) * G].double()
            got = a[b].view(c.hq, d)[h * G:(h + 1) * G].double()
            row = w[h // hr, b * hr + h % hr].double()
            if len(hidden) == 0:
                assert (got == 0).all() and (row == 0).all()
                continue
            if bool(hidden.all()):
                assert torch.isnan(got).all() and torch.isnan(row[:n]).all()
                continue
            s = q @ k.t() / d ** 0.5
            ds = ((d / 16 + 16) * 2 * U * (q.abs() @ k.abs().t()) / d ** 0.5 + 4 * U * s.abs()).amax(1, keepdim=True)
            rel = 2 * ds + 2.0 ** -18
            p = torch.softmax(s.masked_fill(hidden, float("-inf")), dim=1)
            out = p @ v
            tol = (2.0 ** -8 + rel) * (p @ v.abs()) + 2.0 ** -8 * out.abs()
            assert ((got - out).abs() <= 1.02 * tol + 1e-30).all(), (b, h)
            ref = p[:, c.P:].sum(0)
            tol = (p[:, c.P:] * rel).sum(0) + (G + 2) * U * ref
            assert ((row[:n] - ref).abs() <= 1.02 * tol + 1e-30).all(), (b, h)
            assert (row[n:] == 0).all()


# What is hidden: the prefix's first keys (a whole first block and more splits than a warp joins at a
# time), runs of own keys that fill a warp's share or a whole split, and every key of one sequence.
@pytest.mark.parametrize("shape, first, own", [
    ((1, 8, 2, 128, 3, 300, 130, [130, 77, 0]), 200, (0, 64)),
    ((1, 8, 2, 64, 3, 0, 130, [130, 77, 64]), 0, (0, 64)),              # the third sequence has hidden keys alone
    ((1, 34, 2, 128, 5, 300, 130, [130, 77, 64, 0, 33]), 200, (0, 64)),
    ((1, 34, 2, 64, 5, 0, 130, [130, 77, 64, 0, 33]), 0, (0, 64)),
    ((1, 34, 2, 128, 5, 300, 130, [130, 77, 64, 0, 33]), 300, (32, 96)),
    ((1, 20, 1, 128, 100, 6000, 64, [i % 65 for i in range(100)]), 140, (0, 32)),   # three blocks of keys an item
    ((2, 2, 2, 128, 1, 20000, 64, [50]), 16000, (0, 50)),               # over 32 splits of the prefix are hidden
    ((1, 2, 1, 128, 1, 0, 20000, [19990]), 0, (0, 15000)),              # and of the own keys
], ids=lambda v: "-".join(map(str, v[:7] if type(v) is tuple else [v])))
def test_keys_that_score_minus_infinity_have_no_weight(shape, first, own):
    need_gpu()
    c = Case(*shape, seed=32)
    hide_prefix = torch.arange(c.P, device="cuda") < first
    at = torch.arange(c.C, device="cuda")
    check_hidden(c, hide_prefix, ((at >= own[0]) & (at < own[1])).expand(c.B, -1))


# Shapes by the path of the prefix kernel that they take, with the launches of a call: items of several
# 128-key blocks, two row tiles or one in the last pair, and more items than CTAs (a CTA's second item
# uses the Q tiles, the O columns and the barriers again).
ROUTES = [  # tp, Hq, Hkv, d, B, P, C, launches
    (1, 20, 1, 128, 100, 6000, 64, 3),     # 47 blocks in 16 splits, 2000 rows: 8 pairs, the last of 208 rows
    (2, 24, 4, 64, 170, 4000, 20, 3),      # 32 blocks in 8 splits, 1020 rows
    (1, 8, 2, 64, 180, 9000, 32, 3),       # 71 blocks in 24 splits, 720 rows: 208 in the last pair
    (4, 4, 4, 128, 340, 5000, 0, 2),       # no own caches: 40 blocks in 14 splits, 340 rows: 84 in the last pair
    (8, 128, 8, 64, 330, 400, 8, 3),       # 168 items of four blocks: some CTAs take two
    (1, 128, 8, 128, 322, 500, 8, 3),      # the same, one row tile in a head's last pair
    (1, 320, 8, 128, 37, 1500, 2000, 3),   # long own caches leave the prefix 38 CTAs
    (1, 4, 1, 128, 1, 100, 30, 1),
]


@pytest.mark.parametrize("shape", ROUTES, ids=lambda s: "-".join(map(str, s)))
def test_prefix_items_of_several_blocks_and_several_items(shape):
    need_gpu()
    *sizes, launches = shape
    B, C = sizes[4], sizes[6]
    c = Case(*sizes, [(i * 37 + 5) % (C + 1) for i in range(B)], seed=41)
    # the maxima of neighbouring blocks rise by over 64 log2 units for the first sequence's first head
    # and move up and down by less for the others
    ramp = ((torch.arange(c.P, device="cuda") // 128) % 3)[:, None] * 6.0
    for h in range(c.hkv):
        cols = slice(h * c.d, (h + 1) * c.d)
        q = c.q[0, h * (c.hq // c.hkv) * c.d:][:c.d].float()
        c.kp[:, cols] += (ramp * torch.sign(q)).to(BF16)
    before = tp.tp_launch_count()
    a, w = c.run()
    assert tp.tp_launch_count() - before == launches
    c.check(a, w)
    a2, w2 = c.run(alias=True)
    assert torch.equal(a, a2) and torch.equal(w, w2)
    assert tp.tp_device_status()[0] == tp.TP_OK


@pytest.mark.parametrize("q_std", [4.0, 30.0])
def test_sharp_scores_through_the_three_kernels(q_std):
    need_gpu()
    c = Case(2, 36, 2, 128, 90, 7000, 150, [(i * 29) % 151 for i in range(90)], seed=42, q_std=q_std)
    before = tp.tp_launch_count()
    a, w = c.run()
    assert tp.tp_launch_count() - before == 3
    c.check(a, w)
