"""tp_cache_evict against a per-sequence selection in Python: positions, lengths and copies are exact."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def expect(weights, length, budget, first, recent):
    """Kept positions of one (sequence, head), from the rule."""
    if length <= budget:
        return list(range(length))
    middle = range(first, length - recent)

    def rank(j):
        w = weights[j]
        return (-(w if w == w else float("-inf")), w != w, j)  # NaN below everything, -0 equal to 0

    best = sorted(middle, key=rank)[:budget - first - recent]
    return sorted(list(range(first)) + best + list(range(length - recent, length)))


class Cache:
    def __init__(self, tp_size, hkv, d, B, C, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq = max(hkv, tp_size)
        self.plan = tp.tp_plan_create(tp_size, self.hq * d, self.hq, hkv, d, tp_size)
        self.n = tp_size if hkv >= tp_size else 1
        self.h, self.d, self.B, self.C = hkv // self.n, d, B, C
        self.k, self.v = ([torch.randn(B * C, self.h * d, generator=g, device="cuda").bfloat16() for _ in range(self.n)]
                          for _ in range(2))
        self.w = [torch.rand(B * self.h, C, generator=g, device="cuda") for _ in range(self.n)]

    def outputs(self, rows, budget):
        new = lambda: [torch.full((self.B * rows, self.h * self.d), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
                       for _ in range(self.n)]
        return (new(), new(), [torch.full((self.B * self.h, rows), 9.0, device="cuda") for _ in range(self.n)],
                torch.full((self.B,), -5, dtype=torch.int32, device="cuda"),
                torch.full((self.n, self.B * self.h, budget), -7, dtype=torch.int32, device="cuda"))

    def check(self, lens, budget, first, recent, before, after, rows):
        """`before`: copies of (k, v, w); `after`: the call's outputs."""
        k, v, w = before
        ko, vo, wo, lo, kept = after
        torch.cuda.synchronize()
        assert lo.tolist() == [min(max(x, 0), self.C, budget) if x <= budget else min(x, self.C, budget) for x in lens]
        d = self.d
        for s in range(self.n):
            for b, length in enumerate(lens):
                length = min(max(length, 0), self.C)
                for h in range(self.h):
                    at = expect(w[s][b * self.h + h].tolist(), length, budget, first, recent)
                    got = kept[s, b * self.h + h].tolist()
                    assert got == at + [-1] * (budget - len(at)), (s, b, h)
                    src = torch.tensor([b * self.C + j for j in at], dtype=torch.int64, device="cuda")
                    cols = slice(h * d, (h + 1) * d)
                    for new, old in ((ko, k), (vo, v)):
                        assert torch.equal(new[s][b * rows:b * rows + len(at), cols], old[s][src, cols])
                    row = wo[s][b * self.h + h]
                    assert torch.equal(row[:len(at)].view(torch.int32), w[s][b * self.h + h][at].view(torch.int32))
                    assert (row[len(at):] == 0).all()


@pytest.mark.parametrize("tp_size,hkv,d,B,C,lens,budget,first,recent", [
    (1, 1, 128, 1, 1, [1], 1, 0, 0),
    (1, 2, 64, 2, 9, [9, 0], 4, 1, 1),
    (2, 2, 128, 3, 40, [40, 17, 16], 16, 4, 8),
    (2, 4, 8, 2, 33, [33, 32], 5, 0, 5),          # nothing between the first and the recent
    (4, 2, 72, 3, 100, [100, 99, 3], 60, 0, 0),   # replicated K/V, an odd head size
    (1, 1, 128, 2, 5000, [5000, 4097], 2100, 4, 64),
    (1, 1, 16, 1, 50000, [49999], 1000, 2, 30),   # more keys than shared memory holds
    (1, 3, 128, 2, 600, [600, 512], 512, 512, 0),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_against_rule(tp_size, hkv, d, B, C, lens, budget, first, recent, in_place):
    need_gpu()
    c = Cache(tp_size, hkv, d, B, C, seed=C + budget)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = tuple([t.clone() for t in x] for x in (c.k, c.v, c.w))
    if in_place:
        kept = torch.empty(c.n, B * c.h, budget, dtype=torch.int32, device="cuda")
        after = (c.k, c.v, c.w, lengths, kept)
        rows = C
    else:
        rows = min(budget, C) + 3
        after = c.outputs(rows, budget)
    tp.tp_cache_evict(c.plan, lengths, c.k, c.v, c.w, budget, first, recent, *after)
    c.check(lens, budget, first, recent, before, after, rows)
    if not in_place:  # rows past the new length are left alone
        for b, length in enumerate(lens):
            n = min(length, budget)
            assert (after[0][0][b * rows + n:(b + 1) * rows] == 7.0).all()


@pytest.mark.parametrize("values", [[0.0], [1.0, 1.0, 2.0], [0.0, -0.0, 1e-45, -1e-45], [float("nan"), 1.0, float("-inf")],
                                    [float("inf"), 3.0, float("-inf"), -2.0], [1.0, 1.0 + 2 ** -23, 1.0 - 2 ** -24]])
@pytest.mark.parametrize("length,budget", [(64, 20), (1000, 300), (2049, 2048)])
def test_ties_signs_and_special_weights(values, length, budget):
    need_gpu()
    c = Cache(1, 1, 64, 1, length, seed=3)
    g = torch.Generator().manual_seed(length)
    pick = torch.randint(0, len(values), (length,), generator=g)
    c.w[0][0].copy_(torch.tensor(values, dtype=torch.float32)[pick].cuda())
    before = tuple([t.clone() for t in x] for x in (c.k, c.v, c.w))
    after = c.outputs(budget, budget)
    lengths = torch.tensor([length], dtype=torch.int32, device="cuda")
    tp.tp_cache_evict(c.plan, lengths, c.k, c.v, c.w, budget, 2, 5, *after)
    c.check([length], budget, 2, 5, before, after, budget)


def test_bad_lengths_are_clamped_and_reported():
    need_gpu()
    c = Cache(1, 1, 64, 2, 30, seed=1)
    before = tuple([t.clone() for t in x] for x in (c.k, c.v, c.w))
    after = c.outputs(10, 10)
    tp.tp_cache_evict(c.plan, torch.tensor([31, -4], dtype=torch.int32, device="cuda"), c.k, c.v, c.w, 10, 1, 1, *after)
    c.check([30, 0], 10, 1, 1, before, after, 10)
    assert tp.tp_device_status()[0] == tp.TP_ERR_BAD_LENGTH
    assert tp.tp_device_status()[0] == tp.TP_OK


def test_strided_views_of_one_cache():
    need_gpu()
    B, C, d, hkv, tp_size = 3, 70, 64, 4, 4
    c = Cache(tp_size, hkv, d, B, C, seed=8)
    whole = [torch.randn(B * C, hkv * d, device="cuda").bfloat16() for _ in range(2)]
    c.k, c.v = ([t[:, r * d:(r + 1) * d] for r in range(tp_size)] for t in whole)
    before = ([t.clone() for t in c.k], [t.clone() for t in c.v], [t.clone() for t in c.w])
    lens = [70, 41, 40]
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept = torch.empty(c.n, B * c.h, 40, dtype=torch.int32, device="cuda")
    after = (c.k, c.v, c.w, lengths, kept)
    tp.tp_cache_evict(c.plan, lengths, c.k, c.v, c.w, 40, 0, 7, *after)
    c.check(lens, 40, 0, 7, before, after, C)
