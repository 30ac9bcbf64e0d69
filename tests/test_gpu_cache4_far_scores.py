"""tp_cache4_attn where a warp's first tile of keys scores -infinity in f32: such keys weigh nothing, and the keys
behind them are weighed by their own scores.

The far keys are -2^127 in every value and q is positive, so in 64 bits their scores lie 2^100 and more below the
others': their weights are 0, and the outputs are those over the other keys, within the tolerance that
test_gpu_cache4 derives. A head whose q is zero scores 0 on every key, the far ones too: its output is the mean
of the values within the same roundings (2^-8 each of the weights and of the output, 2^-18 for the joins)."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu
from test_gpu_cache4 import ALL, Attention, ints

pytestmark = pytest.mark.gpu

SHAPES = [  # tp, Hq, Hkv, d, B, C, keys, far ones
    (1, 8, 1, 128, 500, 200, 200, 128), (2, 8, 2, 64, 240, 300, 293, 130),   # a sequence's keys in one CTA
    (1, 20, 2, 128, 100, 333, 333, 150),                                     # two products of heads
    (1, 4, 2, 128, 2, 20000, 20000, 700), (1, 16, 1, 64, 1, 30000, 29990, 5000),  # splits, the first of far keys alone
    (1, 8, 2, 128, 3, 1000, 1000, 300),                                      # CTAs of a cluster
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("zero_head", [False, True])
def test_first_keys_far_below(shape, zero_head):
    need_gpu()
    tp_size, hq, hkv, d, B, C, n, far = shape
    c = Attention(tp_size, hq, hkv, d, B, C, [n] * B, ALL, 0, seed=11)
    k = c.kv[0].to(torch.bfloat16).view(B, C, -1)
    k[:, :far] = -2.0 ** 127
    c.store(k.view(B * C, -1), c.kv[1].to(torch.bfloat16), ints(*[0] * B))
    c.kv = [t.double() for t in c.load(ints(*[0] * B), C)]
    c.q = c.q.abs()
    group = hq // hkv
    if zero_head:
        c.q.view(B, hq, d)[:, group - 1] = 0
    a = c.run()
    assert torch.isfinite(a).all() and torch.equal(a, c.run())
    assert tp.tp_device_status()[0] == tp.TP_OK
    if zero_head:
        v = c.kv[1].view(B, C, hkv, d)[:, :n, 0]
        got = a.view(B, hq, d)[:, group - 1].double()
        want, mag = v.mean(1), v.abs().mean(1)
        assert ((got - want).abs() <= 1.02 * ((2.0 ** -8 + 2.0 ** -18) * mag + 2.0 ** -8 * want.abs())).all()
        a.view(B, hq, d)[:, group - 1] = 0
    c.window = n - far  # what is left of the keys
    c.check(a, skip={(b, 0) for b in range(B)} if zero_head else ())
    if zero_head:  # the first kv head's other heads: those of the same call without the zero one
        c.window, q = ALL, c.q.view(B, hq, d)
        q[:, group - 1] = 1
        same = c.run().view(B, hq, d)
        assert torch.equal(same[:, :group - 1], a.view(B, hq, d)[:, :group - 1])
