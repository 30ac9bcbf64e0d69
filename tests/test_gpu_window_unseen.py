"""tp_window_attn and keys that no query of the call sees: their memory may hold anything, NaN and infinities
among the values included, and the outputs keep their bits."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu
from test_gpu_window_attention import Case

pytestmark = pytest.mark.gpu

SHAPES = [  # tp, Hq, Hkv, d, T, S, window, sinks
    (1, 8, 2, 128, 100, 1500, 200, 4), (1, 8, 2, 64, 100, 1500, 200, 0), (8, 64, 8, 128, 1, 4100, 256, 4),
    (1, 8, 1, 128, 1, 700, 100, 15), (2, 8, 2, 64, 257, 900, 64, 17), (1, 4, 4, 128, 130, 1000, 100, 129),
    (1, 4, 4, 64, 300, 2000, 33, 350), (8, 32, 4, 128, 70, 1515, 64, 200), (1, 7, 1, 128, 111, 1000, 300, 2),
    (1, 1, 1, 64, 3, 5000, 1, 130), (2, 16, 2, 128, 2100, 4000, 384, 21), (1, 1, 1, 128, 2, 300, 5, 290),
    (1, 160, 8, 128, 520, 1300, 100, 1),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("views", [False, True])
def test_memory_of_keys_that_nobody_sees(shape, views):
    need_gpu()
    c = Case(*shape, views=views)
    want = c.run()
    j = torch.arange(c.S, device="cuda")
    unseen = (j <= c.S - c.T - c.window) & (j >= c.sinks)  # the first query's window starts behind them
    assert unseen.any() and torch.isfinite(want).all()
    for bad in (float("nan"), float("inf")):
        c.k[unseen], c.v[unseen] = bad, bad
        a = c.run()
        assert torch.equal(a, want)
    c.k[unseen] = c.v[unseen] = 0
    c.check(want)
    assert tp.tp_device_status()[0] == tp.TP_OK


def test_first_tokens_that_reach_into_the_window():
    """First tokens past the first query's window start: nothing is hidden, and nothing is lost."""
    need_gpu()
    for sinks in (95, 100, 101, 102, 117, 130, 400):
        c = Case(1, 4, 2, 128, 50, 150, 1, sinks, seed=sinks)  # the first window starts at key 100
        c.check(c.run())


def test_the_example_reads_back_what_a_chunk_sees():
    """A prompt's chunks read the window and the first tokens of the cache, not the whole of it, and what else is in
    the memory of the keys does not matter."""
    need_gpu()
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import long_context
    window, chunk, n, sinks = 100, 64, 900, 5
    load, rows, results = tp.tp_cache4_load, [], []

    def spy(plan, first, kc, ks, vc, vs, k_out, v_out, **kw):
        rows.append(k_out[0].shape[0])
        load(plan, first, kc, ks, vc, vs, k_out, v_out, **kw)

    tp.tp_cache4_load = spy
    try:
        for memory in (0.0, float("nan")):
            b = long_context.Block(batch=1, capacity=1000, window=window, sinks=sinks, seed=4)
            for t in b.kv:
                t.fill_(memory)
            g = torch.Generator(device="cuda").manual_seed(2)
            x = torch.randn(n, b.hidden, generator=g, device="cuda")
            b.prompt(0, x, torch.arange(n, dtype=torch.int32, device="cuda").expand(3, n), chunk=chunk)
            results.append(x)
    finally:
        tp.tp_cache4_load = load
    chunks = -(-n // chunk)
    assert sum(rows) <= 2 * chunks * (window + chunk + sinks)  # not of the order of n * chunks / 2
    assert torch.isfinite(results[0]).all() and torch.equal(*results)


def test_the_example_refuses_a_prompt_that_its_cache_does_not_hold():
    need_gpu()
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import long_context
    b = long_context.Block(batch=1, capacity=100)
    for n in (100, 101):
        x = torch.randn(n, b.hidden, device="cuda")
        positions = torch.arange(n, dtype=torch.int32, device="cuda").expand(3, n)
        if n <= 100:
            b.prompt(0, x, positions)
            continue
        with pytest.raises(ValueError, match="100 positions"):
            b.prompt(0, x, positions)
    assert tp.tp_device_status()[0] == tp.TP_OK
