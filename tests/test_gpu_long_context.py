"""The calls for long contexts as they are used together: a prompt in chunks through rotary positions, the
4-bit cache and window attention, then single tokens over the cache; in captured graphs, on several
streams, with a workspace that two graphs share.

Tolerances. What two calls compute from the same values agrees within both calls' roundings of the
weights (2^-8 each) and of the output (2^-8 each); where one of them takes the cache's values rounded to bf16,
that rounding moves a score by at most 2^-8 of its products' sizes and a value by 2^-8."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ALL = 2 ** 31 - 1


def block(**kw):
    import long_context
    return long_context.Block(**kw)


def columns(t, n):
    return list(t.split(t.shape[1] // n, dim=1))


def heads_attention(q, k, v, group, d, seen):
    """float64 softmax attention of [T x Hq*d] over [S x Hkv*d], and the weights' share of |v| and score sizes."""
    T, S = q.shape[0], k.shape[0]
    qh = q.double().view(T, -1, group, d).permute(1, 2, 0, 3)
    kh, vh = (t.double().view(S, -1, d).transpose(0, 1)[:, None] for t in (k, v))
    s = (qh @ kh.transpose(2, 3) / d ** 0.5).masked_fill(~seen, float("-inf"))
    p = torch.softmax(s, -1)
    size = ((qh.abs() @ kh.abs().transpose(2, 3)) / d ** 0.5).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
    back = lambda x: x.permute(2, 0, 1, 3).reshape(T, -1)  # noqa: E731
    return back(p @ vh), back(p @ vh.abs()), back(size.expand(-1, -1, -1, d))


@pytest.mark.parametrize("kv_heads, ranks, d", [(4, 2, 128), (2, 4, 64)])
def test_prompt_then_tokens(kv_heads, ranks, d):
    """Every call's output against float64 on the inputs that the call had."""
    need_gpu()
    q_heads, window, sinks = 8, 70, 3
    b = block(batch=2, ranks=ranks, hidden=512, q_heads=q_heads, kv_heads=kv_heads, head_dim=d, capacity=400, window=window, sinks=sinks,
              sections=(8, 12, 12), seed=3)
    group, seen_calls = q_heads // kv_heads, []
    window_attn, cache_attn, load = tp.tp_window_attn, tp.tp_cache4_attn, tp.tp_cache4_load

    def spy_window(plan, q, k, v, w, s, a, ws, **kw):
        window_attn(plan, q, k, v, w, s, a, ws, **kw)
        T, S = q[0].shape[0], k[0].shape[0]
        pos = torch.arange(S - T, S, device="cuda")[:, None]
        j = torch.arange(S, device="cuda")
        want, mag, _ = heads_attention(torch.cat(q, 1), torch.cat(k, 1), torch.cat(v, 1), group, d,
                                       (j <= pos) & ((j > pos - w) | (j < s)))
        assert ((torch.cat(a, 1).double() - want).abs() <= 1.05 * 2.0 ** -8 * (mag + want.abs()) + 1e-3 * mag).all()
        seen_calls.append("window")

    def spy_cache(plan, q, kc, ks, vc, vs, lengths, w, s, a, ws, **kw):
        cache_attn(plan, q, kc, ks, vc, vs, lengths, w, s, a, ws, **kw)
        n = int(lengths.max())
        k, v = (torch.empty(b.batch * n, b.kv_cols, device="cuda") for _ in range(2))
        load(plan, torch.zeros_like(lengths), kc, ks, vc, vs, columns(k, b.sources), columns(v, b.sources))
        for i, m in enumerate(lengths.tolist()):
            j = torch.arange(m, device="cuda")
            at = slice(i * n, i * n + m)
            want, mag, _ = heads_attention(torch.cat(q, 1)[i:i + 1], k[at], v[at], group, d, (j >= m - w) | (j < s))
            assert ((torch.cat(a, 1)[i:i + 1].double() - want).abs() <= 1.05 * 2.0 ** -8 * (mag + want.abs()) + 1e-3 * mag).all()
        seen_calls.append("cache")

    tp.tp_window_attn, tp.tp_cache4_attn = spy_window, spy_cache
    try:
        for s, n in enumerate((130, 61)):
            x = torch.randn(n, 512, device="cuda")
            b.prompt(s, x, torch.arange(n, dtype=torch.int32, device="cuda").expand(3, n), chunk=50)
            assert torch.isfinite(x).all()
        x = torch.randn(2, 512, device="cuda")
        for _ in range(3):
            b.step(x, b.lengths.expand(3, 2).contiguous())
    finally:
        tp.tp_window_attn, tp.tp_cache4_attn = window_attn, cache_attn
    assert seen_calls == ["window"] * 5 + ["cache"] * 3 and b.lengths.tolist() == [133, 64]
    assert tp.tp_device_status()[0] == tp.TP_OK


def test_window_and_cache_attention_agree():
    """One token over the cache, and over the cache's values as a bf16 cache of their own."""
    need_gpu()
    b = block(batch=1, ranks=1, q_heads=16, kv_heads=4, capacity=1000, window=300, sinks=5)
    k, v = (torch.randn(900, b.kv_cols, device="cuda").to(BF16) for _ in range(2))
    zero, n = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 900, dtype=torch.int32, device="cuda")
    tp.tp_cache4_store(b.plan, zero, [k], [v], *b.cache)
    tp.tp_cache4_load(b.plan, zero, *b.cache, [k], [v])
    q = torch.randn(1, b.q_cols, device="cuda").to(BF16)
    a = [torch.empty_like(q) for _ in range(2)]
    ws = torch.empty(tp.tp_window_attn_workspace_size(b.plan, 1, 900, 300, 5), dtype=torch.uint8, device="cuda")
    tp.tp_window_attn(b.plan, [q], [k], [v], 300, 5, [a[0]], ws)
    tp.tp_cache4_attn(b.plan, [q], *b.cache, n, 300, 5, [a[1]], b.workspace)
    j = torch.arange(900, device="cuda")
    _, mag, size = heads_attention(q, k, v, 4, 128, (j >= 600) | (j < 5))
    assert ((a[0].double() - a[1].double()).abs() <= (5 * 2.0 ** -8 + 2 * 2.0 ** -8 * size) * mag).all()


def test_steps_in_a_graph():
    """A step whose lengths grow on the device, captured once and replayed, against the same steps issued."""
    need_gpu()
    import copy
    b = block(batch=3, seed=5)
    for s, n in enumerate((40, 511, 700)):
        b.prompt(s, torch.randn(n, b.hidden, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda").expand(3, n))
    x0 = torch.randn(3, b.hidden, device="cuda")
    start, cache0 = b.lengths.clone(), copy.deepcopy(b.cache)
    x = x0.clone()
    for _ in range(4):
        b.step(x, b.lengths.expand(3, 3).contiguous())
    want, want_cache = x.clone(), copy.deepcopy(b.cache)

    def reset():
        x.copy_(x0)
        b.lengths.copy_(start)
        for ts, os_ in zip(b.cache, cache0):
            for t, o in zip(ts, os_):
                t.copy_(o)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(x, b.lengths.expand(3, 3).contiguous())
    for _ in range(2):
        reset()
        for _ in range(4):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want) and b.lengths.tolist() == (start + 4).tolist()
        for ts, os_ in zip(b.cache, want_cache):
            for t, o in zip(ts, os_):
                assert torch.equal(t.view(torch.uint8), o.view(torch.uint8))


def test_two_graphs_share_a_workspace():
    """Calls of different sizes through one workspace, in two graphs replayed in turn: nothing is kept in it."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda r, c: torch.randn(r, c, generator=g, device="cuda").to(BF16)  # noqa: E731
    plan = tp.tp_plan_create(1, 2048, 16, 2, 128, 1)
    cases = []
    for T, S, window in ((1, 5000, ALL), (7, 1500, 700)):
        q, k, v = draw(T, 2048), draw(S, 256), draw(S, 256)
        cases.append((q, k, v, window, torch.zeros_like(q), tp.tp_window_attn_workspace_size(plan, T, S, window, 4)))
    long = 20000  # more splits than a cluster has
    codes = [torch.randint(0, 256, (2 * long, 64), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scale = [torch.rand(2 * long, 4, generator=g, device="cuda").to(BF16) for _ in range(2)]
    cache = [[codes[0]], [scale[0]], [codes[1]], [scale[1]]]
    q1, a1, n1 = draw(1, 2048), torch.zeros(1, 2048, device="cuda", dtype=BF16), torch.full((1,), 19999, dtype=torch.int32, device="cuda")
    need = tp.tp_cache4_attn_workspace_size(plan, 1, long, ALL, 0)
    assert need > 0 and all(c[5] > 0 for c in cases)
    ws = torch.empty(max([need] + [c[5] for c in cases]), dtype=torch.uint8, device="cuda")

    def one(c):
        tp.tp_window_attn(plan, [c[0]], [c[1]], [c[2]], c[3], 4, [c[4]], ws)

    def other():
        tp.tp_cache4_attn(plan, [q1], *cache, n1, ALL, 0, [a1], ws)

    want = []
    for f, out in ((lambda: one(cases[0]), cases[0][4]), (lambda: one(cases[1]), cases[1][4]), (other, a1)):
        ws.fill_(255)
        f()
        want.append(out.clone())
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        one(cases[0])
        other()
    with torch.cuda.graph(graphs[1]):
        one(cases[1])
    for _ in range(3):
        for t in (cases[0][4], cases[1][4], a1):
            t.zero_()
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(cases[0][4], want[0]) and torch.equal(cases[1][4], want[1]) and torch.equal(a1, want[2])


def test_streams_at_once():
    """The same work on four streams at once, each with its own outputs and workspace."""
    need_gpu()
    b = block(batch=2, seed=8)
    for s, n in enumerate((600, 333)):
        b.prompt(s, torch.randn(n, b.hidden, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda").expand(3, n))
    q = torch.randn(2, b.q_cols, device="cuda").to(BF16)
    k, v = (torch.randn(700, b.kv_cols, device="cuda").to(BF16) for _ in range(2))
    q2 = torch.randn(300, b.q_cols, device="cuda").to(BF16)
    pos = torch.arange(300, dtype=torch.int32, device="cuda").expand(3, 300).contiguous()
    torch.cuda.synchronize()
    results = []
    for stream in [torch.cuda.Stream() for _ in range(4)] + [torch.cuda.current_stream()]:
        with torch.cuda.stream(stream):
            a, a2, r = torch.empty_like(q), torch.empty_like(q2), torch.empty_like(q2)
            ws = torch.empty_like(b.workspace)
            ws2 = torch.empty(tp.tp_window_attn_workspace_size(b.plan, 300, 700, 100, 4), dtype=torch.uint8, device="cuda")
            for _ in range(5):
                tp.tp_cache4_attn(b.plan, b.shards(q, 2), *b.cache, b.lengths, b.window, b.sinks, b.shards(a, 2), ws)
                tp.tp_window_attn(b.plan, b.shards(q2, 2), b.shards(k, 2), b.shards(v, 2), 100, 4, b.shards(a2, 2), ws2)
                tp.tp_rotary(b.plan, pos, b.freq, b.shards(a2, 2), None, b.shards(r, 2), None, axis=b.axis)
            results.append((a, a2, r, ws, ws2))
    torch.cuda.synchronize()
    for other in results[:-1]:
        for x, y in zip(other[:3], results[-1][:3]):
            assert torch.equal(x, y)


def test_the_example_runs():
    need_gpu()
    import long_context
    long_context.main(steps=5)
