"""The long-context calls where offsets pass 32 bits: the same data near the end of large tensors and in small ones.
Attention applies no positions, so the small case's outputs are those of the large one; where the sizes lead to other
splits or tiles both are within their roundings (P and A to bf16, 2^-8 each, a side) of one softmax."""
import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def normal(rows, cols, seed):
    return torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def close(a, b, v):
    return ((a.float() - b.float()).abs() <= 4 * 2.0 ** -8 * v.float().abs().max()).all()


def test_cache_in_4_bits():
    need_gpu()
    plan, n, d = tp.tp_plan_create(1, 512, 4, 2, 128, 1), 100, 128
    k, v, q = normal(n, 2 * d, 1), normal(n, 2 * d, 2), normal(1, 4 * d, 3)
    got = []
    for C in (1 << 25, 128):  # codes of 2^32 bytes and more, and few
        rows = 2 * C
        codes = [torch.empty(rows, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scale = [torch.full((rows, d // 32), float("nan"), dtype=BF16, device="cuda") for _ in range(2)]
        cache = [codes[0]], [scale[0]], [codes[1]], [scale[1]]
        length = torch.tensor([C - n], dtype=torch.int32, device="cuda")
        tp.tp_cache4_store(plan, length, [k], [v], *cache)
        back = [torch.empty(n, 2 * d, dtype=BF16, device="cuda") for _ in range(2)]
        tp.tp_cache4_load(plan, length, *cache, [back[0]], [back[1]])
        a = torch.empty_like(q)
        ws = torch.empty(tp.tp_cache4_attn_workspace_size(plan, 1, C, 90, 0), dtype=torch.uint8, device="cuda")
        tp.tp_cache4_attn(plan, [q], *cache, length + n, 90, 0, [a], ws)
        torch.cuda.synchronize()
        assert tp.tp_device_status()[0] == tp.TP_OK
        got.append((*back, a))
        del codes, scale, cache
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].isfinite().all() and got[0][2].isfinite().all() and close(got[0][2], got[1][2], v)


def test_window():
    need_gpu()
    plan, d, S = tp.tp_plan_create(1, 512, 4, 1, 128, 1), 128, (1 << 24) + 5  # K and V of 2^32 bytes and more
    q, few = normal(7, 4 * d, 4), [normal(1000, d, 5), normal(1000, d, 6)]
    outs = []
    for size in (S, 1000):
        kv = []
        for x in few:
            t = torch.zeros(size, d, dtype=BF16, device="cuda")
            t[:4], t[-600:] = x[:4], x[-600:]
            kv.append(t)
        a = torch.empty_like(q)
        ws = torch.empty(tp.tp_window_attn_workspace_size(plan, 7, size, 500, 4), dtype=torch.uint8, device="cuda")
        tp.tp_window_attn(plan, [q], [kv[0]], [kv[1]], 500, 4, [a], ws)
        torch.cuda.synchronize()
        assert tp.tp_device_status()[0] == tp.TP_OK
        outs.append(a)
        del kv, t
    assert outs[0].isfinite().all() and close(*outs, few[1])


def test_rotary():
    need_gpu()
    T, pitch = 1100, 1 << 21  # rows over 2^31 values
    plan = tp.tp_plan_create(1, 256, 2, 2, 128, 1)
    q = normal(T, 256, 7)
    positions = torch.arange(T, dtype=torch.int32, device="cuda") * 1001
    freq = torch.logspace(0, -4, 64, device="cuda")
    want = torch.empty_like(q)
    tp.tp_rotary(plan, positions, freq, [q], None, [want], None)
    wide = torch.empty(T * pitch, dtype=BF16, device="cuda").view(T, pitch)[:, -256:]
    wide.copy_(q)
    tp.tp_rotary(plan, positions, freq, [wide], None, [wide], None)
    torch.cuda.synchronize()
    assert torch.equal(wide, want)
