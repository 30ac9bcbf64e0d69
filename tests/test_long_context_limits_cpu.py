"""The documented limits of the long-context calls, both sides of each: what is within them passes every check (and then meets a
failed rank, before any CUDA call), what is beyond is TP_ERR_UNSUPPORTED."""
import pytest

import tensor_sharded_linear_gqa_gb300 as tp
from test_long_context_cpu import BF, FAKE, U8, T, arr


@pytest.fixture(autouse=True)
def failed_rank():
    tp.tp_set_rank_health(0, False)
    yield
    tp.tp_set_rank_health(0, True)


def plan(hq, hkv, d):
    return tp.tp_plan_create(1, hq * d, hq, hkv, d, 1)


def window(p, t, s):
    hq, hkv, d = p.dims.num_q_heads, p.dims.num_kv_heads, p.dims.head_dim
    q, a, k = T(BF, t, hq * d), T(BF, t, hq * d, ptr=2 * FAKE), T(BF, s, hkv * d)
    return tp.raw_status("tp_window_attn", p.handle, arr(q), arr(k), arr(k), 8, 0, arr(a), FAKE, 1 << 50, None)


def cache(p, batch, cap):
    rows, d = batch * p.dims.num_kv_heads * cap, p.dims.head_dim
    return [arr(t) for t in [T(U8, rows, d // 2), T(BF, rows, d // 32)] * 2]


def copies(p, batch, n, cap):
    k = arr(T(BF, batch * n, p.dims.num_kv_heads * p.dims.head_dim))
    return {tp.raw_status("tp_cache4_store", p.handle, batch, FAKE, None, k, k, *cache(p, batch, cap), None),
            tp.raw_status("tp_cache4_load", p.handle, batch, FAKE, *cache(p, batch, cap), k, k, None)}


def attention(p, batch, cap):
    cols = p.dims.num_q_heads * p.dims.head_dim
    q, a = arr(T(BF, batch, cols)), arr(T(BF, batch, cols, ptr=2 * FAKE))
    return tp.raw_status("tp_cache4_attn", p.handle, batch, q, *cache(p, batch, cap), FAKE, 8, 0, a, FAKE, 1 << 50, None)


WITHIN, BEYOND = tp.TP_ERR_RANK_FAILED, tp.TP_ERR_UNSUPPORTED


@pytest.mark.parametrize("hq, hkv", [(4, 2), (1, 1), (152, 8), (7, 1)])
def test_tokens_by_heads_of_the_window(hq, hkv):
    p, most = plan(hq, hkv, 64), 2 ** 28 // hq
    assert window(p, most, most) == WITHIN and window(p, most + 1, most + 1) == BEYOND


def test_keys_of_the_window():
    p = plan(4, 2, 128)
    assert window(p, 3, 2 ** 31 - 257) == WITHIN and window(p, 3, 2 ** 31 - 256) == BEYOND


@pytest.mark.parametrize("hq, hkv", [(152, 1), (152, 8), (4, 2)])
def test_copies_know_no_q_heads(hq, hkv):
    p = plan(hq, hkv, 64)
    for batch in (55188, 55189, 65535):
        assert copies(p, batch, 1, 1) == {WITHIN}
    assert copies(p, 65536, 1, 1) == {BEYOND}


@pytest.mark.parametrize("hkv", [1, 8])
def test_tokens_of_a_copy(hkv):
    p, most = plan(hkv, hkv, 128), (2 ** 31 - 1024) // hkv
    assert copies(p, 1, most, 5) == {WITHIN} and copies(p, 1, most + 1, 5) == {BEYOND}


@pytest.mark.parametrize("hq, hkv", [(4, 2), (1, 1), (152, 8), (7, 1)])
def test_rows_of_the_attention(hq, hkv):
    p, most = plan(hq, hkv, 64), 2 ** 23 // hq
    assert attention(p, most, 1) == WITHIN and attention(p, most + 1, 1) == BEYOND
    size = lambda batch: tp.tp_cache4_attn_workspace_size(p, batch, 20000, 2 ** 31 - 1, 0)  # noqa: E731
    assert size(most) > 0 and size(most + 1) == 0 and size(2 ** 62) == 0


def test_heads_of_a_group():
    assert attention(plan(65535, 1, 64), 2, 1) == WITHIN and attention(plan(65536, 1, 64), 2, 1) == BEYOND


def test_capacity():
    p = plan(2, 1, 64)
    assert attention(p, 1, 2 ** 31 - 257) == WITHIN and attention(p, 1, 2 ** 31 - 256) == BEYOND
    assert copies(p, 1, 1, 2 ** 31 - 257) == {WITHIN} and copies(p, 1, 1, 2 ** 31 - 256) == {BEYOND}
