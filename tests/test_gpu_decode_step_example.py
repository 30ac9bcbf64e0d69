"""The decode-step example against the same layer in float64 torch: several steps, one of them behind an
eviction. The reference rounds where the layer's buffers do (e4m3 codes, bf16 q/k/v, attention output
and feed-forward activations); a code on the border may still fall to the other side, so the residual
stream is compared within the bf16 bound of the other block tests."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

from gpu_util import BF16_TOL, need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Reference:
    def __init__(self, layer, hq, hkv, d):
        self.l, self.hq, self.hkv, self.d = layer, hq, hkv, d
        B = layer.batch
        self.k = [[[] for _ in range(hkv)] for _ in range(B)]  # own keys by sequence and kv head
        self.v = [[[] for _ in range(hkv)] for _ in range(B)]
        self.w = [[[] for _ in range(hkv)] for _ in range(B)]

    def norm8(self, x, w):
        y = x / (x.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
        scale = y.abs().amax(1, keepdim=True) / 448.0
        return (y / scale).float().to(torch.float8_e4m3fn).double() * scale

    def step(self, r):
        l, d, G = self.l, self.d, self.hq // self.hkv
        bf = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
        x = self.norm8(r, l.norm1)
        qkv = bf(x @ (l.w_qkv.double() * l.s_qkv.double()[:, None]).t() + l.b_qkv.double())
        q, k, v = qkv.split([l.q_cols, l.kv_cols, l.kv_cols], dim=1)
        a = torch.zeros(l.batch, self.hq, d, dtype=torch.float64, device="cuda")
        P = l.k_prefix.shape[0]
        for b in range(l.batch):
            for h in range(self.hkv):
                cols = slice(h * d, (h + 1) * d)
                self.k[b][h].append(k[b, cols])
                self.v[b][h].append(v[b, cols])
                self.w[b][h].append(0.0)
                keys = torch.cat([l.k_prefix[:, cols].double(), torch.stack(self.k[b][h])])
                vals = torch.cat([l.v_prefix[:, cols].double(), torch.stack(self.v[b][h])])
                p = torch.softmax(q[b].view(self.hq, d)[h * G:(h + 1) * G] @ keys.t() / math.sqrt(d), dim=1)
                a[b, h * G:(h + 1) * G] = p @ vals
                self.w[b][h] = [x + y for x, y in zip(self.w[b][h], p[:, P:].sum(0).tolist())]
        r = r + bf(a.view(l.batch, -1)) @ l.w_o.double().t()
        x = self.norm8(r, l.norm2)
        z = x @ (l.w_up.double() * l.s_up.double()[:, None]).t() + l.b_up.double()
        return r + bf(0.5 * z * (1 + torch.erf(z / math.sqrt(2)))) @ l.w_down.double().t()

    def evict(self, budget, first, recent):
        kept = {}
        for b in range(self.l.batch):
            for h in range(self.hkv):
                w = self.w[b][h]
                n = len(w)
                keep = list(range(n))
                if n > budget:
                    middle = sorted(range(first, n - recent), key=lambda j: (-w[j], j))[:budget - first - recent]
                    keep = sorted(list(range(first)) + middle + list(range(n - recent, n)))
                kept[b, h] = keep
                for store in (self.k, self.v, self.w):
                    store[b][h] = [store[b][h][j] for j in keep]
        return kept


@pytest.mark.parametrize("ranks,kv_heads", [(2, 2), (4, 2), (1, 4)])
def test_steps_and_eviction_against_float64(ranks, kv_heads):
    need_gpu()
    m = example()
    layer = m.Layer(batch=5, ranks=ranks, hidden=256, q_heads=8, kv_heads=kv_heads, head_dim=64, ffn=512, prefix=150,
                    capacity=12, seed=ranks)
    ref = Reference(layer, 8, kv_heads, 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    residual = torch.randn(5, 256, generator=g, device="cuda")
    r = residual.double()
    for step in range(15):
        if layer.longest == layer.capacity:
            kept = layer.evict(6, 1, 2)
            want = ref.evict(6, 1, 2)
            heads = layer.weights[0].shape[0] // 5
            for (b, h), keep in want.items():
                assert kept[h // heads, b * heads + h % heads].tolist() == keep
        layer.step(residual)
        r = ref.step(r)
        torch.cuda.synchronize()
        err = ((residual.double() - r).abs().max() / r.abs().max()).item()
        assert err <= BF16_TOL, (step, err)
    assert layer.longest == 9


def test_main_runs(capsys):
    need_gpu()
    example().main(steps=60)
    assert "evictions" in capsys.readouterr().out
