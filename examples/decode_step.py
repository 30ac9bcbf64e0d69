"""Decode steps of one tensor-parallel decoder layer behind a shared prompt, from the library's calls:

  norm (8-bit output) -> q/k/v product with bias -> cache row -> attention over the shared prefix and
  the sequences' own caches -> output product onto the residual -> norm (8-bit output) -> feed-forward
  product with GELU -> second product onto the residual; when the caches are full, eviction of the
  keys with the least accumulated attention weight.

Run it on a GB300 after the library is built:  python examples/decode_step.py
PyTorch supplies device memory, the weights' random values and the cache rows' placement.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_sharded_linear_gqa_gb300 as tp  # noqa: E402

EPS = 1e-5
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def quantise(w):
    """e4m3 codes of w's rows and one scale each."""
    scale = w.abs().amax(1) / 448.0
    return (w / scale[:, None]).to(E4M3), scale


class Layer:
    """Weights of one layer, sharded over `ranks`, and the state of a batch that decodes behind one prefix."""

    def __init__(self, batch=16, ranks=2, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, ffn=4096, prefix=1000,
                 capacity=48, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.batch, self.ranks, self.hidden, self.capacity = batch, ranks, hidden, capacity
        self.plan = tp.tp_plan_create(ranks, hidden, q_heads, kv_heads, head_dim, ffn)
        self.sources = ranks if kv_heads >= ranks else 1  # copies of K/V: one per rank, or one for all
        self.q_cols, self.kv_cols = q_heads * head_dim, kv_heads * head_dim
        self.norm1, self.norm2 = 1.0 + normal(hidden, std=0.1), 1.0 + normal(hidden, std=0.1)
        self.w_qkv, self.s_qkv = quantise(normal(self.q_cols + 2 * self.kv_cols, hidden, std=0.03))
        self.b_qkv = normal(self.q_cols + 2 * self.kv_cols, std=0.1)
        self.w_o = normal(hidden, self.q_cols, std=0.02).to(BF16)
        self.w_up, self.s_up = quantise(normal(ffn, hidden, std=0.03))
        self.b_up = normal(ffn, std=0.1)
        self.w_down = normal(hidden, ffn, std=0.02).to(BF16)
        self.k_prefix, self.v_prefix = (normal(prefix, self.kv_cols).to(BF16) for _ in range(2))
        self.k_own, self.v_own = (torch.zeros(batch * capacity, self.kv_cols, dtype=BF16, device="cuda") for _ in range(2))
        heads = kv_heads // self.sources
        self.weights = [torch.zeros(batch * heads, capacity, device="cuda") for _ in range(self.sources)]
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.longest = 0
        # buffers that every step uses again
        self.x8 = torch.empty(batch, hidden, dtype=E4M3, device="cuda")
        self.x8_scale = torch.empty(batch, device="cuda")
        self.qkv = torch.empty(batch, self.q_cols + 2 * self.kv_cols, dtype=BF16, device="cuda")
        self.a = torch.empty(batch, self.q_cols, dtype=BF16, device="cuda")
        self.h = torch.empty(batch, ffn, dtype=BF16, device="cuda")
        self.workspace = torch.empty(tp.tp_prefix_attn_workspace_size(self.plan, batch, prefix, capacity, True),
                                     dtype=torch.uint8, device="cuda")

    def shards(self, t, n, dim):
        return list(t.split(t.shape[dim] // n, dim=dim))

    def step(self, residual):
        """One token of every sequence: `residual` [batch x hidden] f32 is updated in place."""
        if self.longest == self.capacity:  # the new rows would lie in the next sequence's cache
            raise RuntimeError("the caches are full: evict first")
        n, s = self.ranks, self.sources
        tp.tp_add_rmsnorm(residual, None, self.norm1, EPS, None, self.x8, self.x8_scale)
        tp.tp_linear_epilogue(n, tp.TP_SHARD_COLUMN, [self.x8], self.shards(self.w_qkv, n, 0), self.qkv, bias=self.b_qkv,
                              x_scale=self.x8_scale, w_scale=self.s_qkv)
        q, k, v = self.qkv.split([self.q_cols, self.kv_cols, self.kv_cols], dim=1)
        rows = torch.arange(self.batch, device="cuda") * self.capacity + self.lengths
        self.k_own[rows], self.v_own[rows] = k, v
        self.lengths += 1
        self.longest += 1
        tp.tp_prefix_attn(self.plan, self.shards(q, n, 1), self.shards(self.k_prefix, s, 1), self.shards(self.v_prefix, s, 1),
                          self.shards(self.k_own, s, 1), self.shards(self.v_own, s, 1), self.lengths,
                          self.shards(self.a, n, 1), self.workspace, weight_in=self.weights, weight_out=self.weights)
        tp.tp_linear_epilogue(n, tp.TP_SHARD_ROW, self.shards(self.a, n, 1), self.shards(self.w_o, n, 1), residual,
                              residual=residual)
        tp.tp_add_rmsnorm(residual, None, self.norm2, EPS, None, self.x8, self.x8_scale)
        tp.tp_linear_epilogue(n, tp.TP_SHARD_COLUMN, [self.x8], self.shards(self.w_up, n, 0), self.h, bias=self.b_up,
                              activation=tp.TP_ACT_GELU, x_scale=self.x8_scale, w_scale=self.s_up)
        tp.tp_linear_epilogue(n, tp.TP_SHARD_ROW, self.shards(self.h, n, 1), self.shards(self.w_down, n, 1), residual,
                              residual=residual)

    def evict(self, budget, n_first, n_recent):
        """Cuts the own caches to `budget` keys a sequence and kv head, in place; returns the kept positions."""
        heads = self.weights[0].shape[0] // self.batch
        kept = torch.empty(self.sources, self.batch * heads, budget, dtype=torch.int32, device="cuda")
        k, v = (self.shards(t, self.sources, 1) for t in (self.k_own, self.v_own))
        tp.tp_cache_evict(self.plan, self.lengths, k, v, self.weights, budget, n_first, n_recent, k, v, self.weights,
                          self.lengths, kept)
        self.longest = min(self.longest, budget)
        return kept


def main(steps=100):
    layer = Layer()
    residual = torch.randn(layer.batch, layer.hidden, device="cuda")
    evictions = 0
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        if layer.longest == layer.capacity:
            layer.evict(budget=layer.capacity // 2, n_first=2, n_recent=8)
            evictions += 1
        layer.step(residual)
    end.record()
    torch.cuda.synchronize()
    status, word = tp.tp_device_status()
    assert status == tp.TP_OK, f"device status {word:#x}"
    assert torch.isfinite(residual).all()
    print(f"{steps} steps of {layer.batch} sequences, {evictions} evictions, own caches now {layer.longest} keys: "
          f"{start.elapsed_time(end) / steps * 1e3:.0f} us a step, |residual| {residual.abs().mean().item():.3f}")


if __name__ == "__main__":
    main()
