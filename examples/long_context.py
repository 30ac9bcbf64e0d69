"""A long conversation through one tensor-parallel attention block whose cache is held in 4 bits:

  the prompt, a chunk of tokens at a time: norm -> q/k/v product -> rotary positions -> keys and values into
  the 4-bit cache -> attention over a sliding window and the first tokens (what the chunk sees of
  the cache, and no more, is read back) -> output product onto the residual;
  then one token at a time for every sequence: the same with attention over the 4-bit cache itself.

Run it on a GB300 after the library is built:  python examples/long_context.py
PyTorch supplies device memory, the weights' random values and the lengths' additions.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_sharded_linear_gqa_gb300 as tp  # noqa: E402

EPS = 1e-5
BF16 = torch.bfloat16


class Block:
    """An attention block's weights, sharded over `ranks`, and the 4-bit caches of `batch` sequences."""

    def __init__(self, batch=4, ranks=2, hidden=1024, q_heads=16, kv_heads=4, head_dim=128, capacity=2048, window=512, sinks=4,
                 theta=1e6, sections=(16, 24, 24), seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

        self.batch, self.ranks, self.hidden, self.capacity = batch, ranks, hidden, capacity
        self.window, self.sinks, self.head_dim = window, sinks, head_dim
        self.plan = tp.tp_plan_create(ranks, hidden, q_heads, kv_heads, head_dim, ranks)
        self.sources = ranks if kv_heads >= ranks else 1
        self.heads = kv_heads // self.sources  # of a source
        self.q_cols, self.kv_cols = q_heads * head_dim, kv_heads * head_dim
        self.norm = 1.0 + normal(hidden, std=0.1).float()
        self.w_qkv = normal(self.q_cols + 2 * self.kv_cols, hidden, std=0.04)
        self.w_o = normal(hidden, self.q_cols, std=0.02)
        pairs = sum(sections)
        self.freq = (theta ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
        self.axis, self.axes = tp.rotary_axes(sections), len(sections)
        rows = batch * self.heads * capacity
        self.cache = [[torch.zeros(rows, cols, dtype=dtype, device="cuda") for _ in range(self.sources)]
                      for cols, dtype in ((head_dim // 2, torch.uint8), (head_dim // 32, BF16)) * 2]
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        # keys and values of a prompt in bf16, by position; those that no token of a chunk sees are never read back
        self.kv = [torch.zeros(capacity, self.kv_cols, dtype=BF16, device="cuda") for _ in range(2)]
        size = tp.tp_cache4_attn_workspace_size(self.plan, batch, capacity, window, sinks)
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")

    def shards(self, t, n, dim=1):
        return list(t.split(t.shape[dim] // n, dim=dim))

    def of(self, sequence):
        """One sequence's part of the caches: its rows are neighbours."""
        per = self.heads * self.capacity
        return [[t[sequence * per:(sequence + 1) * per] for t in ts] for ts in self.cache]

    def project(self, residual, positions):
        """q, k, v of the tokens' norm, q and k turned by their positions [axes x tokens]."""
        x = torch.empty(residual.shape, dtype=BF16, device="cuda")
        tp.tp_add_rmsnorm(residual, None, self.norm, EPS, None, x)
        qkv = torch.empty(residual.shape[0], self.w_qkv.shape[0], dtype=BF16, device="cuda")
        tp.tp_linear_epilogue(self.ranks, tp.TP_SHARD_COLUMN, [x], self.shards(self.w_qkv, self.ranks, 0), qkv)
        q, k, v = qkv.split([self.q_cols, self.kv_cols, self.kv_cols], dim=1)
        qs, ks = self.shards(q, self.ranks), self.shards(k, self.sources)
        tp.tp_rotary(self.plan, positions, self.freq, qs, ks, qs, ks, axis=self.axis)
        return qs, ks, self.shards(v, self.sources)

    def output(self, a, residual):
        tp.tp_linear_epilogue(self.ranks, tp.TP_SHARD_ROW, self.shards(a, self.ranks), self.shards(self.w_o, self.ranks), residual,
                              residual=residual)

    def prompt(self, sequence, residual, positions, chunk=256):
        """A sequence's prompt [tokens x hidden] f32, updated in place, into its empty cache."""
        if residual.shape[0] > self.capacity:
            raise ValueError(f"a prompt of {residual.shape[0]} tokens, the cache has {self.capacity} positions")
        cache = self.of(sequence)
        for t0 in range(0, residual.shape[0], chunk):
            part = residual[t0:t0 + chunk]
            n = part.shape[0]
            q, k, v = self.project(part, positions[:, t0:t0 + n].contiguous())
            tp.tp_cache4_store(self.plan, torch.full((1,), t0, dtype=torch.int32, device="cuda"), k, v, *cache)
            # the keys that the chunk sees, as their codes say: those from its first token's window on, and the first ones
            keys, values = (self.shards(t[:t0 + n], self.sources) for t in self.kv)
            near = max(0, t0 - self.window + 1)
            for first, end in ((near, t0 + n), (0, min(near, self.sinks))):
                if first < end:
                    tp.tp_cache4_load(self.plan, torch.full((1,), first, dtype=torch.int32, device="cuda"), *cache,
                                      [t[first:end] for t in keys], [t[first:end] for t in values])
            a = torch.empty(n, self.q_cols, dtype=BF16, device="cuda")
            size = tp.tp_window_attn_workspace_size(self.plan, n, t0 + n, self.window, self.sinks)
            tp.tp_window_attn(self.plan, q, keys, values, self.window, self.sinks, self.shards(a, self.ranks),
                              torch.empty(size, dtype=torch.uint8, device="cuda"))
            self.output(a, part)
        self.lengths[sequence] = residual.shape[0]

    def step(self, residual, positions):
        """One token of every sequence: `residual` [batch x hidden] f32 is updated in place."""
        q, k, v = self.project(residual, positions)
        tp.tp_cache4_store(self.plan, self.lengths, k, v, *self.cache)
        self.lengths += 1
        a = torch.empty(self.batch, self.q_cols, dtype=BF16, device="cuda")
        tp.tp_cache4_attn(self.plan, q, *self.cache, self.lengths, self.window, self.sinks, self.shards(a, self.ranks), self.workspace)
        self.output(a, residual)


def main(steps=100):
    block = Block()
    for s in range(block.batch):
        n = 300 + 211 * s
        block.prompt(s, torch.randn(n, block.hidden, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda").expand(3, n))
    residual = torch.randn(block.batch, block.hidden, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        block.step(residual, block.lengths.expand(3, block.batch).contiguous())
    end.record()
    torch.cuda.synchronize()
    status, word = tp.tp_device_status()
    assert status == tp.TP_OK, f"device status {word:#x}"
    assert torch.isfinite(residual).all()
    print(f"{steps} steps of {block.batch} sequences, now {block.lengths.tolist()} tokens: "
          f"{start.elapsed_time(end) / steps * 1e3:.0f} us a step, |residual| {residual.abs().mean().item():.3f}")


if __name__ == "__main__":
    main()
