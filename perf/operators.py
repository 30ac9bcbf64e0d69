"""The decode-step operators around the sharded projections, as cases that can be timed.

Four operators, each in its plain form (elementary torch operations in 32 bits) and through the
library's calls:

  norm    residual addition and root-mean-square norm of one or several per-rank partials, with a
          bf16 output or an e4m3 output with one scale a token       (tp_add_rmsnorm)
  linear  column- or row-parallel product with the dequantisation, bias, activation and residual in
          its epilogue, bf16 or e4m3 operands                        (tp_linear_epilogue)
  attn    attention of one new token per sequence over a prefix that the whole batch shares and each
          sequence's own cache, with the keys' accumulated weights   (tp_prefix_attn)
  evict   eviction from the own caches by accumulated attention weight (tp_cache_evict)

``own = False`` runs the plain forms, ``own = True`` the library's calls.
"""
import math

import torch

own = False

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
EPS = 1e-5
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -96  # the row maximum that a scale is taken from is at least this


def listed():
    return [
        # one token of a hidden-4096 layer: nothing but latency
        {"name": "norm_token", "op": "norm", "T": 1, "D": 4096, "n": 1, "x": "bf16", "res": "bf16", "y": "bf16"},
        # decode batch: eight ranks' f32 partials of a row-parallel layer, 8-bit output for the next product
        {"name": "norm_decode_tp8", "op": "norm", "T": 64, "D": 4096, "n": 8, "x": "f32", "res": "f32", "y": "e4m3"},
        # prefill of a hidden-8192 layer: the combined f32 output of a row-parallel layer
        {"name": "norm_prefill", "op": "norm", "T": 4096, "D": 8192, "n": 1, "x": "f32", "res": "bf16", "y": "bf16"},
        # output projection of one token, with bias and residual, over eight ranks' input slices
        {"name": "linear_token", "op": "linear", "shard": "row", "tp": 8, "T": 1, "K": 4096, "N": 4096, "in": "bf16",
         "bias": True, "act": "none", "res": "bf16", "y": "bf16"},
        # first feed-forward product of an odd decode batch in 8 bits: weight streaming
        {"name": "linear_decode_e4m3", "op": "linear", "shard": "column", "tp": 8, "T": 61, "K": 4096, "N": 14336,
         "in": "e4m3", "bias": True, "act": "gelu", "res": "none", "y": "bf16"},
        # output projection of a prefill that is no whole number of tiles
        {"name": "linear_prefill_row", "op": "linear", "shard": "row", "tp": 8, "T": 2047, "K": 8192, "N": 8192,
         "in": "bf16", "bias": False, "act": "none", "res": "f32", "y": "f32"},
        # the widest product of a hidden-8192 prefill, in 8 bits
        {"name": "linear_prefill_e4m3", "op": "linear", "shard": "column", "tp": 8, "T": 4096, "K": 8192, "N": 28672,
         "in": "e4m3", "bias": True, "act": "silu", "res": "none", "y": "bf16"},
        # a single short conversation after a short shared prompt: latency
        {"name": "attn_single", "op": "attn", "tp": 1, "B": 1, "Hq": 16, "Hkv": 4, "d": 128, "P": 100, "C": 64,
         "lo": 33, "hi": 33, "weights": True},
        # decode batch behind a long system prompt, ragged own caches, some still empty
        {"name": "attn_batch_tp8", "op": "attn", "tp": 8, "B": 61, "Hq": 64, "Hkv": 8, "d": 128, "P": 4099, "C": 512,
         "lo": 0, "hi": 511, "weights": True},
        # the largest: a document of 32k tokens shared by 128 sequences, kv heads replicated over the ranks
        {"name": "attn_document_rep", "op": "attn", "tp": 8, "B": 128, "Hq": 32, "Hkv": 4, "d": 128, "P": 32768, "C": 2048,
         "lo": 1, "hi": 2048, "weights": False},
        # one sequence's cache goes a little over its budget
        {"name": "evict_single", "op": "evict", "tp": 1, "B": 1, "Hkv": 4, "d": 128, "C": 640, "lo": 577, "hi": 577,
         "budget": 512, "first": 4, "recent": 64},
        # a decode batch's caches are cut to half; the short ones stay whole
        {"name": "evict_batch_tp8", "op": "evict", "tp": 8, "B": 64, "Hkv": 8, "d": 128, "C": 2048, "lo": 700, "hi": 2048,
         "budget": 1024, "first": 4, "recent": 256},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "attn", "evict"])
    if op == "norm":
        n = rng.choice([1, 1, 2, 4, 8])
        d = _log(rng, 64, 8192)
        return {"op": op, "T": _log(rng, 1, 4096 // n), "D": d if rng.random() < 0.3 else -(-d // 8) * 8, "n": n,
                "x": rng.choice(["f32", "bf16"]), "res": rng.choice(["f32", "bf16", "none"]),
                "y": rng.choice(["bf16", "e4m3"])}
    if op == "linear":
        tp = rng.choice([1, 2, 4, 8])
        shard = rng.choice(["column", "row"])
        k, n = _log(rng, 128, 8192), _log(rng, 128, 8192)
        if shard == "row":
            k = -(-k // (16 * tp)) * 16 * tp  # every rank's slice starts on a 16-byte boundary
        else:
            n = -(-n // (8 * tp)) * 8 * tp  # every rank's output columns do
        return {"op": op, "shard": shard, "tp": tp, "T": _log(rng, 1, 4096), "K": k, "N": n,
                "in": rng.choice(["bf16", "e4m3"]), "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "relu", "gelu", "silu"]), "res": rng.choice(["none", "bf16", "f32"]),
                "y": rng.choice(["bf16", "f32"])}
    hkv = rng.choice([1, 2, 4, 8])
    tp = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128])
    if op == "attn":
        g = rng.choice([1, 2, 3, 4, 7, 8, 16])
        while (hkv * g) % tp:
            tp //= 2
        b = _log(rng, 1, 128)
        p = 0 if rng.random() < 0.1 else _log(rng, 1, 32768 if hkv * g <= 32 else 4096)
        c = _log(rng, 1, 2048 if hkv <= 4 else 512)
        hi = rng.randint(0, c)
        return {"op": op, "tp": tp, "B": b, "Hq": hkv * g, "Hkv": hkv, "d": d, "P": p, "C": c,
                "lo": rng.randint(0, hi), "hi": hi, "weights": rng.random() < 0.6}
    b, c = _log(rng, 1, 64), _log(rng, 2, 2048)
    hi = rng.randint(1, c)
    budget = rng.randint(1, c)
    first = rng.randint(0, min(4, budget))
    return {"op": op, "tp": tp, "B": b, "Hkv": hkv, "d": d, "C": c, "lo": rng.randint(0, hi), "hi": hi, "budget": budget,
            "first": first, "recent": rng.randint(0, budget - first)}


# ---- inputs ----------------------------------------------------------------------
def _lengths(case, gen):
    """Sequence lengths spread evenly over [lo, hi], in an order of the seed's."""
    b = case["B"]
    every = torch.linspace(case["lo"], case["hi"], b, dtype=torch.float64).round().to(torch.int32)
    return every[torch.randperm(b, generator=gen)].cuda()


def _length_list(case):
    b = case["B"]
    return torch.linspace(case["lo"], case["hi"], b, dtype=torch.float64).round().to(torch.int64).tolist()


def _padded(rows, cols, dtype):
    """An uninitialised [rows x cols] view whose rows start on 16-byte boundaries."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _normal(rows, cols, dtype, gen, std=1.0):
    out = _padded(rows, cols, dtype)
    out.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * std)
    return out


def _quantised(rows, cols, gen, std=1.0):
    """e4m3 codes and one scale a row, of normal values."""
    v = torch.randn(rows, cols, generator=gen, device="cuda") * std
    scale = v.abs().amax(1) / E4M3_MAX
    out = _padded(rows, cols, E4M3)
    out.copy_((v / scale[:, None]).to(E4M3))
    return out, scale


def _bf16_big(rows, cols, gen, std=1.0):
    """A normal bf16 matrix, drawn without an f32 copy of the whole."""
    return torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(0.0, std, generator=gen)


def _kv_sources(case):
    """(number of K/V copies, kv heads in each): sharded over the ranks, or one copy where they are replicated."""
    return (case["tp"], case["Hkv"] // case["tp"]) if case["Hkv"] >= case["tp"] else (1, case["Hkv"])


def _columns(t, parts):
    return list(t.split(t.shape[1] // parts, dim=1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    cpu = torch.Generator().manual_seed(seed * 1000003 + 29)
    s = {"case": case}
    if case["op"] == "norm":
        T, D, n = case["T"], case["D"], case["n"]
        s["x"] = [_normal(T, D, TYPES[case["x"]], gen) for _ in range(n)]
        s["res"] = _normal(T, D, TYPES[case["res"]], gen, 4.0) if case["res"] != "none" else None
        s["w"] = (1.0 + 0.2 * torch.randn(1, D, generator=gen, device="cuda")).to(BF16)
        s["res_out"] = _padded(T, D, TYPES[case["res"]]) if case["res"] != "none" else None
        s["y"] = _padded(T, D, TYPES[case["y"]])
        s["scale"] = torch.empty(T, device="cuda") if case["y"] == "e4m3" else None
    elif case["op"] == "linear":
        T, K, N, tp_size = case["T"], case["K"], case["N"], case["tp"]
        if case["in"] == "e4m3":
            s["x"], s["xs"] = _quantised(T, K, gen)
            s["w"], s["ws"] = _quantised(N, K, gen, 0.02)
        else:
            s["x"], s["xs"] = _normal(T, K, BF16, gen), None
            s["w"], s["ws"] = _normal(N, K, BF16, gen, 0.02), None
        s["bias"] = torch.randn(1, N, generator=gen, device="cuda") * 0.5 if case["bias"] else None
        s["res"] = _normal(T, N, TYPES[case["res"]], gen) if case["res"] != "none" else None
        s["y"] = _padded(T, N, TYPES[case["y"]])
        row = case["shard"] == "row"
        s["xr"] = _columns(s["x"], tp_size) if row else [s["x"]]
        s["wr"] = _columns(s["w"], tp_size) if row else list(s["w"].split(N // tp_size, dim=0))
    else:
        B, C, d, Hkv = case["B"], case["C"], case["d"], case["Hkv"]
        nkv, hr = _kv_sources(case)
        s["len"] = _lengths(case, cpu)
        s["k"], s["v"] = (_bf16_big(B * C, Hkv * d, gen) for _ in range(2))
        s["kr"], s["vr"] = _columns(s["k"], nkv), _columns(s["v"], nkv)
        # accumulated weights: most keys little, a few much, some never looked at
        wt = torch.rand(nkv, B * hr, C, generator=gen, device="cuda").pow(6) * 4.0
        s["wt"] = torch.where(torch.rand(wt.shape, generator=gen, device="cuda") < 0.05, torch.zeros_like(wt), wt)
        if case["op"] == "attn":
            P, Hq = case["P"], case["Hq"]
            s["q"] = _bf16_big(B, Hq * d, gen, 2.0)
            s["kp"], s["vp"] = (_bf16_big(P, Hkv * d, gen) for _ in range(2))
            s["qr"], s["kpr"], s["vpr"] = _columns(s["q"], case["tp"]), _columns(s["kp"], nkv), _columns(s["vp"], nkv)
            s["a"] = torch.empty(B, Hq * d, dtype=BF16, device="cuda")
            s["ar"] = _columns(s["a"], case["tp"])
            s["wt_out"] = torch.empty_like(wt) if case["weights"] else None
        else:
            n = case["budget"]
            s["ko"], s["vo"] = (torch.zeros(B * n, Hkv * d, dtype=BF16, device="cuda") for _ in range(2))
            s["kor"], s["vor"] = _columns(s["ko"], nkv), _columns(s["vo"], nkv)
            s["wt_out"] = torch.zeros(nkv, B * hr, n, device="cuda")
            s["kept"] = torch.empty(nkv, B * hr, n, dtype=torch.int32, device="cuda")
            s["len_out"] = torch.empty_like(s["len"])
    if own:
        import tensor_sharded_linear_gqa_gb300 as tp

        s["tp"] = tp
        if case["op"] in ("attn", "evict"):
            hq = case.get("Hq", max(case["Hkv"], case["tp"]))
            s["plan"] = tp.tp_plan_create(case["tp"], hq * case["d"], hq, case["Hkv"], case["d"], case["tp"])
            # the caches outlive the calls: their descriptors are made once
            for name in ("k", "v"):
                s[name + "_own"] = tp.arr(s[name + "r"])
            s["wt_in"] = tp.arr(list(s["wt"]))
            if s["wt_out"] is not None:
                s["wt_to"] = tp.arr(list(s["wt_out"]))
        if case["op"] == "attn":
            s["kp_own"], s["vp_own"] = tp.arr(s["kpr"]), tp.arr(s["vpr"])
            s["ws"] = torch.empty(tp.tp_prefix_attn_workspace_size(s["plan"], case["B"], case["P"], case["C"], case["weights"]),
                                  dtype=torch.uint8, device="cuda")
        if case["op"] == "evict":
            s["ko_own"], s["vo_own"] = tp.arr(s["kor"]), tp.arr(s["vor"])
    return s


# ---- one pass ----------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    tp, case = s["tp"], s["case"]
    if case["op"] == "norm":
        tp.tp_add_rmsnorm(s["x"], s["res"], s["w"], EPS, s["res_out"], s["y"], s["scale"])
        return _some(y=s["y"], scale=s["scale"], res=s["res_out"])
    if case["op"] == "linear":
        tp.tp_linear_epilogue(case["tp"], tp.TP_SHARD_ROW if case["shard"] == "row" else tp.TP_SHARD_COLUMN, s["xr"], s["wr"],
                              s["y"], bias=s["bias"], activation=tp.ACTIVATIONS[case["act"]], residual=s["res"],
                              x_scale=s["xs"], w_scale=s["ws"])
        return _some(y=s["y"])
    if case["op"] == "attn":
        tp.tp_prefix_attn(s["plan"], s["qr"], s["kp_own"], s["vp_own"], s["k_own"], s["v_own"], s["len"], s["ar"], s["ws"],
                          weight_in=s["wt_in"] if case["weights"] else None,
                          weight_out=s["wt_to"] if case["weights"] else None)
        return _some(a=s["a"], weights=s["wt_out"])
    tp.tp_cache_evict(s["plan"], s["len"], s["k_own"], s["v_own"], s["wt_in"], case["budget"], case["first"], case["recent"],
                      s["ko_own"], s["vo_own"], s["wt_to"], s["len_out"], s["kept"])
    return _some(k=s["ko"], v=s["vo"], weights=s["wt_out"], lengths=s["len_out"], kept=s["kept"])


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


# ---- plain forms ---------------------------------------------------------------------
def _plain_norm(s):
    z = torch.stack([x.float() for x in s["x"]]).sum(0)
    if s["res"] is not None:
        z = z + s["res"].float()
    y = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    res = z.to(s["res"].dtype) if s["res"] is not None else None
    if s["case"]["y"] != "e4m3":
        return _some(y=y.to(TYPES[s["case"]["y"]]), res=res)
    scale = y.abs().amax(1).clamp_min(SCALE_FLOOR) / E4M3_MAX
    return _some(y=(y / scale[:, None]).to(E4M3), scale=scale, res=res)


_ACT = {"none": lambda z: z, "relu": lambda z: z.clamp_min(0.0), "silu": lambda z: z / (1.0 + torch.exp(-z)),
        "gelu": lambda z: 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))}


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        z = z * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _ACT[s["case"]["act"]](z)
    if s["res"] is not None:
        z = z + s["res"].float()
    return _some(y=z.to(TYPES[s["case"]["y"]]))


def _by_head(wt, case):
    """[sources, B * heads, .] -> [B, Hkv, .]"""
    nkv, hr = _kv_sources(case)
    return wt.view(nkv, case["B"], hr, wt.shape[-1]).transpose(0, 1).reshape(case["B"], case["Hkv"], wt.shape[-1])


def _by_source(wt, case):
    """[B, Hkv, .] -> [sources, B * heads, .]"""
    nkv, hr = _kv_sources(case)
    return wt.view(case["B"], nkv, hr, wt.shape[-1]).transpose(0, 1).reshape(nkv, case["B"] * hr, wt.shape[-1])


def _plain_attn(s):
    case = s["case"]
    B, Hq, Hkv, d, P, C = (case[k] for k in ("B", "Hq", "Hkv", "d", "P", "C"))
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    scale = 1.0 / math.sqrt(d)
    qh = q.transpose(0, 1).reshape(Hkv, -1, d)  # every row of the batch, by kv head
    kp, vp = (t.float().view(P, Hkv, d).transpose(0, 1) for t in (s["kp"], s["vp"]))
    ko, vo = (t.float().view(B, C, Hkv, d).transpose(1, 2) for t in (s["k"], s["v"]))
    seen = (torch.arange(C, device="cuda") < s["len"][:, None])[:, None, None, :]
    s1 = (qh @ kp.transpose(1, 2) * scale).view(Hkv, B, Hq // Hkv, P).transpose(0, 1)
    s2 = (q @ ko.transpose(2, 3) * scale).masked_fill(~seen, float("-inf"))
    top = s2.amax(-1, keepdim=True)
    if P:
        top = torch.maximum(top, s1.amax(-1, keepdim=True))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p1, p2 = torch.exp(s1 - top), torch.exp(s2 - top)
    total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    o1 = (p1.transpose(0, 1).reshape(Hkv, B * (Hq // Hkv), P) @ vp).view(Hkv, B, Hq // Hkv, d).transpose(0, 1)
    share = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    a = (o1 + p2 @ vo) * share
    wt = None
    if case["weights"]:
        wt = (p2 * share).sum(2) + _by_head(s["wt"], case)
        wt = _by_source(wt.masked_fill(~seen[:, 0], 0.0), case)
    return _some(a=a.reshape(B, Hq * d).to(BF16), weights=wt)


def _plain_evict(s):
    case = s["case"]
    B, Hkv, d, C, n = (case[k] for k in ("B", "Hkv", "d", "C", "budget"))
    at = torch.arange(C, device="cuda")
    length = s["len"].long()[:, None, None]
    wt = _by_head(s["wt"], case)
    key = wt.masked_fill((at < case["first"]) | (at >= length - case["recent"]), float("inf")).masked_fill(at >= length, float("-inf"))
    kept = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n]
    kept = torch.sort(kept.masked_fill(kept >= length, C), dim=-1).values
    there = kept < C
    src = kept.clamp_max(C - 1)
    new_wt = torch.gather(wt, 2, src).masked_fill(~there, 0.0)
    place = src[..., None].expand(-1, -1, -1, d)
    ko, vo = (torch.gather(t.view(B, C, Hkv, d).transpose(1, 2), 2, place).masked_fill(~there[..., None], 0.0)
              .transpose(1, 2).reshape(B * n, Hkv * d) for t in (s["k"], s["v"]))
    return _some(k=ko, v=vo, weights=_by_source(new_wt, case), lengths=s["len"].clamp_max(n),
                 kept=_by_source(kept.masked_fill(~there, -1).to(torch.int32), case))


_PLAIN = {"norm": _plain_norm, "linear": _plain_linear, "attn": _plain_attn, "evict": _plain_evict}


# ---- what a pass cannot do without -----------------------------------------------------
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1, "none": 0}


def work(case):
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        scale = 4 * T if case["y"] == "e4m3" else 0
        return {"bytes": T * D * (case["n"] * _SIZE[case["x"]] + 2 * _SIZE[case["res"]] + _SIZE[case["y"]]) + 2 * D + scale,
                "flops": T * D * (case["n"] + 5)}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        size = _SIZE[case["in"]]
        scales = 4 * (T + N) if case["in"] == "e4m3" else 0
        return {"bytes": (T + N) * K * size + T * N * (_SIZE[case["res"]] + _SIZE[case["y"]]) + (4 * N if case["bias"] else 0) + scales,
                "flops": 2 * T * K * N}
    B, C, d, Hkv = case["B"], case["C"], case["d"], case["Hkv"]
    lengths = _length_list(case)
    keys = sum(lengths)
    if case["op"] == "attn":
        Hq, P = case["Hq"], case["P"]
        wt = 4 * Hkv * (keys + B * C) if case["weights"] else 0
        return {"bytes": 4 * B * Hq * d + 4 * Hkv * d * (P + keys) + wt + 4 * B,
                "flops": 4 * Hq * d * (B * P + keys)}
    kept = sum(min(x, case["budget"]) for x in lengths)
    # scores of the caches that lose keys are all read; the others' are copied with their keys
    over = sum(x for x in lengths if x > case["budget"])
    fit = keys - over
    return {"bytes": Hkv * (4 * (over + fit) + 4 * kept + 8 * d * kept + 4 * B * case["budget"]) + 8 * B, "flops": Hkv * over}


# ---- the definition in 64 bits -----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        total = s["x"][0].to(f8)
        for x in s["x"][1:]:
            total = total + x.to(f8)
        res = None
        if s["res"] is not None:
            total = total + s["res"].to(f8)
            res = total
        norm = (total.pow(2).sum(1) / case["D"] + EPS).sqrt()
        y = total / norm[:, None] * s["w"].to(f8)
        if case["y"] != "e4m3":
            return _some(y=y, res=res)
        scale = torch.clamp(y.abs().max(1).values, min=SCALE_FLOOR) / E4M3_MAX
        return _some(y=y / scale[:, None], scale=scale, res=res)
    if case["op"] == "linear":
        out = []
        w = s["w"].to(f8)
        for r0 in range(0, case["T"], 512):  # rows in blocks: a 64-bit copy of one block at a time
            x = s["x"][r0:r0 + 512].to(f8)
            if s["xs"] is not None:
                x = x * s["xs"][r0:r0 + 512, None].to(f8)
            z = torch.matmul(x, w.T)
            if s["ws"] is not None:
                z *= s["ws"].to(f8)
            if s["bias"] is not None:
                z += s["bias"].to(f8)
            if case["act"] == "relu":
                z = torch.where(z > 0, z, torch.zeros_like(z))
            elif case["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif case["act"] == "gelu":
                z = z * torch.special.ndtr(z)
            if s["res"] is not None:
                z = z + s["res"][r0:r0 + 512].to(f8)
            out.append(z)
        return {"y": torch.cat(out)}
    B, C, d, Hkv = case["B"], case["C"], case["d"], case["Hkv"]
    lengths = s["len"].tolist()
    nkv, hr = _kv_sources(case)
    if case["op"] == "attn":
        Hq, P = case["Hq"], case["P"]
        G = Hq // Hkv
        a = torch.zeros(B, Hq, d, dtype=f8, device="cuda")
        wt = s["wt"].to(f8).clone()
        for h in range(Hkv):
            kp, vp = s["kp"][:, h * d:(h + 1) * d].to(f8), s["vp"][:, h * d:(h + 1) * d].to(f8)
            for b in range(B):
                n = lengths[b]
                k = torch.cat([kp, s["k"][b * C:b * C + n, h * d:(h + 1) * d].to(f8)])
                v = torch.cat([vp, s["v"][b * C:b * C + n, h * d:(h + 1) * d].to(f8)])
                row = wt[h // hr, b * hr + h % hr]
                row[n:] = 0.0
                if P + n == 0:
                    continue
                p = torch.softmax(s["q"][b].view(Hq, d)[h * G:(h + 1) * G].to(f8) @ k.T / math.sqrt(d), dim=1)
                a[b, h * G:(h + 1) * G] = p @ v
                row[:n] += p[:, P:].sum(0)
        return _some(a=a.view(B, Hq * d), weights=wt if case["weights"] else None)
    # eviction: of the keys between the first and the recent ones, those with the most weight, the lower index first
    size = case["budget"]
    k, v = torch.zeros(B * size, Hkv * d, dtype=f8, device="cuda"), torch.zeros(B * size, Hkv * d, dtype=f8, device="cuda")
    wt = torch.zeros(nkv, B * hr, size, dtype=f8, device="cuda")
    for b in range(B):
        n = lengths[b]
        for h in range(Hkv):
            row = s["wt"][h // hr, b * hr + h % hr, :n]
            kept = list(range(n))
            if n > size:
                middle = range(case["first"], n - case["recent"])
                value = row.tolist()
                best = sorted(middle, key=lambda j: (-value[j], j))[:size - case["first"] - case["recent"]]
                kept = sorted(set(kept) - set(middle) | set(best))
            src = torch.tensor(kept, dtype=torch.int64, device="cuda")
            at, cols = slice(b * size, b * size + len(kept)), slice(h * d, (h + 1) * d)
            k[at, cols], v[at, cols] = s["k"][b * C + src, cols].to(f8), s["v"][b * C + src, cols].to(f8)
            wt[h // hr, b * hr + h % hr, :len(kept)] = row[src].to(f8)
    return {"k": k, "v": v, "weights": wt, "lengths": None, "kept": None}
