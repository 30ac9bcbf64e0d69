"""The operators of attention over long contexts, as cases that can be timed.

Four operators, each in its plain form (elementary torch operations in 32 bits) and through the
library's calls:

  rotary  rotation of q and k by positions with one or several axes (time, height, width)
          (tp_rotary)
  window  attention of a prompt's tokens, or of a later chunk of it, over a sliding window and a few
          first tokens that stay visible                             (tp_window_attn)
  store   new keys and values into caches held in 4 bits, and read back as the values that the
          codes stand for                                            (tp_cache4_store, tp_cache4_load)
  cache4  attention of one new token per sequence over those caches, with window and first tokens
          (tp_cache4_attn)

``own = False`` runs the plain forms, ``own = True`` the library's calls.
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
ALL = 2 ** 31 - 1  # a window that hides nothing
GROUP = 32         # values of a head that share a scale in the 4-bit cache


def listed():
    return [
        # one token of one sequence far into its context: nothing but latency
        {"name": "rotary_token", "op": "rotary", "tp": 1, "T": 1, "Hq": 16, "Hkv": 4, "d": 128, "rot": 128, "axes": "64",
         "layout": "halves", "type": "bf16", "first": 100000, "theta": 1e6},
        # an odd prefill whose heads are rotated in part, neighbouring values as pairs, held in f32
        {"name": "rotary_partial_f32", "op": "rotary", "tp": 2, "T": 2047, "Hq": 16, "Hkv": 4, "d": 64, "rot": 32, "axes": "16",
         "layout": "neighbours", "type": "f32", "first": 0, "theta": 1e4},
        # a prefill of text and video tokens with time, height and width axes, over eight ranks
        {"name": "rotary_video_tp8", "op": "rotary", "tp": 8, "T": 8192, "Hq": 64, "Hkv": 8, "d": 128, "rot": 128,
         "axes": "16+24+24", "layout": "halves", "type": "bf16", "first": 0, "theta": 1e6},
        # one new token over a bf16 cache, window far below the context: latency
        {"name": "window_token_tp8", "op": "window", "tp": 8, "T": 1, "S": 8000, "Hq": 64, "Hkv": 8, "d": 128, "window": 4096,
         "sinks": 4},
        # an odd chunk of a prompt behind earlier chunks, kv heads replicated over the ranks
        {"name": "window_chunk_rep", "op": "window", "tp": 8, "T": 515, "S": 2563, "Hq": 32, "Hkv": 4, "d": 128, "window": 512,
         "sinks": 1},
        # a short prompt of a small model: heads of 64, a group of four, a window that is no whole block
        {"name": "window_prompt_d64", "op": "window", "tp": 2, "T": 2047, "S": 2047, "Hq": 16, "Hkv": 4, "d": 64, "window": 300,
         "sinks": 4},
        # the largest: a long prompt over eight ranks
        {"name": "window_prompt_tp8", "op": "window", "tp": 8, "T": 16384, "S": 16384, "Hq": 64, "Hkv": 8, "d": 128,
         "window": 1024, "sinks": 4},
        # a decode batch's new keys and values go into ragged caches
        {"name": "store_step_tp8", "op": "store", "tp": 8, "B": 61, "n": 1, "Hkv": 8, "d": 128, "C": 4096, "lo": 0, "hi": 4095},
        # a prompt's keys and values go into its cache
        {"name": "store_prompt", "op": "store", "tp": 1, "B": 1, "n": 16384, "Hkv": 8, "d": 128, "C": 16500, "lo": 7, "hi": 7},
        # a single conversation, short and odd: latency
        {"name": "cache4_single", "op": "cache4", "tp": 1, "B": 1, "Hq": 16, "Hkv": 4, "d": 128, "C": 640, "lo": 577, "hi": 577,
         "window": ALL, "sinks": 0},
        # a decode batch with a window over ragged caches, some still empty
        {"name": "cache4_window_tp8", "op": "cache4", "tp": 8, "B": 61, "Hq": 64, "Hkv": 8, "d": 128, "C": 4096, "lo": 0,
         "hi": 4096, "window": 1024, "sinks": 4},
        # the largest: long contexts of a batch, everything visible
        {"name": "cache4_long_tp8", "op": "cache4", "tp": 8, "B": 64, "Hq": 64, "Hkv": 8, "d": 128, "C": 16384, "lo": 5000,
         "hi": 16384, "window": ALL, "sinks": 0},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "window", "store", "cache4"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
    tp = rng.choice([1, 2, 4, 8])
    while hq % tp:
        tp //= 2
    if op == "rotary":
        pairs = d // 2 if rng.random() < 0.6 else _log(rng, 1, d // 2)
        axes = [pairs]
        if rng.random() < 0.5 and pairs >= 3:
            a, b = sorted(rng.sample(range(1, pairs), 2))
            axes = [a, b - a, pairs - b]
        return {"op": op, "tp": tp, "T": _log(rng, 1, 8192), "Hq": hq, "Hkv": hkv, "d": d, "rot": 2 * pairs, "axes": "+".join(map(str, axes)),
                "layout": rng.choice(["halves", "neighbours"]), "type": rng.choice(["bf16", "bf16", "f32"]),
                "first": rng.choice([0, _log(rng, 1, 1000000)]), "theta": rng.choice([1e4, 5e5, 1e6])}
    window = ALL if rng.random() < 0.2 else _log(rng, 1, 2048)
    sinks = rng.choice([0, 0, 1, 4, 4, rng.randint(5, 200)])
    if op == "window":
        t = _log(rng, 1, 4096)
        s = t if rng.random() < 0.5 else t + _log(rng, 1, 8192)
        case = {"op": op, "tp": tp, "T": t, "S": s, "Hq": hq, "Hkv": hkv, "d": d, "window": window, "sinks": sinks}
        while work(case)["flops"] > 5e11:  # many rows of an open window: fewer of them
            case["T"] //= 2
        return case
    c = _log(rng, 1, 16384)
    b = _log(rng, 1, 64 if c <= 4096 else 16)
    if op == "store":
        n = min(c, _log(rng, 1, max(1, 16384 // b)))
        hi = rng.randint(0, c - n)
        return {"op": op, "tp": min(tp, 8), "B": b, "n": n, "Hkv": hkv, "d": d, "C": c, "lo": rng.randint(0, hi), "hi": hi}
    hi = rng.randint(1, c)
    return {"op": op, "tp": tp, "B": b, "Hq": hq, "Hkv": hkv, "d": d, "C": c, "lo": rng.randint(0, hi) if b > 1 else hi, "hi": hi,
            "window": window, "sinks": sinks}


# ---- inputs ----------------------------------------------------------------------
def _length_list(case):
    return torch.linspace(case["lo"], case["hi"], case["B"], dtype=torch.float64).round().to(torch.int64).tolist()


def _kv_sources(case):
    """(number of K/V copies, kv heads in each): sharded over the ranks, or one copy where they are replicated."""
    return (case["tp"], case["Hkv"] // case["tp"]) if case["Hkv"] >= case["tp"] else (1, case["Hkv"])


def _axes(case):
    """Pairs of each axis, in order."""
    return [int(x) for x in case["axes"].split("+")]


def _columns(t, parts):
    return list(t.split(t.shape[1] // parts, dim=1))


def _normal(rows, cols, dtype, gen, std=1.0):
    return torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _positions(case, cpu):
    """int32 [axes x T]: one axis counts the tokens; of several, text counts alike on all, and frames of a
    video stand still in time while height and width run over the picture."""
    T, first = case["T"], case["first"]
    if len(_axes(case)) == 1:
        return torch.arange(first, first + T, dtype=torch.int32)[None].cuda()
    h, w = 12 + int(torch.randint(0, 9, (1,), generator=cpu)), 17 + int(torch.randint(0, 9, (1,), generator=cpu))
    text = T // 5
    i = torch.arange(max(T - text, 0))
    grid = torch.stack([i // (h * w), i // w % h, i % w]) + text
    return (torch.cat([torch.arange(text).expand(3, text), grid], 1) + first).to(torch.int32).cuda()


def _quantise(x):
    """Codes 0..15 and bf16 scales of f32 values [.., d]: scale = max|x| / 7 of 32 neighbours, value = (code - 8) * scale."""
    g = x.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1) / 7.0).to(BF16)
    s = scale.float()[..., None]
    code = torch.where(s > 0, torch.clamp(torch.round(g / torch.where(s > 0, s, torch.ones_like(s))), -8, 7), torch.zeros_like(g))
    return (code + 8).to(torch.uint8).flatten(-2), scale


def _pack(code, threads):
    """Codes of a head [.., d] to its row of d/2 bytes. Of the 32 values that share a scale, thread i of
    `threads` (4 for keys, 8 for values) has the i-th part; its parts of all groups are neighbours in the row."""
    g = code.unflatten(-1, (-1, threads, GROUP // threads // 2, 2)).transpose(-4, -3)
    return (g[..., 0] | g[..., 1] << 4).flatten(-3)


def _unpack(row, threads):
    per = GROUP // threads // 2
    g = row.unflatten(-1, (threads, -1, per))
    return torch.stack([g & 15, g >> 4], -1).transpose(-4, -3).flatten(-4)


def _decode(codes, scale, threads):
    """f32 values of rows of codes and their scales."""
    v = _unpack(codes, threads).float() - 8.0
    return (v.unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


def _filled_cache(case, threads, gen):
    """Codes and scales of a cache of normal keys (or values) with a few channels that stand out."""
    B, C, d, Hkv = case["B"], case["C"], case["d"], case["Hkv"]
    nkv, hr = _kv_sources(case)
    rows = B * hr * C
    codes = torch.empty(nkv, rows, d // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(nkv, rows, d // GROUP, dtype=BF16, device="cuda")
    channel = 1.0 + 3.0 * (torch.rand(d, generator=gen, device="cuda") < 0.05)
    for s in range(nkv):
        for r in range(0, rows, 1 << 20):
            part = slice(r, min(rows, r + (1 << 20)))
            x = torch.randn(part.stop - part.start, d, generator=gen, device="cuda") * channel
            code, scale[s, part] = _quantise(x)
            codes[s, part] = _pack(code, threads)
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 41)
    cpu = torch.Generator().manual_seed(seed * 1000003 + 53)
    s = {"case": case}
    n, d, Hkv = case["tp"], case["d"], case["Hkv"]
    nkv, hr = _kv_sources(case)
    op = case["op"]
    if op == "rotary":
        T, Hq, dt = case["T"], case["Hq"], TYPES[case["type"]]
        s["q"], s["k"] = _normal(T, Hq * d, dt, gen), _normal(T, Hkv * d, dt, gen)
        s["pos"] = _positions(case, cpu)
        pairs = case["rot"] // 2
        s["freq"] = (case["theta"] ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
        s["axis"] = torch.repeat_interleave(torch.arange(len(_axes(case))), torch.tensor(_axes(case))).cuda()
        s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    elif op == "window":
        T, S, Hq = case["T"], case["S"], case["Hq"]
        s["q"] = _normal(T, Hq * d, BF16, gen, 2.0)
        s["k"], s["v"] = (_normal(S, Hkv * d, BF16, gen) for _ in range(2))
        s["a"] = torch.empty(T, Hq * d, dtype=BF16, device="cuda")
    else:
        B, C = case["B"], case["C"]
        every = torch.linspace(case["lo"], case["hi"], B, dtype=torch.float64).round().to(torch.int32)
        s["len"] = every[torch.randperm(B, generator=cpu)].cuda()
        if op == "store":
            s["k"], s["v"] = (_normal(B * case["n"], Hkv * d, BF16, gen) for _ in range(2))
            for name in ("k", "v"):
                s[name + "c"] = torch.zeros(nkv, B * hr * C, d // 2, dtype=torch.uint8, device="cuda")
                s[name + "s"] = torch.zeros(nkv, B * hr * C, d // GROUP, dtype=BF16, device="cuda")
                s[name + "o"] = torch.empty(B * case["n"], Hkv * d, dtype=BF16, device="cuda")
        else:
            s["kc"], s["ks"] = _filled_cache(case, 4, gen)
            s["vc"], s["vs"] = _filled_cache(case, 8, gen)
            s["q"] = _normal(B, case["Hq"] * d, BF16, gen, 2.0)
            s["a"] = torch.empty(B, case["Hq"] * d, dtype=BF16, device="cuda")
    if own:
        import tensor_sharded_linear_gqa_gb300 as tp

        s["tp"] = tp
        hq = case.get("Hq", max(Hkv, n))
        s["plan"] = tp.tp_plan_create(n, hq * d, hq, Hkv, d, n)
        if op == "rotary":
            s["axis_own"] = tp.rotary_axes(_axes(case))
        if op in ("store", "cache4"):  # the caches outlive the calls: their descriptors are made once
            for name in ("kc", "ks", "vc", "vs"):
                s[name + "_own"] = tp.arr(list(s[name]))
        size = 0
        if op == "window":
            size = tp.tp_window_attn_workspace_size(s["plan"], case["T"], case["S"], case["window"], case["sinks"])
        if op == "cache4":
            size = tp.tp_cache4_attn_workspace_size(s["plan"], case["B"], case["C"], case["window"], case["sinks"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        for name, parts in (("q", n), ("qo", n), ("a", n), ("k", nkv), ("v", nkv), ("ko", nkv), ("vo", nkv)):
            if name in s:
                s[name + "r"] = _columns(s[name], parts)
    return s


# ---- one pass ----------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    tp, case = s["tp"], s["case"]
    if case["op"] == "rotary":
        tp.tp_rotary(s["plan"], s["pos"], s["freq"], s["qr"], s["kr"], s["qor"], s["kor"], axis=s["axis_own"],
                     layout=tp.TP_ROTARY_HALVES if case["layout"] == "halves" else tp.TP_ROTARY_NEIGHBOURS)
        return {"q": s["qo"], "k": s["ko"]}
    if case["op"] == "window":
        tp.tp_window_attn(s["plan"], s["qr"], s["kr"], s["vr"], case["window"], case["sinks"], s["ar"], s["ws"])
        return {"a": s["a"]}
    cache = s["kc_own"], s["ks_own"], s["vc_own"], s["vs_own"]
    if case["op"] == "store":
        tp.tp_cache4_store(s["plan"], s["len"], s["kr"], s["vr"], *cache)
        tp.tp_cache4_load(s["plan"], s["len"], *cache, s["kor"], s["vor"])
        return {"k": s["ko"], "v": s["vo"]}
    tp.tp_cache4_attn(s["plan"], s["qr"], *cache, s["len"], case["window"], case["sinks"], s["ar"], s["ws"])
    return {"a": s["a"]}


# ---- plain forms ---------------------------------------------------------------------
def _pairs(x, pairs, layout):
    """First and second value of every pair of x [.., 2 * pairs]."""
    if layout == "halves":
        return x[..., :pairs], x[..., pairs:]
    return x[..., 0::2], x[..., 1::2]


def _plain_rotary(s):
    case = s["case"]
    d, pairs = case["d"], case["rot"] // 2
    angle = s["pos"].double()[s["axis"]].t() * s["freq"].double()  # far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].float().unflatten(1, (-1, d))
        a, b = _pairs(x[..., :2 * pairs], pairs, case["layout"])
        ra, rb = a * cos - b * sin, a * sin + b * cos
        turned = torch.cat([ra, rb], -1) if case["layout"] == "halves" else torch.stack([ra, rb], -1).flatten(-2)
        out[name] = torch.cat([turned, x[..., 2 * pairs:]], -1).flatten(1).to(s[name].dtype)
    return out


def _plain_window(s):
    case = s["case"]
    T, S, Hq, Hkv, d, window, sinks = (case[k] for k in ("T", "S", "Hq", "Hkv", "d", "window", "sinks"))
    G = Hq // Hkv
    k, v = (t.view(S, Hkv, d).transpose(0, 1).float() for t in (s["k"], s["v"]))
    out = torch.empty(T, Hkv, G, d, dtype=BF16, device="cuda")
    step = 512
    for t0 in range(0, T, step):  # rows in blocks, each over the keys that some row of it sees
        t1 = min(T, t0 + step)
        at = torch.arange(S - T + t0, S - T + t1, device="cuda")
        lo, hi = max(0, S - T + t0 - window + 1), S - T + t1
        first = min(sinks, lo)
        j = torch.cat([torch.arange(first, device="cuda"), torch.arange(lo, hi, device="cuda")])
        kb, vb = (torch.cat([x[:, :first], x[:, lo:hi]], 1) for x in (k, v))
        hidden = (j > at[:, None]) | ((j <= at[:, None] - window) & (j >= sinks))
        q = s["q"][t0:t1].view(-1, Hkv, G, d).permute(1, 2, 0, 3).float()
        score = (q @ kb[:, None].transpose(2, 3) / math.sqrt(d)).masked_fill_(hidden, float("-inf"))
        p = torch.exp(score - score.amax(-1, keepdim=True))
        a = (p @ vb[:, None]) / p.sum(-1, keepdim=True)
        out[t0:t1] = a.permute(2, 0, 1, 3)
    return {"a": out.view(T, Hq * d)}


def _plain_store(s):
    case = s["case"]
    B, n, C, d = (case[k] for k in ("B", "n", "C", "d"))
    nkv, hr = _kv_sources(case)
    at = s["len"].long()[:, None] + torch.arange(n, device="cuda")                        # [B, n]
    row = (torch.arange(B * hr, device="cuda").view(B, 1, hr) * C + at[..., None])        # [B, n, heads]
    out = {}
    for name, threads in (("k", 4), ("v", 8)):
        x = s[name].float().view(B, n, nkv, hr, d)
        code, scale = _quantise(x)
        code = _pack(code, threads)
        for src in range(nkv):
            s[name + "c"][src][row] = code[:, :, src]
            s[name + "s"][src][row] = scale[:, :, src]
        back = [_decode(s[name + "c"][src][row], s[name + "s"][src][row], threads) for src in range(nkv)]
        out[name] = torch.stack(back, 2).view(B * n, -1).to(BF16)
    return out


def _plain_cache4(s):
    case = s["case"]
    B, C, d, Hq, Hkv, window, sinks = (case[k] for k in ("B", "C", "d", "Hq", "Hkv", "window", "sinks"))
    nkv, hr = _kv_sources(case)
    G = Hq // Hkv
    q = s["q"].float().view(B, nkv, hr, G, d)
    out = torch.empty(B, nkv, hr, G, d, dtype=BF16, device="cuda")
    j = torch.arange(C, device="cuda")
    step = max(1, (1 << 18) // max(1, hr * C))
    for b0 in range(0, B, step):  # sequences in blocks: an f32 copy of one block's caches at a time
        b1 = min(B, b0 + step)
        length = s["len"][b0:b1].long()[:, None]
        seen = ((j < length) & ((j >= length - window) | (j < sinks)))[:, None, None, :]
        for src in range(nkv):
            rows = slice(b0 * hr * C, b1 * hr * C)
            k, v = (_decode(s[c + "c"][src, rows], s[c + "s"][src, rows], t).view(b1 - b0, hr, C, d) for c, t in (("k", 4), ("v", 8)))
            score = (q[b0:b1, src] @ k.transpose(2, 3) / math.sqrt(d)).masked_fill(~seen, float("-inf"))
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
            total = p.sum(-1, keepdim=True)
            out[b0:b1, src] = torch.where(total > 0, (p @ v) / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(total))
    return {"a": out.view(B, Hq * d)}


_PLAIN = {"rotary": _plain_rotary, "window": _plain_window, "store": _plain_store, "cache4": _plain_cache4}


# ---- what a pass cannot do without -----------------------------------------------------
def _seen(position, window, sinks):
    """Keys that the query at `position` sees."""
    lo = max(0, position - window + 1)
    return position + 1 - lo + min(sinks, lo)


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "rotary":
        n = case["T"] * (case["Hq"] + Hkv)
        return {"bytes": 2 * n * d * (4 if case["type"] == "f32" else 2) + 4 * case["T"] * len(_axes(case)) + 2 * case["rot"],
                "flops": 3 * n * case["rot"]}
    if case["op"] == "window":
        T, S, Hq, window, sinks = (case[k] for k in ("T", "S", "Hq", "window", "sinks"))
        pairs = sum(_seen(S - T + i, window, sinks) for i in range(T))
        keys = S - max(0, S - T - window + 1) + min(sinks, max(0, S - T - window + 1))
        return {"bytes": 4 * T * Hq * d + 4 * keys * Hkv * d, "flops": 4 * Hq * d * pairs}
    row = d // 2 + 2 * (d // GROUP)  # bytes of a head's key or value in the cache
    if case["op"] == "store":
        heads = case["B"] * case["n"] * Hkv
        return {"bytes": 2 * heads * (2 * d + 2 * row + 2 * d) + 4 * case["B"], "flops": 2 * heads * 4 * d}
    keys = sum(_seen(x - 1, case["window"], case["sinks"]) for x in _length_list(case) if x > 0)
    return {"bytes": 2 * Hkv * keys * row + 4 * case["B"] * case["Hq"] * d + 4 * case["B"], "flops": 4 * case["Hq"] * d * keys}


# ---- the definition in 64 bits -----------------------------------------------------------
def _value_table(d, piece):
    """Byte and shift of every value of a head's row: the 32 values of a group lie in pieces of `piece`
    values; the row has the first pieces of all groups, then the second ones, and so on."""
    byte, shift = [], []
    for j in range(d):
        group, inside = divmod(j, GROUP)
        nibble = (inside // piece * (d // GROUP) + group) * piece + inside % piece
        byte.append(nibble // 2)
        shift.append(4 * (nibble % 2))
    return torch.tensor(byte, device="cuda"), torch.tensor(shift, device="cuda", dtype=torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    d, Hkv, op = case["d"], case["Hkv"], case["op"]
    nkv, hr = _kv_sources(case)
    if op == "rotary":
        pairs = case["rot"] // 2
        out = {}
        turn = torch.polar(torch.ones((), dtype=f8, device="cuda"),
                           torch.stack([s["pos"][a].to(f8) * f for a, f in zip(s["axis"].tolist(), s["freq"].to(f8))], 1))
        for name in ("q", "k"):
            x = s[name].to(f8).view(case["T"], -1, d)
            y = x.clone()
            i = torch.arange(pairs, device="cuda")
            one, two = (i, i + pairs) if case["layout"] == "halves" else (2 * i, 2 * i + 1)
            z = torch.complex(x[:, :, one], x[:, :, two]) * turn[:, None]
            y[:, :, one], y[:, :, two] = z.real, z.imag
            out[name] = y.view(case["T"], -1)
        return out
    if op == "window":
        T, S, Hq, window, sinks = (case[k] for k in ("T", "S", "Hq", "window", "sinks"))
        G = Hq // Hkv
        a = torch.empty(T, Hq, d, dtype=f8, device="cuda")
        step = 1024
        for h in range(Hkv):
            k, v = (s[n][:, h * d:(h + 1) * d].to(f8) for n in ("k", "v"))
            for t0 in range(0, T, step):
                t1 = min(T, t0 + step)
                at = torch.arange(t0, t1, device="cuda") + (S - T)
                j = torch.arange(S, device="cuda")
                j = j[(j < sinks) | (j > S - T + t0 - window)]
                j = j[j <= S - T + t1 - 1]
                gone = (j[None] > at[:, None]) | ((j[None] < at[:, None] - (window - 1)) & (j[None] >= sinks))
                q = s["q"][t0:t1, h * G * d:(h + 1) * G * d].to(f8).reshape(-1, d)
                z = (q @ k[j].T).view(t1 - t0, G, -1) / math.sqrt(d)
                z = torch.where(gone[:, None], -math.inf, z)
                a[t0:t1, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[j]
        return {"a": a.view(T, Hq * d)}
    if op == "store":
        out = {}
        for name in ("k", "v"):
            x = s[name].to(f8).view(-1, GROUP)
            scale = (x.abs().max(1, keepdim=True).values / 7).to(BF16).to(f8)
            q = torch.round(x / scale).clamp(-8, 7) * scale
            out[name] = torch.where(scale > 0, q, torch.zeros_like(q)).view(case["B"] * case["n"], Hkv * d)
        return out
    B, C, Hq, window, sinks = (case[k] for k in ("B", "C", "Hq", "window", "sinks"))
    G = Hq // Hkv
    a = torch.zeros(B, Hq, d, dtype=f8, device="cuda")
    lengths = s["len"].tolist()
    tables = {"k": _value_table(d, 8), "v": _value_table(d, 4)}
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        j = j[(j < sinks) | (j >= n - window)]
        for h in range(Hkv):
            row = (b * hr + h % hr) * C + j
            x = {}
            for name in ("k", "v"):
                byte, shift = tables[name]
                code = (s[name + "c"][h // hr][row][:, byte] >> shift) % 16
                x[name] = (code.to(f8) - 8) * s[name + "s"][h // hr][row].to(f8).repeat_interleave(GROUP, 1)
            p = torch.softmax(s["q"][b].view(Hq, d)[h * G:(h + 1) * G].to(f8) @ x["k"].T / math.sqrt(d), 1)
            a[b, h * G:(h + 1) * G] = p @ x["v"]
    return {"a": a.view(B, Hq * d)}
