"""The operators around the routed-expert block of a decode step, as measured workloads.

Five kinds of case: "write" (keys and values into an 8-bit paged cache, and the
touched blocks read back), "read" (a cached prefix read back), "attention" (over
that cache, for single tokens and for prompts), "linear" (a projection with
4-bit weights) and "sample" (temperature, top-k, top-p and min-p from given
random numbers).  Each has a plain form in elementary torch operations, the
framework's call, and its definition in 64 bits.
"""
import math

import torch

own = False          # True: run() makes the framework's calls; False: the plain forms

DEV = "cuda"
TINY = 2.0 ** -100   # smallest magnitude a block's scale is made for


def listed():
    return [
        # one decode step of a few sequences writes one token each: the smallest call, all latency
        dict(name="append_4", op="write", seqs=4, new=1, ctx=900, kv_heads=8, head_dim=64, block=64, fmt="e4m3", seed_len=1),
        # prompts of a batch written at once, ragged, some continuing a half-full block
        dict(name="write_prompts", op="write", seqs=6, new=2700, ctx=130, kv_heads=4, head_dim=128, block=64, fmt="int8", seed_len=2),
        # cached prefixes read back for reuse elsewhere
        dict(name="read_prefixes", op="read", seqs=5, new=13000, ctx=0, kv_heads=8, head_dim=64, block=128, fmt="e4m3", seed_len=3),
        # single-stream decode over a cache of a few thousand tokens, grouped heads, sinks
        dict(name="decode_1", op="attention", seqs=1, new=1, ctx=4321, q_heads=64, kv_heads=8, head_dim=64, block=64,
             fmt="e4m3", window=0, sinks=True, seed_len=4),
        # the same heads in a sliding-window layer, four streams, a long cache of which little is visible
        dict(name="decode_window", op="attention", seqs=4, new=1, ctx=9000, q_heads=64, kv_heads=8, head_dim=64, block=64,
             fmt="int8", window=128, sinks=True, seed_len=5),
        # a serving batch with long ragged caches: the largest stream of bytes
        dict(name="decode_batch", op="attention", seqs=64, new=1, ctx=12000, q_heads=32, kv_heads=4, head_dim=128, block=64,
             fmt="int8", window=0, sinks=False, seed_len=6),
        # a prompt's chunk against the cache that holds it and what came before: the most arithmetic
        dict(name="prompt_chunk", op="attention", seqs=2, new=2100, ctx=3000, q_heads=32, kv_heads=4, head_dim=128, block=64,
             fmt="e4m3", window=0, sinks=False, seed_len=7),
        # an attention projection of one token, MXFP4 with bias
        dict(name="project_1", op="linear", tokens=1, rows=5120, cols=2880, fmt="mxfp4", group=32, bias=True, out="bf16"),
        # an output projection over a vocabulary for four tokens, int4
        dict(name="head_4", op="linear", tokens=4, rows=151936, cols=2048, fmt="int4", group=64, bias=False, out="fp32"),
        # a projection of a batch of tokens, odd row count
        dict(name="project_13", op="linear", tokens=13, rows=4097, cols=4096, fmt="mxfp4", group=32, bias=True, out="bf16"),
        # one stream's next token, every filter on
        dict(name="sample_1", op="sample", rows=1, vocab=32000, filters="all"),
        # a batch's next tokens over a large odd vocabulary, filters mixed per row
        dict(name="sample_64", op="sample", rows=64, vocab=151643, filters="mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:                     # no drawn case costs more than the largest listed ones
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= 8e8 and w["flops"] <= (2.7e11 if case["op"] == "attention" and case["new"] > 8 else 1.3e10):
            return case


def _draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention", "linear", "linear", "sample", "sample"])
    heads = rng.choice([(64, 8, 64), (32, 4, 128), (16, 16, 64), (24, 8, 128), (32, 2, 64), (10, 1, 128), (40, 2, 128)])
    cache = dict(kv_heads=heads[1], head_dim=heads[2], block=rng.choice([32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                 seed_len=rng.randrange(1 << 20))
    if op in ("write", "read"):
        seqs = _log_int(rng, 1, 40)
        return dict(op=op, seqs=seqs, new=_log_int(rng, 1, max(2, 16000 // seqs)), ctx=_log_int(rng, 1, 700) if op == "write" else 0, **cache)
    if op == "attention":
        window = rng.choice([0, 0, 128, _log_int(rng, 1, 2000)])
        if rng.random() < 0.7:      # decode: one token or a few
            seqs = _log_int(rng, 1, 64)
            new, ctx = rng.choice([1, 1, 1, 2, 5]), _log_int(rng, 1, 12000)
        else:                       # prompts
            seqs = _log_int(rng, 1, 6)
            new, ctx = _log_int(rng, 17, 4200 // seqs), _log_int(rng, 1, 3000)
        return dict(op=op, seqs=seqs, new=new, ctx=ctx, q_heads=heads[0], window=window, sinks=rng.random() < 0.5, **cache)
    if op == "linear":
        fmt = rng.choice(["mxfp4", "int4"])
        group = 32 if fmt == "mxfp4" else rng.choice([32, 64, 128])
        cols = max(32, group) * _log_int(rng, 2, 8192 // max(32, group))
        return dict(op=op, tokens=_log_int(rng, 1, 64), rows=min(_log_int(rng, 32, 150000), 2 * 10 ** 8 // cols), cols=cols, fmt=fmt,
                    group=group, bias=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]))
    rows = _log_int(rng, 1, 64)
    return dict(op=op, rows=rows, vocab=_log_int(rng, 100, 150000), filters=rng.choice(["none", "all", "mixed"]))


# ------------------------------------------------------------------ lengths

def _lengths(case):
    """(new tokens, cache length after them) of each sequence: spread around the case's, from the case alone."""
    state, new, total = case["seed_len"] * 2654435761 % (1 << 32) or 1, [], []
    for b in range(case["seqs"]):
        state = (state * 1664525 + 1013904223) % (1 << 32)
        f = 0.5 + (state >> 8) / float(1 << 24)             # 0.5 .. 1.5
        n = case["new"] if case["new"] <= 8 else max(1, int(case["new"] * f))
        state = (state * 1664525 + 1013904223) % (1 << 32)
        f = 0.5 + (state >> 8) / float(1 << 24)
        new.append(n)
        total.append(n + int(case["ctx"] * f))
    return new, total


def _pairs(case):
    """Visible (query, key) pairs and visible keys, summed over the sequences."""
    new, total = _lengths(case)
    w, pairs, keys = case.get("window", 0), 0, 0
    for n, t in zip(new, total):
        first = t - n + 1                                   # keys the first query sees without a window
        if w:
            short = max(0, min(n, w - first))               # queries whose window is not full
            pairs += short * first + short * (short - 1) // 2 + (n - short) * min(w, t)
            keys += min(t, w + n - 1)
        else:
            pairs += n * first + n * (n - 1) // 2
            keys += t
    return pairs, keys


def work(case):
    op = case["op"]
    if op in ("write", "read"):
        new, total = _lengths(case)
        per = case["kv_heads"] * case["head_dim"] * 2
        n = sum(new)
        if op == "read":
            return {"bytes": n * per * 3, "flops": n * per}
        back = sum(t - (t - k) // case["block"] * case["block"] for k, t in zip(new, total))
        return {"bytes": n * per * 3 + back * per * 3, "flops": 2 * n * per + back * per}
    if op == "attention":
        pairs, keys = _pairs(case)
        q = sum(_lengths(case)[0]) * case["q_heads"]
        return {"bytes": keys * case["kv_heads"] * case["head_dim"] * 2 + q * (case["head_dim"] * 4 + 4),
                "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}
    if op == "linear":
        m, n, k = case["tokens"], case["rows"], case["cols"]
        scales = n * k // 32 if case["fmt"] == "mxfp4" else 2 * n * k // case["group"]
        return {"bytes": n * k // 2 + scales + (2 * n if case["bias"] else 0) + 2 * m * k + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    return {"bytes": case["rows"] * case["vocab"] * 4, "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _kv_values(shape, g, head_dim):
    """Keys or values [..., head_dim]: normal, with a few channels much larger than the rest, as trained models have."""
    v = torch.randn(shape, generator=g, device=DEV)
    loud = 1.0 + 5.0 * (torch.rand(head_dim, generator=g, device=DEV) < 0.04)
    return v * loud


def _prepare_cache(case, g):
    new, total = _lengths(case)
    B, blk, H, D = case["seqs"], case["block"], case["kv_heads"], case["head_dim"]
    per_seq = [-(-t // blk) for t in total]
    nb = sum(per_seq) + 3
    order = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(per_seq) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(per_seq):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    codes = torch.empty(nb, H, 2, blk * D, dtype=torch.uint8, device=DEV)
    scales = torch.empty(nb, H, 2, dtype=torch.float32, device=DEV)
    for i in range(2):
        x = _kv_values((nb, H, blk, D), g, D).bfloat16().float()
        s = _scale_of(x.abs().amax((2, 3)), case["fmt"])
        c = _encode(x * (1.0 / s)[..., None, None], case["fmt"])
        codes[:, :, i] = (c if i == 0 else c.transpose(2, 3)).reshape(nb, H, blk * D)
        scales[:, :, i] = s
        del x, c
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(codes=codes, scales=scales, table=table, cu=i32(cu), kv_len=i32(total), T=cu[-1], max_new=max(new), max_len=max(total))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("write", "read", "attention"):
        s.update(_prepare_cache(case, g))
        T, H, D = s["T"], case["kv_heads"], case["head_dim"]
        new, total = _lengths(case)
        if op == "write":
            kv = _kv_values((T, 2, H, D), g, D).bfloat16()
            s["k"], s["v"] = kv[:, 0], kv[:, 1]             # rows of one fused projection: strided
            back = [t - (t - k) // case["block"] * case["block"] for k, t in zip(new, total)]
            cu = [0]
            for n in back:
                cu.append(cu[-1] + n)
            s.update(cu_back=torch.tensor(cu, dtype=torch.int32, device=DEV), T_back=cu[-1])
        elif op == "read":
            s.update(cu_back=s["cu"], T_back=T)
        if op == "attention":
            Hq = case["q_heads"]
            s["q"] = (torch.randn(T, Hq, D, generator=g, device=DEV) * 1.5).bfloat16()
            s["sinks"] = torch.randn(Hq, generator=g, device=DEV) if case["sinks"] else None
            s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=DEV)
        else:
            s["k_back"] = torch.empty(s["T_back"], H, D, dtype=torch.bfloat16, device=DEV)
            s["v_back"] = torch.empty(s["T_back"], H, D, dtype=torch.bfloat16, device=DEV)
        if own:
            import bit_moe_decode_02_gb300 as moe
            fmt = moe.MOE_KV_E4M3 if case["fmt"] == "e4m3" else moe.MOE_KV_INT8
            s["cache"] = moe.moe_kv_cache_of(s["codes"], s["scales"], case["block"], case["head_dim"], fmt)
            s["batch"] = moe.moe_kv_batch_of(s["cu"], s["kv_len"], s["table"], s["T"])
            if op != "attention":
                s["batch_back"] = moe.moe_kv_batch_of(s["cu_back"], s["kv_len"], s["table"], s["T_back"])
    elif op == "linear":
        m, n, k = case["tokens"], case["rows"], case["cols"]
        s["codes"] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g, device=DEV)
        if case["fmt"] == "mxfp4":
            s["scales"] = torch.randint(117, 125, (n, k // 32), dtype=torch.uint8, generator=g, device=DEV)
        else:
            s["scales"] = (torch.randn(n, k // case["group"], generator=g, device=DEV) * 0.02).abs().half()
        s["bias"] = torch.randn(n, generator=g, device=DEV).bfloat16() if case["bias"] else None
        s["x"] = torch.randn(m, k, generator=g, device=DEV).bfloat16()
        s["y"] = torch.empty(m, n, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
        if own:
            import bit_moe_decode_02_gb300 as moe
            s["w"] = moe.moe_linear_of(s["codes"], s["scales"], s["bias"], moe.MOE_FMT_MXFP4 if case["fmt"] == "mxfp4" else moe.MOE_FMT_INT4,
                                       case["group"])
    else:
        m, v = case["rows"], case["vocab"]
        logits = torch.randn(m, v, generator=g, device=DEV) * 2.2
        logits += 6.0 * (torch.rand(m, v, generator=g, device=DEV) < 20.0 / v)      # a few likely tokens
        s["logits"] = logits.bfloat16().float()                                     # ties, as a bf16 model's logits have
        r = lambda: torch.rand(m, generator=g, device=DEV)  # noqa: E731
        s["temperature"] = 0.5 + r()
        s["top_k"] = torch.randint(1, 200, (m,), generator=g, device=DEV, dtype=torch.int32)
        s["top_p"] = 0.7 + 0.29 * r()
        s["min_p"] = 0.1 * r()
        s["u"] = r()
        if case["filters"] == "none":
            s["top_k"], s["top_p"], s["min_p"] = None, None, None
        elif case["filters"] == "mixed":
            row = torch.arange(m, device=DEV)
            s["temperature"] = torch.where(row % 8 == 7, torch.zeros_like(s["temperature"]), s["temperature"])
            s["top_k"] = torch.where(row % 4 < 2, torch.zeros_like(s["top_k"]), s["top_k"])
            s["top_p"] = torch.where(row % 4 == 3, torch.ones_like(s["top_p"]), s["top_p"])
            s["min_p"] = torch.where(row % 3 == 0, s["min_p"], torch.zeros_like(s["min_p"]))
        s["token"] = torch.empty(m, dtype=torch.int32, device=DEV)
        s["logprob"] = torch.empty(m, dtype=torch.float32, device=DEV)
    if own:
        s["ops"] = _handle()
    return s


_ops = None


def _handle():
    """The one handle that a program keeps: the operators' workspace."""
    global _ops
    if _ops is None:
        import bit_moe_decode_02_gb300 as moe
        _ops = moe.moe_ops_create()
    return _ops


# -------------------------------------------------------------- plain forms

def _scale_of(amax, fmt):
    """A block's scale from its largest magnitude: amax / 127, or the smallest 2^e with amax <= 448 * 2^e."""
    a = amax.clamp_min(TINY)
    if fmt == "int8":
        return a / torch.full_like(a, 127.0)
    m, e = torch.frexp(a)                                   # a = m * 2^e, m in [0.5, 1)
    return _pow2(e - 9 + (m > 0.875).to(torch.int32))


def _pow2(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    """Values already divided by their scale -> codes, as bytes."""
    if fmt == "int8":
        return x.clamp(-127.0, 127.0).round().to(torch.int8).view(torch.uint8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    return (codes.view(torch.int8) if fmt == "int8" else codes.view(torch.float8_e4m3fn)).float()


def _places(s, cu, T):
    """For each of the T tokens: its sequence, its position and its physical block."""
    case = s["case"]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    pos = s["kv_len"][seq].long() - (cu[seq + 1].long() - t)
    return seq, pos, s["table"][seq, pos // case["block"]].long()


def _plain_write(s):
    case = s["case"]
    blk, D, H, fmt = case["block"], case["head_dim"], case["kv_heads"], case["fmt"]
    _, pos, phys = _places(s, s["cu"], s["T"])
    touched, inv = torch.unique(phys, return_inverse=True)
    n = touched.numel()
    first = torch.full((n,), blk, device=DEV, dtype=torch.long).scatter_reduce(0, inv, pos % blk, "amin")
    fresh = (first == 0)[:, None]
    for i, new in ((0, s["k"]), (1, s["v"])):
        x = torch.nan_to_num(new.float(), nan=0.0, posinf=math.inf, neginf=-math.inf)
        amax = torch.where(x.isinf(), 0.0, x.abs()).amax(2)                     # [T, H]
        amax = torch.zeros(n, H, device=DEV).scatter_reduce(0, inv[:, None].expand(-1, H), amax, "amax")
        old = s["scales"][touched, :, i]
        scale = _scale_of(amax, fmt)
        scale = torch.where(fresh, scale, torch.maximum(old, scale))
        one = 1.0 / scale
        c = s["codes"][touched, :, i].reshape((n, H, blk, D) if i == 0 else (n, H, D, blk))
        c = c if i == 0 else c.transpose(2, 3)
        again = _encode(_decode(c.contiguous(), fmt) * torch.where(fresh, 0.0, old * one)[..., None, None], fmt)
        again = torch.where(fresh[..., None, None], torch.zeros_like(again), again)
        again[inv, :, pos % blk] = _encode(x * one[inv][..., None], fmt)
        s["codes"][touched, :, i] = (again if i == 0 else again.transpose(2, 3)).reshape(n, H, blk * D)
        s["scales"][touched, :, i] = scale


def _plain_read(s):
    case = s["case"]
    blk, D, H, fmt = case["block"], case["head_dim"], case["kv_heads"], case["fmt"]
    _, pos, phys = _places(s, s["cu_back"], s["T_back"])
    nb = s["codes"].shape[0]
    k = s["codes"][:, :, 0].reshape(nb, H, blk, D)[phys, :, pos % blk]
    v = s["codes"][:, :, 1].reshape(nb, H, D, blk)[phys, :, :, pos % blk]
    sc = s["scales"][phys]
    return [(_decode(c.contiguous(), fmt) * sc[:, :, i, None]).bfloat16() for i, c in ((0, k), (1, v))]


def _padded_cache(s, i):
    """Keys (i = 0) or values (1) of every sequence in fp32: [B, L, H, D]."""
    case = s["case"]
    blk, D, H = case["block"], case["head_dim"], case["kv_heads"]
    blocks = s["table"][:, :-(-s["max_len"] // blk)].clamp_min(0).long()          # [B, n]
    c = _decode(s["codes"][:, :, i][blocks], case["fmt"]) * s["scales"][blocks][..., i, None]
    B, n = blocks.shape
    c = c.reshape(B, n, H, blk, D) if i == 0 else c.reshape(B, n, H, D, blk).transpose(3, 4)
    return c.transpose(2, 3).reshape(B, n * blk, H, D)[:, :s["max_len"]]


def _plain_attention(s):
    case = s["case"]
    B, H, Hq, D, w = case["seqs"], case["kv_heads"], case["q_heads"], case["head_dim"], case["window"]
    seq, pos, _ = _places(s, s["cu"], s["T"])
    row = torch.arange(s["T"], device=DEV) - s["cu"][seq].long()
    n, L, G = s["max_new"], s["max_len"], Hq // H
    q = torch.zeros(B, n, Hq, D, device=DEV)
    q[seq, row] = s["q"].float()
    at = torch.full((B, n), -1, device=DEV, dtype=torch.long)
    at[seq, row] = pos
    j = torch.arange(L, device=DEV)
    see = j <= at[..., None]                                                    # [B, n, L]
    if w:
        see &= j > at[..., None] - w
    q = q.reshape(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    x = torch.matmul(q, _padded_cache(s, 0).permute(0, 2, 3, 1)).reshape(B, H, G, n, L) * D ** -0.5
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        m = torch.maximum(m, s["sinks"].reshape(1, H, G, 1, 1))
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(s["sinks"].reshape(1, H, G, 1, 1) - m)
    o = torch.matmul(e.reshape(B, H, G * n, L), _padded_cache(s, 1).permute(0, 2, 1, 3)).reshape(B, H, G, n, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[seq, row]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[seq, row]
    return [o.bfloat16(), lse]


def _plain_linear(s):
    case = s["case"]
    n, k, grp = case["rows"], case["cols"], case["group"]
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).reshape(n, k)
    if case["fmt"] == "mxfp4":
        c = c.int()
        mag, one = c & 7, (c & 1).float()
        value = torch.where(mag < 2, 0.5 * one, (1.0 + 0.5 * one) * _pow2((mag >> 1) - 1))
        w = torch.where(c >= 8, -value, value).reshape(n, k // grp, grp)
        scale = _pow2(s["scales"].int() - 127)
    else:
        w = (c.float() - 8.0).reshape(n, k // grp, grp)
        scale = s["scales"].float()
    y = torch.matmul(s["x"].float(), (w * scale[..., None]).reshape(n, k).t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.bfloat16() if case["out"] == "bf16" else y


def _plain_sample(s):
    l, t = s["logits"], s["temperature"][:, None]
    m, v = l.shape
    l = torch.where(l.isnan(), -math.inf, l)
    top = l.amax(1, keepdim=True)
    z = (l - top) * (1.0 / t.clamp_min(1e-30))
    z = torch.where(l == top, 0.0, torch.where(l.isinf(), -math.inf, z))
    weight = (torch.exp(z) * 2147483648.0).round().long()                       # exact sums: the order cannot matter
    place = torch.sort(l, dim=1, descending=True, stable=True).indices
    w = weight.gather(1, place)
    rank = torch.arange(v, device=DEV)[None]
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    w = torch.where(keep, w, 0)
    total = w.cumsum(1)
    if s["top_p"] is not None:
        p = s["top_p"][:, None].double()
        need = (p * total[:, -1:].double()).ceil().long().clamp_min(1)
        keep &= (total - w < need) | (p >= 1.0)
    if s["min_p"] is not None:
        keep &= w.double() >= s["min_p"][:, None].double().clamp(0.0, 1.0) * 2147483648.0
    w = torch.where(keep, w, 0)
    w = torch.zeros_like(w).scatter(1, place, w)                                # back in the vocabulary's order
    total = w.cumsum(1)
    u = s["u"][:, None].double().clamp(0.0, 1.0 - 2.0 ** -24)
    token = (total.double() <= u * total[:, -1:].double()).sum(1, keepdim=True)
    best = (l == top).int().argmax(1, keepdim=True)
    greedy = t <= 0
    token = torch.where(greedy, best, token)
    logprob = torch.where(greedy, 0.0, z.gather(1, token) - torch.log(total[:, -1:].float() / 2147483648.0))
    return [token[:, 0].int(), logprob[:, 0]]


# ---------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        import bit_moe_decode_02_gb300 as moe
        h = s["ops"]
        if op == "attention":
            moe.moe_attention(h, s["cache"], s["batch"], s["q"], s["out"], s["lse"], s["sinks"], s["case"]["window"])
            return [s["out"], s["lse"]]
        if op == "linear":
            moe.moe_linear(h, s["w"], s["x"], s["y"])
            return s["y"]
        if op == "sample":
            moe.moe_sample(h, s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["token"], s["logprob"])
            return [s["token"], s["logprob"]]
        if op == "write":
            moe.moe_kv_write(h, s["cache"], s["batch"], s["k"], s["v"])
        moe.moe_kv_read(h, s["cache"], s["batch_back"], s["k_back"], s["v_back"])
        return [s["k_back"], s["v_back"]] + ([s["scales"]] if op == "write" else [])
    if op == "attention":
        return _plain_attention(s)
    if op == "linear":
        return _plain_linear(s)
    if op == "sample":
        return _plain_sample(s)
    if op == "write":
        _plain_write(s)
    return _plain_read(s) + ([s["scales"]] if op == "write" else [])


# -------------------------------------------------------------------- exact

def _exact_scale(amax, fmt):
    """The stored (fp32) scale of a block, from its definition, as a Python float."""
    a = max(amax, 2.0 ** -100)
    if fmt == "int8":
        return float(torch.tensor(a / 127.0, dtype=torch.float32))
    e = math.ceil(math.log2(a / 448.0))
    while a > 448.0 * 2.0 ** e:
        e += 1
    while a <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** e


def _exact_round(y, fmt):
    """Nearest value of the format to y (in units of the scale), ties to even."""
    if fmt == "int8":
        return y.clamp(-127, 127).round()
    y = y.clamp(-448, 448)
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=y.device), e - 3)
    return torch.round(y / step) * step


def _exact_value(codes, fmt):
    if fmt == "int8":
        return codes.double() - 256.0 * (codes >= 128).double()
    c = codes.to(torch.int64)
    e, f = ((c >> 3) & 15).double(), (c & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (1.0 + f / 8.0) * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), e - 7.0))
    return torch.where(c >= 128, -mag, mag)


def _exact_sequence(s, b, i, length):
    """Keys or values of sequence b, [length, H, D], and of each token its block's scale."""
    case = s["case"]
    blk, D, H = case["block"], case["head_dim"], case["kv_heads"]
    ids = s["table"][b, :-(-length // blk)].long()
    c = _exact_value(s["codes"][ids][:, :, i], case["fmt"]) * s["scales"][ids][:, :, i, None].double()
    c = c.reshape(-1, H, blk, D) if i == 0 else c.reshape(-1, H, D, blk).permute(0, 1, 3, 2)
    return c.permute(0, 2, 1, 3).reshape(-1, H, D)[:length]


def _exact_write(s):
    case = s["case"]
    new, total = _lengths(case)
    blk, H, fmt = case["block"], case["kv_heads"], case["fmt"]
    backs, scales, at = ([], []), s["scales"].double(), 0
    for b, (n, t) in enumerate(zip(new, total)):
        start = (t - n) // blk * blk
        for i, src in ((0, s["k"]), (1, s["v"])):
            fresh = src[at:at + n].double()
            old = _exact_sequence(s, b, i, t - n)[start:]                       # what the first block holds already
            for first in range(start, t, blk):
                part = fresh[max(0, first - (t - n)):first + blk - (t - n)]
                phys = int(s["table"][b, first // blk])
                had = old.shape[0] if first == start else 0
                amax = part.abs().amax((0, 2)).tolist()
                sc = torch.tensor([_exact_scale(a, fmt) for a in amax], dtype=torch.float64, device=DEV)
                if had:
                    sc = torch.maximum(sc, scales[phys, :, i])
                    grown = (sc > scales[phys, :, i])[None, :, None]
                    held = torch.where(grown, _exact_round(old / sc[None, :, None], fmt) * sc[None, :, None], old)
                    part = torch.cat((held, _exact_round(part / sc[None, :, None], fmt) * sc[None, :, None]))
                else:
                    part = _exact_round(part / sc[None, :, None], fmt) * sc[None, :, None]
                scales[phys, :, i] = sc
                backs[i].append(part)
        at += n
    return [torch.cat(backs[0]), torch.cat(backs[1]), scales]


def _exact_attention(s):
    case = s["case"]
    new, total = _lengths(case)
    H, Hq, D, w = case["kv_heads"], case["q_heads"], case["head_dim"], case["window"]
    out, lse, at = [], [], 0
    for b, (n, t) in enumerate(zip(new, total)):
        keys, values = _exact_sequence(s, b, 0, t), _exact_sequence(s, b, 1, t)
        place = torch.arange(t - n, t, device=DEV)[:, None]
        j = torch.arange(t, device=DEV)[None]
        hidden = (j > place) | ((j <= place - w) if w else (j < 0))
        o, z = [], []
        for h in range(Hq):
            x = s["q"][at:at + n, h].double() @ keys[:, h // (Hq // H)].t() / math.sqrt(D)
            x = x.masked_fill(hidden, -math.inf)
            if s["sinks"] is not None:
                x = torch.cat((x, s["sinks"][h].double().expand(n, 1)), 1)
            z.append(torch.logsumexp(x, 1))
            o.append(torch.softmax(x, 1)[:, :t] @ values[:, h // (Hq // H)])
        out.append(torch.stack(o, 1))
        lse.append(torch.stack(z, 1))
        at += n
    return [torch.cat(out), torch.cat(lse)]


def _exact_linear(s):
    case = s["case"]
    n, k, grp = case["rows"], case["cols"], case["group"]
    if case["fmt"] == "mxfp4":
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
        scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), s["scales"].double() - 127)
    else:
        table = torch.arange(-8, 8, dtype=torch.float64, device=DEV)
        scale = s["scales"].double()
    y = []
    for r in range(0, n, 16384):
        c = s["codes"][r:r + 16384].long()
        w = torch.empty(c.shape[0], k, dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = table[c & 15], table[c >> 4]
        y.append(s["x"].double() @ (w.reshape(-1, k // grp, grp) * scale[r:r + 16384, :, None]).reshape(-1, k).t())
    y = torch.cat(y, 1)
    return y + s["bias"].double() if s["bias"] is not None else y


def _exact_sample(s):
    l = s["logits"].double().cpu()
    got = lambda name, r: None if s[name] is None else float(s[name][r])  # noqa: E731
    logprob = []
    for r in range(l.shape[0]):
        t = got("temperature", r)
        if t <= 0:
            logprob.append(0.0)
            continue
        z = (l[r] - l[r].max()) / t
        w = torch.round(torch.exp(z) * 2.0 ** 31)
        order = torch.sort(l[r].neg(), stable=True).indices                     # ties to the lower index
        k, p, q = got("top_k", r), got("top_p", r), got("min_p", r)
        if k and k > 0:
            order = order[:int(k)]
        total = torch.cumsum(w[order], 0)
        if p is not None and p < 1:
            order = order[:int((total < max(1, math.ceil(p * float(total[-1])))).sum()) + 1]
        if q is not None:
            order = order[w[order] >= q * 2.0 ** 31]
        order = order.sort().values
        total = torch.cumsum(w[order], 0)
        at = order[int((total <= got("u", r) * float(total[-1])).sum())]
        logprob.append(float(z[at]) - math.log(float(total[-1]) / 2.0 ** 31))
    return [None, torch.tensor(logprob, dtype=torch.float64)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        return _exact_attention(s)
    if op == "linear":
        return _exact_linear(s)
    if op == "sample":
        return _exact_sample(s)
    if op == "write":
        return _exact_write(s)
    new, total = _lengths(case)
    return [torch.cat([_exact_sequence(s, b, i, t)[t - n:] for b, (n, t) in enumerate(zip(new, total))]) for i in (0, 1)]
