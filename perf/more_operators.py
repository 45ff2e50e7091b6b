"""The rest of a decode step around the cache, as measured workloads.

Five kinds of case: "write" (keys and values into a paged cache of 4 bits, and the
touched blocks read back), "attention" (over that cache, for single tokens and for
prompts), "rope" (rotary positions of queries and keys), "plan" (block tables,
positions and slots of a step from the requests' lengths) and "lora" (low-rank
adapters of many requests beside a shared projection).  Each has a plain form in
elementary torch operations, the framework's call, and its definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False          # True: run() makes the framework's calls; False: the plain forms

DEV = "cuda"
TINY = 2.0 ** -100   # groups below it are kept as zeros


def listed():
    return [
        # one decode step of a few sequences writes one token each: the smallest call of the cache, all latency
        dict(name="append4_5", op="write", seqs=5, new=1, ctx=900, kv_heads=8, head_dim=64, block=64, seed_len=1),
        # prompts of a batch written at once, ragged, some continuing a half-full block
        dict(name="write4_prompts", op="write", seqs=6, new=2700, ctx=130, kv_heads=4, head_dim=128, block=64, seed_len=2),
        # single-stream decode over a cache of a few thousand tokens: grouped heads, sinks
        dict(name="attend4_1", op="attention", seqs=1, new=1, ctx=4321, q_heads=64, kv_heads=8, head_dim=64, block=64, window=0,
             sinks=True, seed_len=4),
        # a serving batch with long ragged caches: the largest stream of bytes
        dict(name="attend4_batch", op="attention", seqs=64, new=1, ctx=12000, q_heads=32, kv_heads=4, head_dim=128, block=64, window=0,
             sinks=False, seed_len=6),
        # a prompt's chunk against the cache that holds it and what came before, with sinks: the most arithmetic
        dict(name="prompt4_chunk", op="attention", seqs=2, new=2100, ctx=3000, q_heads=32, kv_heads=4, head_dim=128, block=64, window=0,
             sinks=True, seed_len=7),
        # queries and keys of one decode step, scaled for a long context by parts, rows of a fused projection
        dict(name="rope_7", op="rope", seqs=7, new=1, ctx=100000, q_heads=64, k_heads=8, head_dim=64, rot_dim=64, layout="half",
             scaling="parts", type="bf16", seed_len=8),
        # a prompt's, interleaved pairs in part of each head, an odd number of tokens
        dict(name="rope_prompt", op="rope", seqs=3, new=4111, ctx=5000, q_heads=32, k_heads=4, head_dim=128, rot_dim=96,
             layout="interleaved", scaling="none", type="bf16", seed_len=9),
        # a decode step of a serving batch: one token for most requests, some at their end, some idle
        dict(name="plan_step", op="plan", seqs=61, new=1, ctx=4000, block=64, ended=0.05, idle=0.1, short=False, seed_len=10),
        # many requests whose prompts come in at once, more than the free blocks hold
        dict(name="plan_prompts", op="plan", seqs=1000, new=900, ctx=300, block=32, ended=0.1, idle=0.2, short=True, seed_len=11),
        # one token of one request with its adapter
        dict(name="lora_1", op="lora", tokens=1, rows=5120, cols=2880, rank=16, adapters=1, type="bf16", seed_len=12),
        # a batch of requests with adapters of their own or none, odd row count
        dict(name="lora_33", op="lora", tokens=33, rows=4097, cols=4096, rank=32, adapters=20, type="bf16", seed_len=13),
        # the largest: every token of a full batch with its own adapter of a high rank
        dict(name="lora_64", op="lora", tokens=64, rows=8192, cols=8192, rank=64, adapters=64, type="fp32", seed_len=14),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:                     # no drawn case costs more than the largest listed ones
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= 4.1e8 and w["flops"] <= (2.7e11 if case["op"] == "attention" and case["new"] > 8 else 1.3e10):
            return case


def _draw(rng):
    op = rng.choice(["write", "attention", "attention", "attention", "rope", "rope", "plan", "plan", "lora", "lora"])
    heads = rng.choice([(64, 8, 64), (32, 4, 128), (16, 16, 64), (24, 8, 128), (32, 2, 64), (10, 1, 128), (40, 2, 128)])
    some = dict(seed_len=rng.randrange(1 << 20))
    cache = dict(kv_heads=heads[1], head_dim=heads[2], block=rng.choice([32, 64, 128]), **some)
    if op == "write":
        seqs = _log_int(rng, 1, 40)
        return dict(op=op, seqs=seqs, new=_log_int(rng, 1, max(2, 16000 // seqs)), ctx=_log_int(rng, 1, 700), **cache)
    if op == "attention":
        window = rng.choice([0, 0, 128, _log_int(rng, 1, 2000)])
        if rng.random() < 0.7:      # decode: one token or a few
            seqs = _log_int(rng, 1, 64)
            new, ctx = rng.choice([1, 1, 1, 2, 5]), _log_int(rng, 1, 12000)
        else:                       # prompts
            seqs = _log_int(rng, 1, 6)
            new, ctx = _log_int(rng, 17, 4200 // seqs), _log_int(rng, 1, 3000)
        return dict(op=op, seqs=seqs, new=new, ctx=ctx, q_heads=heads[0], window=window, sinks=rng.random() < 0.5, **cache)
    if op == "rope":
        dim = rng.choice([64, 64, 96, 128, 128, 192, 256])
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        return dict(op=op, seqs=_log_int(rng, 1, 16), new=_log_int(rng, 1, 1200), ctx=_log_int(rng, 1, 200000), q_heads=heads[0],
                    k_heads=rng.choice([0, heads[1]]), head_dim=dim, rot_dim=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "parts", "wavelength"]), type=rng.choice(["bf16", "bf16", "fp32"]), **some)
    if op == "plan":
        seqs = _log_int(rng, 1, 1024)
        return dict(op=op, seqs=seqs, new=_log_int(rng, 1, max(2, 400000 // seqs)), ctx=_log_int(rng, 1, 5000), block=rng.choice([32, 64, 128]),
                    ended=rng.choice([0.0, 0.05, 0.5]), idle=rng.choice([0.0, 0.1, 0.5]), short=rng.random() < 0.4, **some)
    tokens = _log_int(rng, 1, 64)
    return dict(op=op, tokens=tokens, rows=_log_int(rng, 32, 16000), cols=8 * _log_int(rng, 8, 2000), rank=8 * rng.choice([1, 2, 3, 4, 8, 16]),
                adapters=rng.randint(1, tokens), type=rng.choice(["bf16", "fp32"]), **some)


# ------------------------------------------------------------------ lengths

def _numbers(case, n):
    """n numbers in [0, 1), from the case alone."""
    state, out = case["seed_len"] * 2654435761 % (1 << 32) or 1, []
    for _ in range(n):
        state = (state * 1664525 + 1013904223) % (1 << 32)
        out.append((state >> 8) / float(1 << 24))
    return out


def _lengths(case):
    """(new tokens, cache length after them) of each sequence: spread around the case's."""
    f = _numbers(case, 2 * case["seqs"])
    new = [case["new"] if case["new"] <= 8 else max(1, int(case["new"] * (0.5 + x))) for x in f[::2]]
    return new, [n + int(case["ctx"] * (0.5 + x)) for n, x in zip(new, f[1::2])]


def _requests(case):
    """Of a step's plan: each request's new tokens (-1: it has ended), its cached tokens, free blocks, the blocks in all, the
    room for tokens."""
    new, total = _lengths(case)
    had = [t - n for n, t in zip(new, total)]
    f = _numbers(dict(seed_len=case["seed_len"] + 7), case["seqs"])
    new = [-1 if x < case["ended"] else 0 if x < case["ended"] + case["idle"] else n for n, x in zip(new, f)]
    blk = case["block"]
    need = sum(-(-(h + n) // blk) - -(-h // blk) for h, n in zip(had, new) if n > 0)
    free = int(need * 0.8) if case["short"] else need + 5
    return new, had, free, sum(-(-h // blk) for h in had) + free, sum(max(n, 0) for n in new) + 3


def _adapters(case):
    """Each token's adapter (-1: none): the first tokens have one each, some of the others share them."""
    f = _numbers(case, case["tokens"])
    n = case["adapters"]
    return [m if m < n else -1 if x < 0.2 else int(x * 1000) % n for m, x in enumerate(f)]


def _pairs(case):
    """Visible (query, key) pairs and visible keys, summed over the sequences."""
    new, total = _lengths(case)
    w, pairs, keys = case["window"], 0, 0
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
    if op == "write":
        new, total = _lengths(case)
        per = case["kv_heads"] * case["head_dim"] * 2
        n = sum(new)
        back = sum(t - (t - k) // case["block"] * case["block"] for k, t in zip(new, total))
        return {"bytes": (n + back) * per * 2 + (n + back) * per * 17 // 32, "flops": 2 * n * per + back * per}
    if op == "attention":
        pairs, keys = _pairs(case)
        q = sum(_lengths(case)[0]) * case["q_heads"]
        return {"bytes": keys * case["kv_heads"] * case["head_dim"] * 2 * 17 // 32 + q * (case["head_dim"] * 4 + 4),
                "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}
    if op == "rope":
        n = sum(_lengths(case)[0])
        values = n * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        return {"bytes": 2 * values * (2 if case["type"] == "bf16" else 4) + 4 * n + 4 * case["rot_dim"],
                "flops": 3 * n * (case["q_heads"] + case["k_heads"]) * case["rot_dim"]}
    if op == "plan":
        new, had, free, _, room = _requests(case)
        blk = case["block"]
        taken = min(free, sum(-(-(h + n) // blk) - -(-h // blk) for h, n in zip(had, new) if n > 0))
        back = sum(-(-h // blk) for h, n in zip(had, new) if n < 0)
        return {"bytes": 20 * case["seqs"] + 16 * room + 8 * (taken + back), "flops": 4 * room + 8 * case["seqs"]}
    m, n, k, r = case["tokens"], case["rows"], case["cols"], case["rank"]
    index = _adapters(case)
    used, some = len(set(index) - {-1}), sum(i >= 0 for i in index)
    return {"bytes": 2 * used * r * (n + k) + 2 * m * k + 2 * m * n * (2 if case["type"] == "bf16" else 4), "flops": 2 * some * r * (n + k)}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _kv_values(shape, g, head_dim):
    """Keys or values [..., head_dim]: normal, with a few channels much larger than the rest, as trained models have."""
    v = torch.randn(shape, generator=g, device=DEV)
    loud = 1.0 + 5.0 * (torch.rand(head_dim, generator=g, device=DEV) < 0.04)
    return v * loud


def _starts(new):
    return _i32(np.concatenate(([0], np.cumsum(new))).tolist())


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
    codes = torch.empty(nb, H, 2, blk * D * 17 // 32, dtype=torch.uint8, device=DEV)
    for i in range(2):
        codes[:, :, i] = _pack(*_quantise(_kv_values((nb, H, blk, D), g, D).bfloat16()), i)
    return dict(codes=codes, table=table, cu=_starts(new), kv_len=_i32(total), T=sum(new), max_new=max(new), max_len=max(total))


def _prepare_plan(case, g):
    new, had, free, blocks, room = _requests(case)
    blk, B = case["block"], case["seqs"]
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    per = [-(-h // blk) for h in had]
    table = torch.full((B, max(-(-(h + max(n, 0)) // blk) for h, n in zip(had, new)) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    head = int(torch.randint(0, blocks, (1,), generator=g, device=DEV))
    ring = torch.full((blocks,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(free, device=DEV)) % blocks] = order[at:]
    e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device=DEV)  # noqa: E731
    return dict(n_new=_i32(new), had=_i32(had), table=table, ring=ring, pool=_i32([head, free]), room=room, kv_len=e(B), cu=e(B + 1),
                seq=e(room), position=e(room), slot=e(room, torch.int64), pool_out=e(2), admitted=e(1))


ROPE = {"none": dict(), "linear": dict(factor=4.0), "parts": dict(factor=32.0, length=4096, low=1.0, high=32.0),
        "wavelength": dict(factor=8.0, length=8192, low=1.0, high=4.0)}
BASE = 150000.0


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if own:
        import bit_moe_decode_02_gb300 as moe
    if op in ("write", "attention"):
        s.update(_prepare_cache(case, g))
        T, H, D = s["T"], case["kv_heads"], case["head_dim"]
        new, total = _lengths(case)
        if own:
            s["cache"] = moe.moe_kv_cache_of(s["codes"], None, case["block"], D, moe.MOE_KV_MXFP4)
            s["batch"] = moe.moe_kv_batch_of(s["cu"], s["kv_len"], s["table"], T)
        if op == "write":
            kv = _kv_values((T, 2, H, D), g, D).bfloat16()
            s["k"], s["v"] = kv[:, 0], kv[:, 1]             # rows of one fused projection: strided
            back = [t - (t - k) // case["block"] * case["block"] for k, t in zip(new, total)]
            s.update(cu_back=_starts(back), T_back=sum(back))
            s["k_back"] = torch.empty(s["T_back"], H, D, dtype=torch.bfloat16, device=DEV)
            s["v_back"] = torch.empty(s["T_back"], H, D, dtype=torch.bfloat16, device=DEV)
            if own:
                s["batch_back"] = moe.moe_kv_batch_of(s["cu_back"], s["kv_len"], s["table"], s["T_back"])
        else:
            Hq = case["q_heads"]
            s["q"] = (torch.randn(T, Hq, D, generator=g, device=DEV) * 1.5).bfloat16()
            s["sinks"] = torch.randn(Hq, generator=g, device=DEV) if case["sinks"] else None
            s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=DEV)
    elif op == "rope":
        new, total = _lengths(case)
        T, Hq, Hk, D = sum(new), case["q_heads"], case["k_heads"], case["head_dim"]
        t = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        x = torch.randn(T, Hq + Hk, D, generator=g, device=DEV).to(t)
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:] if Hk else None                  # rows of one fused projection: strided
        s["q_out"] = torch.empty(T, Hq, D, dtype=t, device=DEV)
        s["k_out"] = torch.empty(T, Hk, D, dtype=t, device=DEV) if Hk else None
        s["position"] = torch.cat([torch.arange(n - k, n, dtype=torch.int32, device=DEV) for k, n in zip(new, total)])
        s["mscale"] = 0.1 * math.log(32.0) + 1.0 if case["scaling"] == "parts" else 1.0
        if own:
            kind = dict(none=moe.MOE_ROPE_PLAIN, linear=moe.MOE_ROPE_LINEAR, parts=moe.MOE_ROPE_PARTS, wavelength=moe.MOE_ROPE_WAVELENGTH)
            layout = moe.MOE_ROPE_HALF if case["layout"] == "half" else moe.MOE_ROPE_INTERLEAVED
            s["rope"] = moe.moe_rope_of(case["rot_dim"], BASE, layout, kind[case["scaling"]], mscale=s["mscale"], **ROPE[case["scaling"]])
    elif op == "plan":
        s.update(_prepare_plan(case, g))
        if own:
            s["step"] = moe.moe_kv_pool_of(s["ring"], s["table"], case["block"])
    else:
        m, n, k, r = case["tokens"], case["rows"], case["cols"], case["rank"]
        a = case["adapters"]
        t = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        s["a"] = (torch.randn(a, r, k, generator=g, device=DEV) * k ** -0.5).bfloat16()
        s["b"] = (torch.randn(a, n, r, generator=g, device=DEV) * 0.1).bfloat16()
        s["factor"] = 0.5 + torch.rand(a, generator=g, device=DEV)
        s["index"] = _i32(_adapters(case))
        s["x"] = torch.randn(m, k, generator=g, device=DEV).bfloat16()
        s["y"] = torch.randn(m, n, generator=g, device=DEV).to(t)
        s["out"] = torch.empty_like(s["y"])
        if own:
            s["w"] = moe.moe_lora_of(s["a"], s["b"], s["factor"])
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

def _pow2(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """Keys or values [..., D] -> E2M1 codes (a byte each) and the scale bytes of their groups of 32."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=math.inf, neginf=-math.inf).unflatten(-1, (-1, 32))
    amax = torch.where(x.isinf(), 0.0, x.abs()).amax(-1)
    m, e = torch.frexp(amax.clamp_min(TINY))                # amax = m 2^e, m in [0.5, 1); 6 = 0.75 * 2^3
    e = e - 3 + (m > 0.75).int()
    zero = amax < TINY
    y = x * _pow2(-e)[..., None]
    a = torch.where(zero[..., None], 0.0, y.abs())
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where((y < 0) & (code > 0), code + 8, code)
    return code.to(torch.uint8).flatten(-2), torch.where(zero, 0, e + 127).to(torch.uint8)


def _pack(code, scale, i):
    """Codes [..., blk, D] and scale bytes [..., blk, D / 32] of K (i = 0) or V (1) -> a block's bytes."""
    lead, (blk, D) = code.shape[:-2], code.shape[-2:]
    if i == 0:
        c = code[..., 0::2] | code[..., 1::2] << 4                              # [blk, D / 2]
        z = scale.reshape(*lead, blk // 32, 4, 4, 2, D // 32).movedim(-3, -1)    # sub, t / 8, t % 2, group, t / 2 % 4
        return torch.cat((c.flatten(-2), z.flatten(-5)), -1)
    c = code[..., 0::2, :] | code[..., 1::2, :] << 4                            # two tokens a byte: [blk / 2, D]
    c = c.reshape(*lead, blk // 32, 4, 4, D // 32, 4, 8)                        # sub, c, byte, group, e, r
    c = c.movedim((-3, -1, -5, -2, -4), (-5, -4, -3, -2, -1))                   # sub, group, r, c, e, byte
    return torch.cat((c.flatten(-6), scale.unflatten(-2, (blk // 32, 32)).transpose(-1, -2).flatten(-3)), -1)


def _unpack(bytes_, i, blk, D):
    """The inverse of _pack: codes [..., blk, D] and scale bytes [..., blk, D / 32]."""
    lead, n = bytes_.shape[:-1], blk * D // 2
    c, z = bytes_[..., :n], bytes_[..., n:]
    if i == 0:
        code = torch.stack((c & 15, c >> 4), -1).reshape(*lead, blk, D)
        return code, z.reshape(*lead, blk // 32, 4, 2, D // 32, 4).movedim(-1, -3).reshape(*lead, blk, D // 32)
    c = c.reshape(*lead, blk // 32, D // 32, 8, 4, 4, 4).movedim((-3, -1, -5, -2, -4), (-5, -4, -3, -2, -1))
    c = torch.stack((c & 15, c >> 4), -4)                                       # sub, c, byte, nibble, group, e, r
    return c.reshape(*lead, blk, D), z.reshape(*lead, blk // 32, D // 32, 32).transpose(-1, -2).reshape(*lead, blk, D // 32)


def _decode(code, scale):
    c = code.int()
    mag, one = c & 7, (c & 1).float()
    value = torch.where(mag < 2, 0.5 * one, (1.0 + 0.5 * one) * _pow2((mag >> 1) - 1))
    value = torch.where(c >= 8, -value, value).unflatten(-1, (-1, 32))
    return (value * torch.where(scale == 0, 0.0, _pow2(scale.int() - 127))[..., None]).flatten(-2)


def _places(s, cu, T):
    """For each of the T tokens: its sequence, its position and its physical block."""
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    pos = s["kv_len"][seq].long() - (cu[seq + 1].long() - t)
    return seq, pos, s["table"][seq, pos // s["case"]["block"]].long()


def _plain_write_one(s, x, i):
    blk, D = s["case"]["block"], s["case"]["head_dim"]
    _, pos, phys = _places(s, s["cu"], s["T"])
    touched, inv = torch.unique(phys, return_inverse=True)
    first = torch.full((touched.numel(),), blk, device=DEV, dtype=torch.long).scatter_reduce(0, inv, pos % blk, "amin")
    code, scale = _unpack(s["codes"][touched, :, i], i, blk, D)
    fresh = (first == 0)[:, None, None, None]
    code, scale = torch.where(fresh, 0, code), torch.where(fresh, 0, scale)
    code[inv, :, pos % blk], scale[inv, :, pos % blk] = _quantise(x)
    s["codes"][touched, :, i] = _pack(code, scale, i)


def _plain_read_one(s, i):
    _, pos, phys = _places(s, s["cu_back"], s["T_back"])
    touched, inv = torch.unique(phys, return_inverse=True)
    blk = s["case"]["block"]
    return _decode(*_unpack(s["codes"][touched, :, i], i, blk, s["case"]["head_dim"]))[inv, :, pos % blk].bfloat16()


def _padded_cache(s, i):
    """Keys (i = 0) or values (1) of every sequence in fp32: [B, L, H, D]."""
    case = s["case"]
    blk, D, H = case["block"], case["head_dim"], case["kv_heads"]
    blocks = s["table"][:, :-(-s["max_len"] // blk)].clamp_min(0).long()          # [B, n]
    c = _decode(*_unpack(s["codes"][:, :, i], i, blk, D))[blocks]                 # [B, n, H, blk, D]
    B, n = blocks.shape
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


def _frequencies(case):
    """Angle of one position for each pair, in 64 bits."""
    rot, p = case["rot_dim"], ROPE[case["scaling"]]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = torch.exp(i * (-2.0 / rot * math.log(BASE)))
    if case["scaling"] == "linear":
        f = f / p["factor"]
    elif case["scaling"] == "parts":
        at = lambda turns: rot * math.log(p["length"] / (2 * math.pi * turns)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(at(p["high"]), 0.0), min(at(p["low"]), rot // 2 - 1.0)
        x = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = f * (1.0 - x) + f / p["factor"] * x
    elif case["scaling"] == "wavelength":
        x = ((p["length"] * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0.0, 1.0)
        f = f * x + f / p["factor"] * (1.0 - x)
    return f


def _plain_rotate(x, c, s, half, rot):
    """x [T, H, D], c and s [T, rot / 2] in 64 bits."""
    y, c, s = x.double(), c[:, None], s[:, None]
    u, v = (y[..., :rot // 2], y[..., rot // 2:rot]) if half else (y[..., 0:rot:2], y[..., 1:rot:2])
    a, b = u * c - v * s, v * c + u * s
    r = torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((r, y[..., rot:]), -1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    t = s["position"].double()[:, None] * _frequencies(case)
    c, sn, half, rot = torch.cos(t) * s["mscale"], torch.sin(t) * s["mscale"], case["layout"] == "half", case["rot_dim"]
    q = _plain_rotate(s["q"], c, sn, half, rot)
    return [q] if s["k"] is None else [q, _plain_rotate(s["k"], c, sn, half, rot)]


def _plain_plan(s):
    blk, room, ring = s["case"]["block"], s["room"], s["ring"]
    size, head, count = ring.numel(), s["pool"][0].long(), s["pool"][1].long()
    had, n = s["had"].long(), s["n_new"].long().clamp_min(0)
    ended = s["n_new"] < 0
    held = (had + blk - 1) // blk
    need = (had + n + blk - 1) // blk - held
    fits = (need.cumsum(0) <= count) & (n.cumsum(0) <= room)
    n, need = torch.where(fits, n, 0), torch.where(fits, need, 0)
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu, taken = torch.cat((zero, n.cumsum(0))), torch.cat((zero, need.cumsum(0)))
    # new blocks, in the order of the sequences
    k = torch.arange(int(taken[-1]), device=DEV)
    b = torch.searchsorted(taken[1:], k, right=True)
    s["table"][b, held[b] + k - taken[b]] = ring[(head + k) % size]
    t = torch.arange(room, device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    real = seq < had.numel()
    at = seq.clamp_max(had.numel() - 1)
    pos = torch.where(real, had[at] + t - cu[at], 0)
    slot = s["table"][at, pos // blk].long() * blk + pos % blk
    # blocks that come back, in the order of the sequences
    j = torch.arange(s["table"].shape[1], device=DEV)
    back = s["table"][(j[None] < held[:, None]) & ended[:, None]]
    ring[(head + count + torch.arange(back.numel(), device=DEV)) % size] = back
    count = count - taken[-1] + back.numel()
    return [cu.int(), torch.where(ended, 0, had + n).int(), s["table"], torch.where(real, seq, -1).int(), torch.where(real, pos, -1).int(),
            torch.where(real, slot, -1), ring, torch.stack(((head + taken[-1]) % size, count)).int(), fits.sum()[None].int()]


def _plain_lora(s):
    on = s["index"] >= 0
    i = s["index"].clamp_min(0).long()
    used, at = torch.unique(i, return_inverse=True)
    x = s["x"].float()
    h = torch.einsum("ark,mk->amr", s["a"][used].float(), x)                    # of every adapter in use, then the token's own
    h = h[at, torch.arange(x.shape[0], device=DEV)] * (s["factor"][i] * on)[:, None]
    one = (at[None] == torch.arange(used.numel(), device=DEV)[:, None])[..., None]
    d = torch.bmm(h[None] * one, s["b"][used].float().transpose(1, 2)).sum(0)
    return (s["y"].float() + d).to(s["y"].dtype)


# ---------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        import bit_moe_decode_02_gb300 as moe
        h = s["ops"]
        if op == "attention":
            moe.moe_attention(h, s["cache"], s["batch"], s["q"], s["out"], s["lse"], s["sinks"], s["case"]["window"])
            return [s["out"], s["lse"]]
        if op == "write":
            moe.moe_kv_write(h, s["cache"], s["batch"], s["k"], s["v"])
            moe.moe_kv_read(h, s["cache"], s["batch_back"], s["k_back"], s["v_back"])
            return [s["k_back"], s["v_back"]]
        if op == "rope":
            moe.moe_rope(h, s["rope"], s["position"], s["q"], s["k"], s["q_out"], s["k_out"])
            return [s["q_out"]] if s["k"] is None else [s["q_out"], s["k_out"]]
        if op == "plan":
            moe.moe_kv_plan(h, s["step"], s["n_new"], s["had"], s["pool"], s["cu"], s["kv_len"], s["pool_out"], s["admitted"], s["seq"],
                            s["position"], s["slot"])
            return [s["cu"], s["kv_len"], s["table"], s["seq"], s["position"], s["slot"], s["ring"], s["pool_out"], s["admitted"]]
        moe.moe_lora(h, s["w"], s["index"], s["x"], s["y"], s["out"])
        return s["out"]
    if op == "attention":
        return _plain_attention(s)
    if op == "rope":
        return _plain_rope(s)
    if op == "plan":
        return _plain_plan(s)
    if op == "lora":
        return _plain_lora(s)
    _plain_write_one(s, s["k"], 0)
    _plain_write_one(s, s["v"], 1)
    return [_plain_read_one(s, 0), _plain_read_one(s, 1)]


# -------------------------------------------------------------------- exact

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_round(x):
    """The stored values of keys or values [..., D] (numpy, 64 bits): by group of 32, from the definition."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    a = np.abs(g).max(-1, keepdims=True)
    e = np.ceil(np.log2(np.maximum(a, TINY) / 6.0))
    e = np.where(a > 6.0 * 2.0 ** e, e + 1, e)
    e = np.where((a <= 6.0 * 2.0 ** (e - 1)) & (a >= TINY), e - 1, e)
    y = np.abs(g) / 2.0 ** e
    step = np.where(y < 2.0, 0.5, np.where(y < 4.0, 1.0, 2.0))                  # distance of neighbours; a tie at a border goes up alike
    y = np.minimum(np.rint(y / step) * step, 6.0)
    return np.where(a < TINY, 0.0, np.copysign(y * 2.0 ** e, g)).reshape(x.shape)


def _exact_block(rec, i, blk, D):
    """One block of one head, bytes -> values [blk, D] in 64 bits, value by value from the layout's definition."""
    t, d = torch.arange(blk, device=DEV)[:, None], torch.arange(D, device=DEV)[None]
    sub, u, grp = t // 32, t % 32, d // 32
    n = blk * D // 2
    if i == 0:
        at, nib = t * (D // 2) + d // 2, d % 2
        z = n + sub * D + ((u // 8 * 2 + u % 2) * (D // 32) + grp) * 4 + u // 2 % 4
    else:
        word = ((sub * (D // 32) + grp) * 8 + d % 8) * 16 + u // 8 * 4 + d // 8 % 4
        at, nib = word * 4 + u % 8 // 2, u % 2
        z = n + (sub * (D // 32) + grp) * 32 + u
    code = rec[..., at].long() >> (4 * nib) & 15
    scale = rec[..., z].double()
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=DEV)[code]
    return torch.where(scale == 0, 0.0, v * torch.pow(2.0, scale - 127.0))


def _exact_sequence(s, b, i, length):
    """Keys or values of sequence b, [length, H, D], in 64 bits."""
    case = s["case"]
    blk, D, H = case["block"], case["head_dim"], case["kv_heads"]
    rec = s["codes"][s["table"][b, :-(-length // blk)].long(), :, i]
    return _exact_block(rec, i, blk, D).transpose(1, 2).reshape(-1, H, D)[:length]


def _exact_write(s):
    new, total = _lengths(s["case"])
    blk, out, at = s["case"]["block"], ([], []), 0
    for b, (n, t) in enumerate(zip(new, total)):
        start = (t - n) // blk * blk
        for i, src in ((0, s["k"]), (1, s["v"])):
            if t - n > start:                                                   # what the first block holds already
                out[i].append(_exact_sequence(s, b, i, t - n)[start:].cpu().numpy())
            out[i].append(_exact_round(src[at:at + n].double().cpu().numpy()))
        at += n
    return [torch.from_numpy(np.concatenate(o)) for o in out]


def _exact_attention(s):
    case = s["case"]
    new, total = _lengths(case)
    H, Hq, D, w = case["kv_heads"], case["q_heads"], case["head_dim"], case["window"]
    out, lse, at = [], [], 0
    for b, (n, t) in enumerate(zip(new, total)):
        keys, values = (_exact_sequence(s, b, i, t) for i in (0, 1))
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


def _exact_rope(s):
    """Complex rotation with angles reduced in numpy, pair by pair."""
    case = s["case"]
    rot, p, kind = case["rot_dim"], ROPE[case["scaling"]], case["scaling"]
    pos = s["position"].cpu().numpy().astype(np.float64)
    turn = []
    for i in range(rot // 2):
        f = BASE ** (-2.0 * i / rot)
        slow = f / p.get("factor", 1.0)
        if kind == "linear":
            f = slow
        elif kind == "parts":
            lo, hi = (rot * math.log(p["length"] / (2 * math.pi * x)) / (2 * math.log(BASE)) for x in (p["high"], p["low"]))
            lo, hi = max(lo, 0.0), min(hi, rot // 2 - 1.0)
            x = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = (1 - x) * f + x * slow
        elif kind == "wavelength":
            length = 2 * math.pi / f
            if length > p["length"] / p["low"]:
                f = slow
            elif length >= p["length"] / p["high"]:
                x = (p["length"] / length - p["low"]) / (p["high"] - p["low"])
                f = x * f + (1 - x) * slow
        turn.append(np.exp(1j * pos * f) * s["mscale"])
    turn = torch.from_numpy(np.stack(turn, 1)).to(DEV)[:, None]
    out = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        y = x.double()
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) if case["layout"] == "half" else torch.complex(y[..., 0:rot:2], y[..., 1:rot:2])
        z = z * turn
        r = torch.cat((z.real, z.imag), -1) if case["layout"] == "half" else torch.view_as_real(z).flatten(-2)
        out.append(torch.cat((r, y[..., rot:]), -1))
    return out


def _exact_lora(s):
    out = s["y"].double()
    for m, i in enumerate(s["index"].tolist()):
        if i >= 0:
            out[m] += float(s["factor"][i]) * (s["b"][i].double() @ (s["a"][i].double() @ s["x"][m].double()))
    return out


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None                                                             # whole numbers
    s = prepare(case, seed)
    return dict(attention=_exact_attention, rope=_exact_rope, lora=_exact_lora, write=_exact_write)[op](s)
