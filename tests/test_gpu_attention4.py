"""Attention over the 4-bit paged cache against its formula in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from kv4_testlib import Cache4  # noqa: E402
from ops_testlib import Cache, attention, handle, i32, ok  # noqa: E402


def check(c, new, lens, heads, window=0, sinks=None, scale=None, qscale=1.0, seed=0, q=None):
    """Against the formula, with the bound of the 8-bit cache: the same roundings are made (f16 probabilities, fp32 scores, one
    rounding to bf16), and codes times their scales are exact in f16."""
    o = handle()
    T = sum(new)
    if q is None:
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        q = (torch.randn(T, heads, c.D, generator=g, device="cuda") * qscale).bfloat16()
    scale = c.D ** -0.5 if scale is None else scale
    out = torch.full((T + 1, heads, c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 1, heads), 9.0, device="cuda")
    moe.moe_attention(o, c.desc, c.batch(new, lens), q, out[:T], lse[:T], sinks, window, scale)
    ok(o)
    want, wlse, bound = attention(c, new, lens, q, scale, window, sinks)
    err = (out[:T].double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), (err / bound).max().item()
    s_mag = max(1.0, float(q.abs().max()) * 24 * c.D * abs(scale))
    assert ((lse[:T].double() - wlse).abs() <= 2.0 ** -19 * (s_mag + wlse.abs())).all()
    assert (out[T] == 9.0).all() and (lse[T] == 9.0).all()
    return out[:T], lse[:T]


@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv", [(8, 8), (16, 2), (6, 2), (20, 1), (64, 2)])
def test_decode(blk, D, heads, kv):
    """One token per sequence, caches from a single token on, ends inside a block whose unused tokens hold the largest values."""
    lens = [1, 2, blk - 1, blk, blk + 1, 333, 1000, 7 * blk]
    c = Cache4(lens, kv, D, blk, seed=1).fill(seed=blk + D + heads, poison=True)
    check(c, [1] * len(lens), lens, heads)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [4096, 40001])
def test_one_long_sequence(D, length):
    c = Cache4([length], 2, D, 64).fill(seed=length)
    check(c, [1], [length], 16, sinks=torch.randn(16, device="cuda"))


@pytest.mark.parametrize("blk,D", [(32, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("heads,kv", [(4, 4), (16, 2), (10, 1)])
@pytest.mark.parametrize("window", [0, 1, 50, 200])
def test_ragged_prompts(blk, D, heads, kv, window):
    """Sequences with no, one and many new tokens in one batch, with and without what came before."""
    new = [0, 1, 300, 17, 2, 129, 64]
    had = [40, 700, 0, 1, 129, 511, 64]
    lens = [a + b for a, b in zip(new, had)]
    c = Cache4(lens, kv, D, blk, seed=2).fill(seed=blk + heads, poison=True)
    check(c, new, lens, heads, window=window, sinks=torch.randn(heads, device="cuda") * 3)


@pytest.mark.parametrize("blk,D", [(32, 64), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("heads,kv", [(32, 32), (64, 8), (80, 8)])
@pytest.mark.parametrize("window", [0, 1, 130])
def test_ragged_prompts_of_many_heads(blk, D, heads, kv, window):
    """As above with enough rows for the tensor-core path: row tiles that are full, partly full and absent."""
    new = [0, 1, 300, 17, 2, 129, 64]
    had = [40, 700, 0, 1, 129, 511, 64]
    lens = [a + b for a, b in zip(new, had)]
    c = Cache4(lens, kv, D, blk, seed=2).fill(seed=blk + heads, poison=True)
    check(c, new, lens, heads, window=window, sinks=torch.randn(heads, device="cuda") * 3 if window != 1 else None)


def test_long_prompt_and_extreme_queries():
    c = Cache4([3000, 2500], 8, 64, 128).fill(seed=3)
    check(c, [3000, 300], [3000, 2500], 16)
    for qscale, scale in ((30.0, None), (2.0 ** 100, 2.0 ** -103), (2.0 ** -110, 2.0 ** 107), (1.0, -0.3), (1.0, 0.0)):
        check(c, [900, 700], [3000, 2500], 16, qscale=qscale, scale=scale)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 5000])
def test_windows(window):
    lens = [1, 64, 65, 130, 1000, 4097]
    c = Cache4(lens, 2, 64, 64).fill(seed=window)
    check(c, [1] * 6, lens, 16, window=window)
    check(c, [1, 2, 3, 4, 5, 6], lens, 16, window=window)


def test_many_sequences():
    n = 700
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(1, 400, (n,), generator=g).tolist()
    c = Cache4(lens, 1, 64, 64).fill(seed=1)
    check(c, [1] * n, lens, 8)


def test_extreme_scores():
    """Softmaxes that are nearly one-hot, queries near both ends of bf16's range, a query of zeros, scale of either sign."""
    lens = [200, 1500]
    c = Cache4(lens, 2, 64, 64).fill(seed=3)
    check(c, [1, 1], lens, 8, qscale=30.0)
    check(c, [1, 1], lens, 8, qscale=2.0 ** 100, scale=2.0 ** -103)
    check(c, [1, 1], lens, 8, qscale=2.0 ** -110, scale=2.0 ** 107)
    check(c, [3, 40], lens, 8, scale=-0.3)
    check(c, [3, 40], lens, 8, scale=0.0)
    check(c, [1, 20], lens, 8, q=torch.zeros(21, 8, 64, dtype=torch.bfloat16, device="cuda"))


def scaled(c, i, by):
    """Move the scale bytes of K (i = 0) or V (1), [blocks, H, blk, D] in value order, by what by(pos, d, shape) gives."""
    for b, n in enumerate(c.lens):
        for j in range(-(-n // c.blk)):
            pid = int(c.table[b, j])
            code, scale = c.unpacked(pid, i)
            pos = torch.arange(j * c.blk, (j + 1) * c.blk, device="cuda")[:, None].expand(c.blk, c.D)
            d = torch.arange(c.D, device="cuda")[None].expand(c.blk, c.D)
            c.repack(pid, i, code, torch.where(scale == 0, 0, (scale + by(pos, d)).clamp(20, 250)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv,new", [(4, 1, [1, 1]), (4, 1, [100, 40]), (32, 16, [700, 400])])
@pytest.mark.parametrize("which", ["tokens", "groups", "both", "rising", "falling"])
def test_scales_of_very_different_size(D, heads, kv, new, which):
    """V scales 2^20 and 2^40 apart between neighbouring tokens, between the head's groups, between blocks: what a group of columns
    adds up from is as exact as if the other groups were not there, and small ones beside large ones are in the sum."""
    lens = [700, 1100]
    c = Cache4(lens, kv, D, 64, seed=2).fill(seed=8)
    by = {"tokens": lambda p, d: p % 3 * 20, "groups": lambda p, d: d // 32 % 2 * -40, "both": lambda p, d: p * 7 % 11 * 4 - d // 32 * 15,
          "rising": lambda p, d: p // 16 - 40, "falling": lambda p, d: 40 - p // 16}[which]
    scaled(c, 1, by)
    check(c, new, lens, heads)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv,new", [(4, 1, [1, 1]), (32, 16, [700, 400])])
def test_keys_of_very_different_size(D, heads, kv, new):
    """A few keys 2^40 larger, which the queries rule out: the other keys' scores are as exact as if they were not there."""
    lens = [700, 1100]
    c = Cache4(lens, kv, D, 64, seed=2).fill(seed=8)
    for b, n in enumerate(lens):
        for j in range(-(-n // 64)):
            pid = int(c.table[b, j])
            code, scale = c.unpacked(pid, 0)
            big = (torch.arange(64, device="cuda") % 9 == 4)[:, None]
            code, scale = torch.where(big, 4 + 8, code), torch.where(big, 165, scale)        # -2 * 2^38 everywhere
            c.repack(pid, 0, code, scale)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.rand(sum(new), heads, D, generator=g, device="cuda").bfloat16()                # positive: scores of -2^40
    check(c, new, lens, heads, q=q)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv,window", [(4, 1, 0), (4, 1, 20), (32, 16, 0), (32, 16, 20)])
def test_tokens_that_a_row_does_not_see_take_no_bits(D, heads, kv, window):
    """Prompts from position 0 whose V grows by 2^30 every eight tokens of a block (without a window: rows see only smaller ones
    first), or with a window every other eight tokens 2^40 larger."""
    lens = [300, 150]
    c = Cache4(lens, kv, D, 64, seed=4).fill(seed=9)
    scaled(c, 1, lambda p, d: torch.where(p // 24 % 2 == 1, 40, 0) if window else torch.where(p < 8, -60, torch.where(p < 16, -30, 0)))
    check(c, lens, lens, heads, window=window)


def test_sinks_of_any_size():
    c = Cache4([100, 3], 2, 64, 64).fill(seed=5)
    for value in (-math.inf, -1e30, 0.0, 60.0, 1e30):
        s = torch.full((4,), value, device="cuda")
        check(c, [1, 3], [100, 3], 4, sinks=s)


def test_missing_blocks_leave_rows_empty():
    """A row none of whose blocks exist is zero, its lse the sink (or -inf); the status word says so."""
    o = handle()
    for new, kv in ((1, 1), (40, 1), (40, 64)):
        for sinks in (None, torch.linspace(0.5, -2.0, 2 * kv, device="cuda")):
            c = Cache4([40, 200], kv, 64, 64).fill(seed=6)
            q = torch.randn(2 * new, 2 * kv, 64, device="cuda").bfloat16()
            out, lse = torch.full_like(q, 5.0), torch.full((2 * new, 2 * kv), 5.0, device="cuda")
            c.dtable[0, 0] = -1
            moe.moe_attention(o, c.desc, c.batch([new, new], [40, 200]), q, out, lse, sinks)
            assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
            assert (out[:new] == 0).all()
            want = torch.full((2 * kv,), -math.inf, device="cuda") if sinks is None else sinks
            assert torch.allclose(lse[:new], want.expand(new, 2 * kv), rtol=0, atol=1e-6)
            ref, _, bound = attention(c, [0, new], [40, 200], q[new:], 64 ** -0.5, 0, sinks)
            assert ((out[new:].double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("heads,kv,new", [(2, 1, [1, 1]), (32, 16, [300, 40])])
def test_a_cache_of_zeros(heads, kv, new):
    """Every group zero, as a fresh cache has: outputs 0, equal weights."""
    c = Cache4([400, 100], kv, 64, 64)
    out, lse = check(c, new, [400, 100], heads)
    assert (out == 0).all()


def test_bad_metadata_sets_the_status():
    o = handle()
    c = Cache4([100, 100], 1, 64, 64).fill(seed=6)
    q = torch.randn(2, 2, 64, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    for cu, lens in (([0, 2, 1], [100, 100]), ([0, 1, 3], [100, 100]), ([0, 1, 2], [100, 0]), ([0, 1, 2], [1 << 30, 100])):
        moe.moe_attention(o, c.desc, moe.moe_kv_batch_of(i32(cu), i32(lens), c.dtable, 2), q, out)
        assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    check(c, [1, 1], [100, 100], 2)


def test_strided_queries_and_repeats():
    """Queries inside a fused projection's rows; the same call twice gives the same bits."""
    o = handle()
    lens = [3000, 50, 1]
    c = Cache4(lens, 2, 64, 64).fill(seed=7)
    fused = torch.randn(3, 16 + 4, 64, device="cuda").bfloat16()
    q = fused[:, :16]
    a, la = check(c, [1, 1, 1], lens, 16, q=q)
    for _ in range(3):
        out, lse = torch.empty_like(a), torch.empty_like(la)
        moe.moe_attention(o, c.desc, c.batch([1, 1, 1], lens), q, out, lse)
        assert torch.equal(out, a) and torch.equal(lse, la)
    moe.moe_attention(o, c.desc, c.batch([1, 1, 1], lens), q, out)        # no lse wanted
    assert torch.equal(out, a)


def test_in_a_graph():
    o = handle()
    lens = [500, 70]
    c = Cache4(lens, 2, 64, 64).fill(seed=9)
    q = torch.randn(2, 8, 64, device="cuda").bfloat16()
    out, b = torch.empty_like(q), c.batch([1, 1], lens)
    moe.moe_attention(o, c.desc, b, q, out)
    want = out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_attention(o, c.desc, b, q, out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("heads,kv,new", [(32, 16, [600, 40]), (8, 2, [1, 3]), (8, 2, [1, 1])])
def test_nan_queries_and_sinks(heads, kv, new):
    """A NaN in one row's query, or in one head's sink, makes those rows' results and log-sum-exps NaN, and no others."""
    o = handle()
    lens, T = [1500, 700], sum(new)
    c = Cache4(lens, kv, 64, 64, seed=6).fill(seed=13)
    g = torch.Generator(device="cuda").manual_seed(1)
    clean = torch.randn(T, heads, 64, generator=g, device="cuda").bfloat16()
    sinks = torch.randn(heads, generator=g, device="cuda")
    for what in ("q", "sink"):
        q, s, bad = clean.clone(), sinks.clone(), torch.zeros(T, heads, dtype=torch.bool, device="cuda")
        if what == "q":
            q[0, 1, 5] = q[T - 1, heads - 1, 63] = float("nan")
            bad[0, 1] = bad[T - 1, heads - 1] = True
        else:
            s[2] = float("nan")
            bad[:, 2] = True
        out, lse = torch.full_like(q, 9.0), torch.full((T, heads), 9.0, device="cuda")
        moe.moe_attention(o, c.desc, c.batch(new, lens), q, out, lse, s)
        ok(o)
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        want, wlse, bound = attention(c, new, lens, clean, 64 ** -0.5, 0, sinks)
        assert ((out.double() - want).abs() <= bound)[~bad].all()
        assert ((lse.double() - wlse).abs() <= 2.0 ** -19 * 64 * 24 * 5)[~bad].all()


@pytest.mark.parametrize("heads,kv,new", [(32, 16, [1, 1, 1]), (32, 16, [600, 33, 400]), (2, 1, [600, 33, 400])])
@pytest.mark.parametrize("gone", [-1, 0])
def test_blocks_before_the_window_may_be_gone(heads, kv, new, gone):
    """Table entries before the window of the first new token, dropped or another's: no row needs them, and neither kernel
    reports or reads them (block 0 holds values that would show)."""
    lens, window, blk = [1000, 333, 740], 50, 32
    c = Cache4(lens, kv, 64, blk, seed=6)
    c.table[c.table == 0] = max(set(range(1, c.codes.shape[0])) - set(c.table.flatten().tolist()))     # block 0 is another's
    c.fill(seed=12)
    c.codes[0, ..., blk * 32:] = 230
    c.dtable = i32(c.table.tolist())
    for b, (n, t) in enumerate(zip(new, lens)):
        c.dtable[b, :max(0, t - n - window + 1) // blk] = gone
    check(c, new, lens, heads, window=window, sinks=torch.randn(heads, device="cuda"))


def test_written_and_attended():
    """Through the cache's own write: prompts, then tokens one by one."""
    o = handle()
    H, D, blk = 2, 128, 64
    c = Cache4([400, 300], H, D, blk)
    g = torch.Generator(device="cuda").manual_seed(2)
    lens = [0, 0]
    for new in ([250, 63], [1, 1], [1, 0], [0, 2], [64, 1], [1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        kv = torch.randn(sum(new), 2, H, D, generator=g, device="cuda").bfloat16()
        moe.moe_kv_write(o, c.desc, c.batch(new, lens), kv[:, 0], kv[:, 1])
        check(c, new, lens, 12, seed=sum(lens))


@pytest.mark.parametrize("fmt", [moe.MOE_KV_E4M3, moe.MOE_KV_INT8, moe.MOE_KV_MXFP4])
@pytest.mark.parametrize("heads,kv,new", [(32, 16, [700, 400]), (8, 2, [1, 1])])
@pytest.mark.parametrize("power", [10, 17, 30])
def test_scores_far_beyond_the_exponent(fmt, heads, kv, new, power):
    """Scores of 2^13 to 2^33: a score's rounding is larger than the room that a probability has.  The largest score takes all;
    rows whose two largest are nearer than what their rounding may be are left out.  The output is rounded to bf16 (2^-8 at most);
    an INT8 block's scale is no power of two and enters the largest probability's exponent, which is rounded to f16: 2^-11 and as
    much from the logarithm and the power, 2^-10 in all."""
    o = handle()
    lens, T = [700, 1100], sum(new)
    c = (Cache4(lens, kv, 64, 64, seed=2) if fmt == moe.MOE_KV_MXFP4 else Cache(lens, kv, 64, 64, fmt, seed=2)).fill(seed=8)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = (torch.randn(T, heads, 64, generator=g, device="cuda") * 2.0 ** power).bfloat16()
    out = torch.empty_like(q)
    moe.moe_attention(o, c.desc, c.batch(new, lens), q, out)
    ok(o)
    assert torch.isfinite(out).all()
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        k, v = (x.repeat_interleave(heads // kv, 1).permute(1, 0, 2) for x in c.values(b, t))
        qq = q[at:at + n].double().permute(1, 0, 2)
        s = qq @ k.transpose(1, 2) / 8
        mag = (qq.abs() @ k.abs().transpose(1, 2) / 8).amax(-1)
        see = torch.arange(t, device="cuda")[None] <= torch.arange(t - n, t, device="cuda")[:, None]
        s = torch.where(see, s, -math.inf)
        top = s.topk(2, -1) if t > 1 else None
        clear = top.values[..., 0] - top.values[..., 1] > mag * 2.0 ** -18 + 40                  # e^-40: nothing in bf16
        want = v.gather(1, top.indices[..., :1].expand(-1, -1, 64))
        err = (out[at:at + n].double().permute(1, 0, 2) - want).abs()
        assert clear.float().mean() > 0.5
        assert (err <= want.abs() * (2.0 ** -8 + 2.0 ** -10) + v.abs().amax() * 1e-12)[clear].all()
        at += n
