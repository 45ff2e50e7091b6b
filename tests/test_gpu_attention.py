"""Attention over the 8-bit paged cache against its formula in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import Cache, attention, handle, i32, ok  # noqa: E402

FMTS = [moe.MOE_KV_E4M3, moe.MOE_KV_INT8]


def check(c, new, lens, heads, window=0, sinks=None, scale=None, qscale=1.0, seed=0, q=None):
    o = handle()
    T = sum(new)
    if q is None:
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        q = (torch.randn(T, heads, c.D, generator=g, device="cuda") * qscale).bfloat16()
    scale = c.D ** -0.5 if scale is None else scale
    out = torch.full((T, heads, c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), 9.0, device="cuda")
    moe.moe_attention(o, c.desc, c.batch(new, lens), q, out, lse, sinks, window, scale)
    ok(o)
    want, wlse, bound = attention(c, new, lens, q, scale, window, sinks)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), (err / bound).max().item()
    s_mag = max(1.0, float(q.abs().max()) * 8 * c.D * abs(scale))
    assert ((lse.double() - wlse).abs() <= 2.0 ** -19 * (s_mag + wlse.abs())).all()
    return out, lse


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv", [(8, 8), (16, 2), (6, 2), (20, 1), (64, 2)])
def test_decode(fmt, blk, D, heads, kv):
    """One token per sequence, caches from a single token on, ends inside a block whose unused tokens hold large codes."""
    lens = [1, 2, blk - 1, blk, blk + 1, 333, 1000, 7 * blk]
    c = Cache(lens, kv, D, blk, fmt, seed=1).fill(seed=blk + D + heads, poison=True)
    check(c, [1] * len(lens), lens, heads)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [4096, 40001])
def test_one_long_sequence(fmt, D, length):
    c = Cache([length], 2, D, 64, fmt).fill(seed=length)
    check(c, [1], [length], 16, sinks=torch.randn(16, device="cuda"))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk,D", [(32, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("heads,kv", [(4, 4), (16, 2), (10, 1)])
@pytest.mark.parametrize("window", [0, 1, 50, 200])
def test_ragged_prompts(fmt, blk, D, heads, kv, window):
    """Sequences with no, one and many new tokens in one batch, with and without what came before."""
    new = [0, 1, 300, 17, 2, 129, 64]
    had = [40, 700, 0, 1, 129, 511, 64]
    lens = [a + b for a, b in zip(new, had)]
    c = Cache(lens, kv, D, blk, fmt, seed=2).fill(seed=blk + heads, poison=True)
    check(c, new, lens, heads, window=window, sinks=torch.randn(heads, device="cuda") * 3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk,D", [(32, 64), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("heads,kv", [(32, 32), (64, 8), (80, 8)])
@pytest.mark.parametrize("window", [0, 1, 130])
def test_ragged_prompts_of_many_heads(fmt, blk, D, heads, kv, window):
    """As above with enough rows for the tensor-core path: row tiles that are full, partly full and absent."""
    new = [0, 1, 300, 17, 2, 129, 64]
    had = [40, 700, 0, 1, 129, 511, 64]
    lens = [a + b for a, b in zip(new, had)]
    c = Cache(lens, kv, D, blk, fmt, seed=2).fill(seed=blk + heads, poison=True)
    check(c, new, lens, heads, window=window, sinks=torch.randn(heads, device="cuda") * 3 if window != 1 else None)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_with_block_scales_of_very_different_size(D):
    """Scales 2^20 apart between neighbouring blocks, in V and then in K: O changes its unit at every tile, maxima jump."""
    lens = [700, 1100]
    for which in (1, 0):
        c = Cache(lens, 16, D, 64, moe.MOE_KV_E4M3).fill(seed=8)
        c.scales[:, :, which] *= torch.pow(2.0, torch.arange(c.scales.shape[0], device="cuda")[:, None] % 3 * (10.0 if which else 3.0))
        check(c, [700, 400], lens, 32)


def test_long_prompt_and_extreme_queries():
    c = Cache([3000, 2500], 8, 64, 128, moe.MOE_KV_INT8).fill(seed=3)
    check(c, [3000, 300], [3000, 2500], 16)
    for qscale, scale in ((30.0, None), (2.0 ** 100, 2.0 ** -103), (2.0 ** -110, 2.0 ** 107), (1.0, -0.3), (1.0, 0.0)):
        check(c, [900, 700], [3000, 2500], 16, qscale=qscale, scale=scale)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 5000])
def test_windows(window):
    lens = [1, 64, 65, 130, 1000, 4097]
    c = Cache(lens, 2, 64, 64, moe.MOE_KV_E4M3).fill(seed=window)
    check(c, [1] * 6, lens, 16, window=window)
    check(c, [1, 2, 3, 4, 5, 6], lens, 16, window=window)


def test_many_sequences():
    n = 700
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(1, 400, (n,), generator=g).tolist()
    c = Cache(lens, 1, 64, 64, moe.MOE_KV_INT8).fill(seed=1)
    check(c, [1] * n, lens, 8)


@pytest.mark.parametrize("fmt", FMTS)
def test_extreme_scores(fmt):
    """Softmaxes that are nearly one-hot, queries near both ends of bf16's range, a query of zeros, scale of either sign."""
    lens = [200, 1500]
    c = Cache(lens, 2, 64, 64, fmt).fill(seed=3)
    check(c, [1, 1], lens, 8, qscale=30.0)
    check(c, [1, 1], lens, 8, qscale=2.0 ** 100, scale=2.0 ** -103)
    check(c, [1, 1], lens, 8, qscale=2.0 ** -110, scale=2.0 ** 107)
    check(c, [3, 40], lens, 8, scale=-0.3)
    check(c, [3, 40], lens, 8, scale=0.0)
    check(c, [1, 20], lens, 8, q=torch.zeros(21, 8, 64, dtype=torch.bfloat16, device="cuda"))


def test_block_scales_of_very_different_size():
    """Neighbouring blocks whose scales are 2^20 apart, in K (a few keys take all) and in V."""
    c = Cache([640], 1, 128, 64, moe.MOE_KV_E4M3).fill(seed=8)
    c.scales[:, :, 1] *= torch.pow(2.0, torch.arange(c.scales.shape[0], device="cuda")[:, None] % 3 * 10.0)
    check(c, [1], [640], 4)
    check(c, [100], [640], 4)


def test_sinks_of_any_size():
    c = Cache([100, 3], 2, 64, 64, moe.MOE_KV_E4M3).fill(seed=5)
    for value in (-math.inf, -1e30, 0.0, 60.0, 1e30):
        s = torch.full((4,), value, device="cuda")
        check(c, [1, 3], [100, 3], 4, sinks=s)


def test_missing_blocks_leave_rows_empty():
    """A row none of whose blocks exist is zero, its lse the sink (or -inf); the status word says so."""
    o = handle()
    for new, kv in ((1, 1), (40, 1), (40, 64)):
        for sinks in (None, torch.linspace(0.5, -2.0, 2 * kv, device="cuda")):
            c = Cache([40, 200], kv, 64, 64, moe.MOE_KV_E4M3).fill(seed=6)
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


def test_bad_metadata_sets_the_status():
    o = handle()
    c = Cache([100, 100], 1, 64, 64, moe.MOE_KV_E4M3).fill(seed=6)
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
    c = Cache(lens, 2, 64, 64, moe.MOE_KV_INT8).fill(seed=7)
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
    c = Cache(lens, 2, 64, 64, moe.MOE_KV_E4M3).fill(seed=9)
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


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv", [(32, 16), (2, 1)])
@pytest.mark.parametrize("window", [0, 20])
def test_blocks_that_a_row_does_not_see_take_no_bits(fmt, blk, D, heads, kv, window):
    """Prompts from position 0 whose later blocks have scales of V 2^20 apart, growing over the first tile of 128 keys; with a
    window, every other block 2^20 larger: rows that see only small blocks are as exact as if the others were not there."""
    lens = [700, 300]
    c = Cache(lens, kv, D, blk, fmt, seed=4).fill(seed=9)
    for b, n in enumerate(lens):
        for j in range(-(-n // blk)):
            c.scales[int(c.table[b, j]), :, 1] *= 2.0 ** (20 * (j % 2) if window else 20 * min(j, 3))
    check(c, lens, lens, heads, window=window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("heads,kv,new", [(32, 16, 650), (32, 16, 1), (2, 1, 40)])
def test_a_much_larger_block_out_of_the_window(fmt, blk, heads, kv, new):
    """A block of V that is 2^60 larger, which earlier rows of the same call see and later ones do not."""
    c = Cache([700], kv, 64, blk, fmt, seed=4).fill(seed=10)
    big = (700 - new) // blk
    c.scales[int(c.table[0, big]), :, 1] *= 2.0 ** 60
    check(c, [new], [700], heads, window=blk)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [64, 128])
@pytest.mark.parametrize("seqs,length,new,heads,kv", [(320, 500, 1, 1, 1), (1, 3000, 600, 32, 16)])
def test_small_probabilities_add_up(fmt, blk, seqs, length, new, heads, kv):
    """One key with a score 26.5 units of log2 above all others and a value of 0, as the first token of a long context may
    be: the output is the sum of many probabilities of 2^-26.5, each of which may lose 2^-31 (2^-30 allowed)."""
    o = handle()
    c = Cache([length] * seqs, kv, 64, blk, fmt, seed=5).fill(seed=11)
    first = torch.from_numpy(c.table[:, 0].astype("int64")).cuda()
    c.codes[:, :, 0] = 0
    c.scales[:, :, 0] = 1.0
    c.codes[first, :, 0, 0] = 0x38 if fmt == moe.MOE_KV_E4M3 else 1           # 1.0 in the first dimension of token 0
    c.codes[first, :, 1] = c.codes[first, :, 1].reshape(seqs, kv, 64, blk).index_fill(3, torch.tensor([0], device="cuda"), 0).flatten(2)
    q = torch.zeros(seqs * new, heads, 64, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 18.375                                                       # 26.5 log2 units
    out, lse = torch.empty_like(q), torch.empty(seqs * new, heads, device="cuda")
    n, t = [new] * seqs, [length] * seqs
    moe.moe_attention(o, c.desc, c.batch(n, t), q, out, lse, scale=1.0)
    ok(o)
    want, wlse, bound = attention(c, n, t, q, 1.0, least=2.0 ** -30)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max().item()
    assert ((lse.double() - wlse).abs() <= 2.0 ** -19 * 32).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("heads,kv", [(32, 16), (2, 1)])
@pytest.mark.parametrize("new", [[1, 1, 1], [600, 33, 400]])
@pytest.mark.parametrize("gone", [-1, 0])
def test_blocks_before_the_window_may_be_gone(fmt, blk, heads, kv, new, gone):
    """Table entries before the window of the first new token, dropped or another's: no row needs them, and neither kernel
    reports or reads them (block 0 holds values that would show)."""
    lens, window = [1000, 333, 740], 50
    c = Cache(lens, kv, 64, blk, fmt, seed=6)
    c.table[c.table == 0] = max(set(range(1, c.codes.shape[0])) - set(c.table.flatten().tolist()))     # block 0 is another's
    c.fill(seed=12)
    c.scales[0] = 2.0 ** 100
    c.dtable = i32(c.table.tolist())
    for b, (n, t) in enumerate(zip(new, lens)):
        c.dtable[b, :max(0, t - n - window + 1) // blk] = gone
    check(c, new, lens, heads, window=window, sinks=torch.randn(heads, device="cuda"))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads,kv,new", [(32, 16, [600, 40]), (8, 2, [1, 3]), (8, 2, [1, 1])])
def test_nan_queries_and_sinks(fmt, heads, kv, new):
    """A NaN in one row's query, or in one head's sink, makes those rows' results and log-sum-exps NaN, and no others."""
    o = handle()
    lens, T = [1500, 700], sum(new)
    c = Cache(lens, kv, 64, 64, fmt, seed=6).fill(seed=13)
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
        assert ((lse.double() - wlse).abs() <= 2.0 ** -19 * 64 * 8 * 5)[~bad].all()
