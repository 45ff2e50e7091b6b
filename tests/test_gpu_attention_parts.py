"""Attention of few rows over many keys on the tensor cores: the keys of 256 rows are cut into parts, which are joined."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from kv4_testlib import Cache4  # noqa: E402
from ops_testlib import Cache, handle, i32, ok  # noqa: E402
from test_gpu_attention import check as check8  # noqa: E402
from test_gpu_attention4 import check as check4  # noqa: E402

FMTS = [moe.MOE_KV_E4M3, moe.MOE_KV_INT8, moe.MOE_KV_MXFP4]


def make(fmt, lens, kv, D, blk, seed=3):
    c = Cache4(lens, kv, D, blk, seed=seed) if fmt == moe.MOE_KV_MXFP4 else Cache(lens, kv, D, blk, fmt, seed=seed)
    return c.fill(seed=seed, poison=True)


def check(fmt, *args, **kw):
    """The joined parts' weights and sums round in fp32 some eight times more, 2^-20 of p |v|, which the bound's 2^-10.5 for f16
    probabilities (2^-11 and the rest) leaves room for."""
    return (check4 if fmt == moe.MOE_KV_MXFP4 else check8)(*args, **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv,new,lens,window", [
    (16, 2, [20], [3000], 0),                                         # one group of rows a head, in as many parts as there are
    (16, 2, [20], [3000], 700),                                       # the first tile is not the cache's first
    (64, 8, [27], [2500], 0),
    (8, 1, [70], [1025], 0),                                          # three groups, eight tiles and a key
    (32, 4, [16, 0, 40, 1], [1100, 300, 2049, 1537], 0),              # parts of some, none of others
    (32, 4, [1, 60, 13], [5000, 60, 1024], 1300),
    (12, 4, [200], [1700], 0),                                        # three heads a kv head: tokens across groups of rows
    (64, 8, [700], [3000], 0),                                        # more groups than SMs: the last 24 in parts
    (64, 8, [700, 90], [1500, 2600], 900),                            # the last 56 of 208 by the bound on their number
])
def test_parts(fmt, blk, D, heads, kv, new, lens, window):
    c = make(fmt, lens, kv, D, blk)
    for sinks in (None, torch.linspace(-4.0, 12.0, heads, device="cuda")):
        check(fmt, c, new, lens, heads, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_whose_first_parts_are_hidden(fmt):
    """Rows of one group whose windows lie in other parts than their neighbours', down to a single key."""
    c = make(fmt, [2600], 2, 64, 32)
    for window in (1, 33, 513):
        check(fmt, c, [1500], [2600], 4, window=window)
        check(fmt, c, [30], [2600], 16, window=window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_replayed_with_other_lengths(fmt, D):
    """The parts are of the lengths on the device: one captured call with many parts, some and none; the same bits each time."""
    o = handle()
    c = make(fmt, [4000, 1500], 2, D, 64)
    q = torch.randn(40, 16, D, device="cuda").bfloat16()
    cu, lens = i32([0, 24, 40]), i32([4000, 1500])
    b = moe.moe_kv_batch_of(cu, lens, c.dtable, 40)
    out, lse = torch.empty_like(q), torch.empty(40, 16, device="cuda")
    moe.moe_attention(o, c.desc, b, q, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_attention(o, c.desc, b, q, out, lse)
    for now in ([4000, 1500], [700, 40], [1024, 1023], [3999, 16], [24, 1500]):
        lens.copy_(torch.tensor(now))
        g.replay()
        want, wlse = check(fmt, c, [24, 16], now, 16, q=q)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    ok(o)


def test_between_single_tokens():
    """Calls of both kernels and of adapters in a row share the handle's workspace: nothing of one stays for the next."""
    o = handle()
    c = make(moe.MOE_KV_E4M3, [5000], 2, 64, 64)
    w = moe.moe_lora_of(torch.randn(2, 16, 512, device="cuda").bfloat16(), torch.randn(2, 256, 16, device="cuda").bfloat16())
    x, y, at = torch.randn(33, 512, device="cuda").bfloat16(), torch.zeros(33, 256, device="cuda"), i32([0, 1, -1] * 11)
    first = None
    for _ in range(3):
        got = [*check(moe.MOE_KV_E4M3, c, [40], [5000], 16), *check(moe.MOE_KV_E4M3, c, [1], [5000], 16)]
        y.zero_()
        moe.moe_lora(o, w, at, x, y)
        got.append(y.clone())
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_without_keys_and_nan(fmt):
    """No block of a sequence exists: zeros, the sink's lse, the status.  A NaN in one query stays in its row."""
    o = handle()
    c = make(fmt, [3000, 1400], 2, 64, 64)
    q = torch.randn(40, 16, 64, device="cuda").bfloat16()
    sinks = torch.linspace(-1.0, 2.0, 16, device="cuda")
    clean, clse = check(fmt, c, [20, 20], [3000, 1400], 16, sinks=sinks, q=q)
    bad = q.clone()
    bad[5, 3, 7] = math.nan
    out, lse = torch.empty_like(q), torch.empty(40, 16, device="cuda")
    b = c.batch([20, 20], [3000, 1400])
    moe.moe_attention(o, c.desc, b, bad, out, lse, sinks)
    ok(o)
    assert out[5, 3].isnan().all() and lse[5, 3].isnan()
    out[5, 3], lse[5, 3] = clean[5, 3], clse[5, 3]
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    c.dtable[1] = -1
    moe.moe_attention(o, c.desc, b, q, out, lse, sinks)
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    assert (out[20:] == 0).all() and torch.allclose(lse[20:], sinks.expand(20, 16), rtol=0, atol=1e-6)
    assert torch.equal(out[:20], clean[:20]) and torch.equal(lse[:20], clse[:20])
