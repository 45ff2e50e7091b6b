"""Attention whose keys are cut into parts, with calls of which the host's rule says so (tests/plan_testlib.py): captured and replayed
with other lengths, with parts of which nothing is visible, and with NaN."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from kv4_testlib import Cache4  # noqa: E402
from ops_testlib import Cache, half_ulp_bf16, handle, i32, ok  # noqa: E402
from plan_testlib import in_parts  # noqa: E402
from test_gpu_attention import check as check8  # noqa: E402
from test_gpu_attention4 import check as check4  # noqa: E402

FMTS = [moe.MOE_KV_E4M3, moe.MOE_KV_INT8, moe.MOE_KV_MXFP4]


def make(fmt, lens, kv, D, blk, seed=3):
    c = Cache4(lens, kv, D, blk, seed=seed) if fmt == moe.MOE_KV_MXFP4 else Cache(lens, kv, D, blk, fmt, seed=seed)
    return c.fill(seed=seed, poison=True)


def check(fmt, *args, **kw):
    return (check4 if fmt == moe.MOE_KV_MXFP4 else check8)(*args, **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk,D", [(32, 64), (64, 128), (128, 64), (128, 128)])
def test_replayed_with_other_lengths(fmt, blk, D):
    """The parts are of the lengths on the device: one captured call with many parts, some and none; the same bits each time."""
    o = handle()
    c = make(fmt, [4000, 1500], 8, D, blk)
    assert in_parts(c, [24, 16], 64)
    q = torch.randn(40, 64, D, device="cuda").bfloat16()
    cu, lens = i32([0, 24, 40]), i32([4000, 1500])
    b = moe.moe_kv_batch_of(cu, lens, c.dtable, 40)
    out, lse = torch.empty_like(q), torch.empty(40, 64, device="cuda")
    moe.moe_attention(o, c.desc, b, q, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_attention(o, c.desc, b, q, out, lse)
    for now in ([4000, 1500], [700, 40], [1024, 1023], [3999, 16], [24, 1500]):
        lens.copy_(torch.tensor(now))
        g.replay()
        want, wlse = check(fmt, c, [24, 16], now, 64, q=q)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    ok(o)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 128])
@pytest.mark.parametrize("gone", [(0, 1024), (1536, 3000), (512, 2560)])
def test_parts_without_keys(fmt, blk, gone):
    """Blocks that are missing, for whole parts: those have no sums and no weight, the status says so, and the rest is the softmax over
    the other keys.  The bound is the one of ops_testlib.attention: f16 probabilities (2^-11 and as much again, for scores of this
    size), one rounding to bf16, and 2^-24 of a value a key below f16's normal numbers."""
    o = handle()
    c = make(fmt, [4000], 8, 64, blk)
    assert in_parts(c, [20], 64)
    q = torch.randn(20, 64, 64, device="cuda").bfloat16()
    c.dtable[0, gone[0] // blk:gone[1] // blk] = -1
    out, lse = torch.empty_like(q), torch.empty(20, 64, device="cuda")
    moe.moe_attention(o, c.desc, c.batch([20], [4000]), q, out, lse)
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    k, v = (x.repeat_interleave(8, 1).permute(1, 0, 2) for x in c.values(0, 4000))
    s = q.double().permute(1, 0, 2) @ k.transpose(1, 2) / 8
    j = torch.arange(4000, device="cuda")
    see = (j <= torch.arange(3980, 4000, device="cuda")[:, None]) & ~((j >= gone[0] // blk * blk) & (j < gone[1] // blk * blk))
    s = torch.where(see, s, -math.inf)
    p = torch.softmax(s, -1)
    want = (p @ v).permute(1, 0, 2)
    total = (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
    bound = (half_ulp_bf16(want) * 1.01 + ((2.0 ** -10 * p + 2.0 ** -24 / total * see) @ v.abs()).permute(1, 0, 2))
    assert ((out.double() - want).abs() <= bound).all()
    wlse, s_mag = torch.logsumexp(s, -1).permute(1, 0), float(q.abs().max()) * 24 * 64 / 8         # as check's
    assert ((lse.double() - wlse).abs() <= 2.0 ** -19 * (s_mag + wlse.abs())).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_without_keys_and_nan(fmt):
    """No block of a sequence exists: zeros, the sink's lse, the status.  A NaN in one query stays in its row."""
    o = handle()
    c = make(fmt, [3000, 1400], 8, 64, 64)
    assert in_parts(c, [20, 20], 64)
    q = torch.randn(40, 64, 64, device="cuda").bfloat16()
    sinks = torch.linspace(-1.0, 2.0, 64, device="cuda")
    clean, clse = check(fmt, c, [20, 20], [3000, 1400], 64, sinks=sinks, q=q)
    bad = q.clone()
    bad[5, 3, 7] = math.nan
    out, lse = torch.empty_like(q), torch.empty(40, 64, device="cuda")
    b = c.batch([20, 20], [3000, 1400])
    moe.moe_attention(o, c.desc, b, bad, out, lse, sinks)
    ok(o)
    assert out[5, 3].isnan().all() and lse[5, 3].isnan()
    out[5, 3], lse[5, 3] = clean[5, 3], clse[5, 3]
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    c.dtable[1] = -1
    moe.moe_attention(o, c.desc, b, q, out, lse, sinks)
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    assert (out[20:] == 0).all() and torch.allclose(lse[20:], sinks.expand(20, 64), rtol=0, atol=1e-6)
    assert torch.equal(out[:20], clean[:20]) and torch.equal(lse[:20], clse[:20])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_within_a_window(fmt, D):
    """Parts that begin where the window does, tokens across groups of rows."""
    for heads, new, lens, window in ((64, [30], [6000], 1500), (24, [100], [5000], 2500), (64, [40, 3], [2600, 5000], 1800)):
        c = make(fmt, lens, 8, D, 64)
        assert in_parts(c, new, heads, window)
        check(fmt, c, new, lens, heads, window=window, sinks=torch.linspace(-4.0, 12.0, heads, device="cuda"))
