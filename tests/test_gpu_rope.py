"""Rotary positions against their formula in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import handle, i32, ok  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
HALF, INTER = moe.MOE_ROPE_HALF, moe.MOE_ROPE_INTERLEAVED


def pairs(x, rot, layout):
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == HALF else (x[..., 0:rot:2], x[..., 1:rot:2])


def reference(x, pos, rot, layout, mscale=1.0, base=10000.0):
    """(result, bound) in float64.  The angle is off by 2^-24 of at most pi, sincospif by two units of 2^-24, a cosine times
    mscale by one rounding, the products and their sum by three: together below 2^-20.5 (|u| + |v|) mscale."""
    x = x.double()
    f = torch.pow(torch.tensor(base, dtype=torch.float64, device="cuda"), -2.0 * torch.arange(rot // 2, device="cuda").double() / rot)
    t = (pos.double()[:, None] * f)[:, None]
    u, v = pairs(x, rot, layout)
    a, b = mscale * (u * t.cos() - v * t.sin()), mscale * (v * t.cos() + u * t.sin())
    out, mag = x.clone(), torch.zeros_like(x)
    for d, s in zip(pairs(out, rot, layout), (a, b)):
        d.copy_(s)
    for d in pairs(mag, rot, layout):
        d.copy_(u.abs() + v.abs())
    return out, mag * abs(mscale) * 2.0 ** -20.5


def rounding(x, dtype):
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -126)))
    return torch.pow(2.0, e - (8 if dtype is BF else 24)) * 1.01


def check(got, x, pos, rot, layout, mscale=1.0):
    want, bound = reference(x, pos, rot, layout, mscale)
    err = (got.double() - want).abs()
    assert (err <= bound + rounding(want, got.dtype)).all(), (err - bound - rounding(want, got.dtype)).max().item()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", [HALF, INTER])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 96), (128, 32), (64, 2), (64, 54), (96, 72), (256, 256), (8, 8), (512, 510), (512, 512)])
@pytest.mark.parametrize("T,hq,hk", [(1, 64, 8), (5, 3, 1), (700, 5, 2), (333, 2, 0)])
def test_formula(dtype, layout, D, rot, T, hq, hk):
    o, g = handle(), torch.Generator(device="cuda").manual_seed(D + rot + T)
    x = torch.randn(T, hq + hk + 1, D, generator=g, device="cuda").to(dtype)      # rows of a fused projection
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    pos = torch.randint(0, 200000, (T,), generator=g, device="cuda", dtype=torch.int32)
    rope = moe.moe_rope_of(rot, 10000.0, layout, mscale=1.25)
    qo, ko = torch.empty(T, hq, D, dtype=dtype, device="cuda"), torch.empty(T, hk, D, dtype=dtype, device="cuda") if hk else None
    moe.moe_rope(o, rope, pos, q, k, qo, ko)
    check(qo, q, pos, rot, layout, 1.25)
    if hk:
        check(ko, k, pos, rot, layout, 1.25)
    # in place in the fused rows; the rest of them stays
    y = x.clone()
    moe.moe_rope(o, rope, pos, y[:, :hq], y[:, hq:hq + hk] if hk else None)
    assert torch.equal(y[:, :hq], qo) and (not hk or torch.equal(y[:, hq:hq + hk], ko)) and torch.equal(y[:, hq + hk:], x[:, hq + hk:])
    ok(o)


def test_far_positions():
    """Positions up to the largest int32: the angle's fraction of a turn stays exact, where fp32 angles would be off by radians."""
    o = handle()
    pos = i32([0, 1, 2, 1 << 24, (1 << 24) + 1, 10 ** 9, 2 ** 31 - 1])
    for layout in (HALF, INTER):
        x = torch.randn(7, 4, 64, device="cuda")
        y = torch.empty_like(x)
        moe.moe_rope(o, moe.moe_rope_of(64, 10000.0, layout), pos, x, None, y)
        want, bound = reference(x, pos, 64, layout)
        # the reference's own angle: 2^31 times a double that is off by 2^-54, and its argument reduction's; as much in the table
        slack = pos.double()[:, None, None] * 2.0 ** -50 * x.double().abs().amax()
        assert ((y.double() - want).abs() <= bound + rounding(want, F32) + slack).all()


def test_position_zero_is_the_identity_and_rotations_add_up():
    o = handle()
    x = torch.randn(50, 2, 128, device="cuda")
    rope = moe.moe_rope_of(128, 500000.0)
    y = torch.empty_like(x)
    moe.moe_rope(o, rope, torch.zeros(50, dtype=torch.int32, device="cuda"), x, None, y)
    assert torch.equal(x, y)
    a, b = torch.arange(50, dtype=torch.int32, device="cuda") * 7, torch.arange(50, dtype=torch.int32, device="cuda") * 1000 + 3
    moe.moe_rope(o, rope, a, y)
    moe.moe_rope(o, rope, b, y)
    z = torch.empty_like(x)
    moe.moe_rope(o, rope, a + b, x, None, z)
    u, v = pairs(x.double().abs(), 128, HALF)
    mag = torch.cat((u + v, u + v), -1)
    assert ((y - z).double().abs() <= mag * 4 * 2.0 ** -20.5).all()               # three rotations, each within its bound, and one's growth


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rot", [64, 54])
def test_negative_positions_leave_rows_alone(dtype, rot):
    o = handle()
    x = torch.randn(9, 6, 64, device="cuda").to(dtype)
    pos = i32([3, -1, 5, 0, -7, -2 ** 31, 8, 9, -1])
    for layout in (HALF, INTER):
        out = torch.full_like(x, 7.0)
        moe.moe_rope(o, moe.moe_rope_of(rot, 10000.0, layout), pos, x, None, out)
        live = pos >= 0
        check(out[live], x[live], pos[live], rot, layout)
        assert (out[~live] == 7.0).all()


def test_odd_values_touch_only_their_pair():
    o = handle()
    x = torch.randn(3, 2, 64, device="cuda").bfloat16()
    x[1, 1, 5], x[2, 0, 40] = float("nan"), float("inf")
    y = torch.empty_like(x)
    pos = i32([10, 11, 12])
    moe.moe_rope(o, moe.moe_rope_of(64, 10000.0), pos, x, None, y)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[1, 1, 5] = bad[1, 1, 37] = bad[2, 0, 40] = bad[2, 0, 8] = True
    assert not torch.isfinite(y[bad]).any()
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    want, bound = reference(clean, pos, 64, HALF)
    assert ((y.double() - want).abs() <= bound + rounding(want, BF))[~bad].all()


@pytest.mark.parametrize("kind,par", [(moe.MOE_ROPE_LINEAR, dict(factor=4.0)), (moe.MOE_ROPE_PARTS, dict(factor=32.0, length=4096, low=1.0, high=32.0)),
                                      (moe.MOE_ROPE_WAVELENGTH, dict(factor=8.0, length=8192, low=1.0, high=4.0))])
def test_scaled_tables(kind, par):
    """The kernel turns by what the table says: angles from the table's own 64-bit fractions."""
    o = handle()
    table = moe.moe_rope_turns(64, 150000.0, kind, **par)
    x, pos = torch.randn(100, 3, 64, device="cuda"), torch.arange(100, dtype=torch.int32, device="cuda") * 1297
    y = torch.empty_like(x)
    moe.moe_rope(o, moe.moe_rope_of(64, 150000.0, scaling=kind, **par), pos, x, None, y)
    t = torch.tensor([[(p * int(f) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for f in table] for p in pos.tolist()], dtype=torch.float64, device="cuda")[:, None]
    u, v = pairs(x.double(), 64, HALF)
    want = torch.cat((u * t.cos() - v * t.sin(), v * t.cos() + u * t.sin()), -1)
    mag = torch.cat((u.abs() + v.abs(),) * 2, -1)
    assert ((y.double() - want).abs() <= mag * 2.0 ** -20.5 + rounding(want, F32)).all()


def test_in_a_graph_and_on_another_stream():
    o = handle()
    x = torch.randn(20, 10, 64, device="cuda").bfloat16()
    pos, rope = torch.arange(20, dtype=torch.int32, device="cuda"), moe.moe_rope_of(64, 10000.0)
    want, got = torch.empty_like(x), torch.empty_like(x)
    moe.moe_rope(o, rope, pos, x, None, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    moe.moe_rope(o, rope, pos, x, None, got, stream=s)
    s.synchronize()
    assert torch.equal(want, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_rope(o, rope, pos, x, None, got)
    pos += 5
    g.replay()
    moe.moe_rope(o, rope, pos, x, None, want)
    assert torch.equal(want, got)


def test_large_offsets():
    """Rows whose offsets pass 2^31 elements."""
    o = handle()
    T, stride = 5, 1 << 29
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((T, 2, 64), (stride, 64, 1))
    x = torch.randn(T, 2, 64, device="cuda").bfloat16()
    q.copy_(x)
    pos, out = torch.arange(T, dtype=torch.int32, device="cuda") + 3, torch.empty_like(x)
    moe.moe_rope(o, moe.moe_rope_of(64, 10000.0), pos, q, None, out)
    check(out, x, pos, 64, HALF)
