"""Projections with 4-bit weights against the dequantised product in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import half_ulp_bf16, handle, ok  # noqa: E402

E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def make(rows, cols, fmt, group, bias, seed, lo=117, hi=125):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g, device="cuda")
    if fmt == moe.MOE_FMT_MXFP4:
        scales = torch.randint(lo, hi, (rows, cols // 32), dtype=torch.uint8, generator=g, device="cuda")
    else:
        scales = (torch.randn(rows, cols // group, generator=g, device="cuda") * 0.02).half()
    b = torch.randn(rows, generator=g, device="cuda").bfloat16() if bias else None
    return codes, scales, b, moe.moe_linear_of(codes, scales, b, fmt, group)


def dense(codes, scales, fmt, group):
    v = torch.tensor(E2M1 if fmt == moe.MOE_FMT_MXFP4 else list(range(-8, 8)), dtype=torch.float64, device="cuda")
    w = torch.stack((v[(codes & 15).long()], v[(codes >> 4).long()]), -1).reshape(codes.shape[0], -1, group)
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), scales.double() - 127) if fmt == moe.MOE_FMT_MXFP4 else scales.double()
    return (w * s[..., None]).reshape(codes.shape[0], -1)


def check(rows, cols, M, fmt, group, bias=False, out=torch.float32, seed=0, x=None, **kw):
    o = handle()
    codes, scales, b, w = make(rows, cols, fmt, group, bias, seed, **kw)
    if x is None:
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        x = torch.randn(M, cols, generator=g, device="cuda").bfloat16()
    y = torch.full((M, rows + 3), 7.0, dtype=out, device="cuda")
    moe.moe_linear(o, w, x, y[:, :rows])
    ok(o)
    W = dense(codes, scales, fmt, group)
    want = x.double() @ W.t() + (b.double() if bias else 0.0)
    mag = x.double().abs() @ W.abs().t() + (b.double().abs() if bias else 0.0)
    # cols / 16 additions of partial sums in fp32, each off by at most 2^-22 of the magnitudes' sum; the smallest
    # elements of x may lose what is below 2^-39 of its largest
    tol = mag * (cols / 16 + 8) * 2.0 ** -22 + x.double().abs().amax(1, keepdim=True) * 2.0 ** -39 * W.abs().sum(1) + 1e-45
    if out is torch.bfloat16:
        tol = tol + half_ulp_bf16(want.abs() + tol)
    err = (y[:, :rows].double() - want).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    assert (y[:, rows:] == 7.0).all()
    return y


F4, I4 = moe.MOE_FMT_MXFP4, moe.MOE_FMT_INT4


@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 32), (I4, 64), (I4, 128), (I4, 256)])
@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("rows,cols", [(64, 256), (1, 256), (17, 512), (129, 768)])
def test_shapes(fmt, group, M, rows, cols):
    check(rows, cols, M, fmt, group, bias=M % 2 == 1, out=torch.bfloat16 if M % 3 == 0 else torch.float32, seed=M)


@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 32)])
@pytest.mark.parametrize("cols", [32, 64, 96, 160, 2880, 2912])
@pytest.mark.parametrize("M", [1, 11])
def test_columns_that_are_odd_multiples_of_32(fmt, group, cols, M):
    check(83, cols, M, fmt, group, bias=True, seed=cols)


@pytest.mark.parametrize("fmt,group,rows,cols,M", [(F4, 32, 5120, 2880, 1), (F4, 32, 2880, 4096, 4), (I4, 64, 50257, 2048, 1),
                                                   (I4, 128, 4097, 8192, 3), (F4, 32, 1000, 32768, 2)])
def test_model_sizes(fmt, group, rows, cols, M):
    check(rows, cols, M, fmt, group, bias=fmt == F4, seed=rows)
    check(rows, cols, M, fmt, group, out=torch.bfloat16, seed=rows)


def test_scale_extremes():
    """E8M0 bytes from 0 on, fp16 scales that are subnormal, of either sign; the last bytes with x small enough."""
    check(64, 256, 2, F4, 32, lo=0, hi=40)
    check(64, 256, 2, F4, 32, lo=0, hi=3, x=(torch.randn(2, 256, device="cuda") * 2.0 ** 20).bfloat16())
    check(64, 256, 2, F4, 32, lo=250, hi=255, x=(torch.randn(2, 256, device="cuda") * 2.0 ** -40).bfloat16())
    o = handle()
    codes, scales, _, _ = make(64, 256, I4, 64, False, 3)
    scales = (scales.float() * 2.0 ** -16).half()
    w = moe.moe_linear_of(codes, scales, None, I4, 64)
    x = torch.randn(3, 256, device="cuda").bfloat16()
    y = torch.empty(3, 64, device="cuda")
    moe.moe_linear(o, w, x, y)
    W = dense(codes, scales, I4, 64)
    assert ((y.double() - x.double() @ W.t()).abs() <= x.double().abs() @ W.abs().t() * 24 * 2.0 ** -22).all()


def test_nan_scale_makes_its_row_nan():
    o = handle()
    codes, scales, _, w = make(40, 256, F4, 32, False, 4)
    scales[7, 3] = 255
    x = torch.randn(3, 256, device="cuda").bfloat16()
    y = torch.empty(3, 40, device="cuda")
    moe.moe_linear(o, w, x, y)
    assert torch.isnan(y[:, 7]).all() and torch.isfinite(y[:, :7]).all() and torch.isfinite(y[:, 8:]).all()


@pytest.mark.parametrize("size", [0.0, 2.0 ** -120, 2.0 ** -30, 2.0 ** 100])
def test_x_of_any_size(size):
    x = (torch.randn(3, 512, device="cuda") * size).bfloat16()
    check(70, 512, 3, I4, 64, x=x)


def test_x_with_a_wide_range_and_tokens_apart():
    """Elements 2^30 apart within a token; a token whose values are infinite or NaN leaves the others as they are."""
    x = torch.randn(4, 512, device="cuda") * torch.pow(2.0, torch.randint(-30, 1, (4, 512), device="cuda").float())
    check(70, 512, 4, F4, 32, x=x.bfloat16())
    o = handle()
    codes, scales, _, w = make(70, 512, I4, 64, False, 5)
    x = torch.randn(4, 512, device="cuda").bfloat16()
    y, z = torch.empty(4, 70, device="cuda"), torch.empty(4, 70, device="cuda")
    moe.moe_linear(o, w, x, y)
    x[1, 100], x[2, 7] = float("inf"), float("nan")
    moe.moe_linear(o, w, x, z)
    ok(o)
    assert torch.equal(y[0], z[0]) and torch.equal(y[3], z[3])
    assert not torch.isfinite(z[2]).any()
    assert not torch.isfinite(z[1]).any()


def test_strided_rows_and_repeats():
    o = handle()
    codes, scales, b, w = make(300, 2880, F4, 32, True, 6)
    big = torch.randn(5, 2880 + 64, device="cuda").bfloat16()
    x = big[:, 64:]
    y, z = torch.empty(5, 300, device="cuda"), torch.empty(5, 300, device="cuda")
    moe.moe_linear(o, w, x, y)
    moe.moe_linear(o, w, x.contiguous(), z)
    ok(o)
    assert torch.equal(y, z)


# Many tokens of many columns: four CTAs share the rows and split the columns in pieces of 256, the last of which
# may be short or none.
@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 32), (I4, 64), (I4, 128), (I4, 256)])
@pytest.mark.parametrize("rows,cols,M", [(40, 1280, 16), (1, 2048, 13), (700, 2304, 12), (2501, 4096, 16), (9, 8192, 16),
                                         (33, 4096, 40), (20000, 4096, 16)])
def test_columns_split_over_ctas(fmt, group, rows, cols, M):
    check(rows, cols, M, fmt, group, bias=M % 2 == 0, out=torch.bfloat16 if rows % 2 else torch.float32, seed=rows + M)


@pytest.mark.parametrize("cols", [1056, 2080, 4128, 8160])
def test_columns_split_over_ctas_with_odd_ends(cols):
    check(77, cols, 16, F4, 32, bias=True, seed=cols)
    check(77, cols, 11, I4, 32, seed=cols + 1)


@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 64)])
def test_parts_of_the_columns_of_other_sizes(fmt, group):
    """Parts of a token that are zero, tiny or huge beside the others."""
    x = torch.randn(16, 4096, device="cuda")
    x[:, :1024] = 0
    x[0:4, 1024:2048] *= 2.0 ** -60
    x[2:6, 2048:] *= 2.0 ** 40
    x[7] = 0
    x[8, :3000] = 0
    check(70, 4096, 16, fmt, group, x=x.bfloat16())


# Wide matrices: x and the cluster's join buffer leave the rings little of the shared memory, so that the split that would
# be fastest may not fit.
@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 32), (I4, 64)])
@pytest.mark.parametrize("rows,cols", [(5120, 13824), (7168, 18432), (8192, 22016), (2560, 11296)])
@pytest.mark.parametrize("M", [9, 13, 16, 40])
def test_wide_matrices(fmt, group, rows, cols, M):
    if cols % group:
        cols += group - cols % group
    check(rows, cols, M, fmt, group, bias=M % 2 == 0, out=torch.bfloat16 if M == 16 else torch.float32, seed=cols + M)


@pytest.mark.parametrize("fmt,group,rows,cols,M", [(I4, 128, 16384, 17536, 16), (I4, 256, 16384, 17664, 15), (F4, 32, 16384, 16384, 16),
                                                   (I4, 64, 40000, 14336, 64), (F4, 32, 300, 32768, 16), (I4, 256, 300, 32768, 16)])
def test_widest_matrices(fmt, group, rows, cols, M):
    check(rows, cols, M, fmt, group, seed=cols + M)


@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 64)])
def test_clusters_with_a_cta_without_columns_repeat(fmt, group):
    """1,280 columns are five pieces: two, two, one and none for a cluster's CTAs, the last of which is ready at once."""
    o = handle()
    _, _, _, w = make(40, 1280, fmt, group, True, 8)
    x = torch.randn(16, 1280, device="cuda").bfloat16()
    y = torch.empty(200, 16, 40, device="cuda")
    for i in range(200):
        moe.moe_linear(o, w, x, y[i])
    ok(o)
    assert torch.equal(y, y[:1].expand_as(y))
    check(40, 1280, 16, fmt, group, bias=True, seed=8)


@pytest.mark.parametrize("fmt,group", [(F4, 32), (I4, 32), (I4, 256)])
@pytest.mark.parametrize("M,cols", [(5, 512), (13, 768), (16, 4096), (11, 1280)])
def test_tokens_of_very_different_size(fmt, group, M, cols):
    """Finite tokens near both ends of bf16's range beside ordinary ones, as rows of memory that nothing has set may be:
    each token's result keeps its own bound (the check's) whatever the others are; with clusters and without."""
    g = torch.Generator(device="cuda").manual_seed(M + cols)
    x = torch.randn(M, cols, generator=g, device="cuda") * 8
    x[1] *= 2.0 ** -100
    x[3] *= 2.0 ** -123
    x[2, 17] = x[M - 1, cols - 3] = 2.0 ** 125
    x = x.bfloat16()
    y = check(70, cols, M, fmt, group, x=x, seed=3)
    ordinary = [m for m in range(M) if m not in (1, 2, 3, M - 1)]
    z = check(70, cols, M, fmt, group, x=torch.where(torch.isin(torch.arange(M, device="cuda"), torch.tensor(ordinary, device="cuda"))[:, None], x, 0.0),
              seed=3)
    assert torch.equal(y[ordinary], z[ordinary])
