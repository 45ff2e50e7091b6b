"""Low-rank adapters beside a projection against their formula in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import handle, i32, ok  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def make(n, rank, rows, cols, seed=0, scaled=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = (torch.randn(n, rank, cols, generator=g, device="cuda") * cols ** -0.5).to(BF)
    b = torch.randn(n, rows, rank, generator=g, device="cuda").to(BF)
    s = torch.randn(n, generator=g, device="cuda") if scaled else None
    return a, b, s


def reference(a, b, s, index, x, y, dtype):
    """(out, bound) in float64.  A chain of fp32 sums: at most cols / 16 + 32 of them for h (columns, warps, parts), 3 rank / 16 + 8
    for the second product, each off by no more than 2^-23 of the sum of magnitudes; h's three bf16 terms leave 2^-25 of it."""
    rank, cols = a.shape[1:]
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64, device="cuda") if y is None else y.double().clone()
    mag = out.abs() * 2.0 ** -23
    for m, i in enumerate(index):
        if 0 <= i < a.shape[0]:
            A, B, f = a[i].double(), b[i].double(), 1.0 if s is None else float(s[i])
            h, hm = A @ x[m].double(), A.abs() @ x[m].double().abs()
            out[m] += f * (B @ h)
            mag[m] += abs(f) * (B.abs() @ (hm * (cols / 16 + 32) + h.abs() * (3 * rank / 16 + 12))) * 2.0 ** -23
    e = torch.floor(torch.log2(out.abs().clamp_min(2.0 ** -126)))
    return out, mag + torch.pow(2.0, e - (8 if dtype is BF else 24)) * 1.01


def check(w, index, x, y, out):
    a, b, s = w.tensors
    want, bound = reference(a, b, s, index, x, y, out.dtype)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max().item()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 8), (65, 72), (256, 1000), (4097, 2880), (300, 8192)])
@pytest.mark.parametrize("M", [1, 3, 64])
def test_formula(dtype, rank, rows, cols, M):
    """Each token with an adapter of its own, one for all, some without."""
    o, n = handle(), 5
    g = torch.Generator(device="cuda").manual_seed(M + rank)
    w = moe.moe_lora_of(*make(n, rank, rows, cols, seed=rank + rows))
    x = torch.randn(M, cols, generator=g, device="cuda").to(BF)
    y = torch.randn(M, rows, generator=g, device="cuda").to(dtype)
    for index in ([m % n for m in range(M)], [3] * M, [(m * 7 % 6) - 1 for m in range(M)], [-1] * M):
        out = torch.full_like(y, 9.0)
        moe.moe_lora(o, w, i32(index), x, y, out)
        ok(o)
        check(w, index, x, y, out)
        same = y.clone()
        moe.moe_lora(o, w, i32(index), x, same)                                   # in place
        assert torch.equal(same, out)


def test_without_scale_or_base():
    o = handle()
    w = moe.moe_lora_of(*make(3, 16, 130, 256, scaled=False))
    x, index = torch.randn(5, 256, device="cuda").to(BF), [2, -1, 0, 0, 1]
    for dtype in (BF, F32):
        out = torch.full((5, 130), 9.0, dtype=dtype, device="cuda")
        moe.moe_lora(o, w, i32(index), x, None, out)
        check(w, index, x, None, out)
        assert (out[1] == 0).all()


def test_strides_and_rows_behind():
    """Parts of wider rows in and out; what lies beside them stays."""
    o = handle()
    w = moe.moe_lora_of(*make(4, 32, 200, 512))
    xw, yw = torch.randn(9, 1024, device="cuda").to(BF), torch.randn(9, 333, device="cuda")
    x, y, index = xw[:, 256:768], yw[:, 100:300], [0, 1, 2, 3, -1, 3, 2, 1, 0]
    before = yw.clone()
    want, bound = reference(*w.tensors, index, x, y, F32)
    moe.moe_lora(o, w, i32(index), x, y)
    assert ((y.double() - want).abs() <= bound).all()
    assert torch.equal(yw[:, :100], before[:, :100]) and torch.equal(yw[:, 300:], before[:, 300:])


@pytest.mark.parametrize("M,n", [(64, 1), (64, 7), (63, 63), (17, 2), (9, 1)])
def test_groups_of_tokens(M, n):
    """Adapters shared by more tokens than a group holds, mixed among one another; a token's result does not depend on the
    others' values."""
    o = handle()
    w = moe.moe_lora_of(*make(n, 16, 96, 640))
    index = [(m * m + 3 * m) % n for m in range(M)]
    x, y = torch.randn(M, 640, device="cuda").to(BF), torch.randn(M, 96, device="cuda")
    out, again = torch.empty_like(y), torch.empty_like(y)
    moe.moe_lora(o, w, i32(index), x, y, out)
    check(w, index, x, y, out)
    z = x * 1000
    z[M // 2] = x[M // 2]
    moe.moe_lora(o, w, i32(index), z, y, again)
    assert torch.equal(out[M // 2], again[M // 2])


def test_odd_values_stay_in_their_token():
    o = handle()
    w = moe.moe_lora_of(*make(2, 24, 100, 256))
    x, y, index = torch.randn(6, 256, device="cuda").to(BF), torch.randn(6, 100, device="cuda"), [0, 0, 0, 1, 1, -1]
    x[1, 7], x[4, 9], x[5, 0] = float("nan"), float("inf"), float("nan")
    out = torch.empty_like(y)
    moe.moe_lora(o, w, i32(index), x, y, out)
    assert not torch.isfinite(out[[1, 4]]).any()
    assert torch.equal(out[5], y[5])
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    want, bound = reference(*w.tensors, index, clean, y, F32)
    assert ((out.double() - want).abs() <= bound)[[0, 2, 3, 5]].all()


def test_adapters_out_of_range():
    """Counted as none, and the status says so."""
    o = handle()
    w = moe.moe_lora_of(*make(2, 8, 40, 64))
    x, y, out = torch.randn(4, 64, device="cuda").to(BF), torch.randn(4, 40, device="cuda"), torch.empty(4, 40, device="cuda")
    index = [1, 2, 2 ** 31 - 1, -2 ** 31]
    moe.moe_lora(o, w, i32(index), x, y, out)
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    check(w, index, x, y, out)
    assert torch.equal(out[1:], y[1:])


def test_offsets_past_32_bits():
    """The last of many large adapters."""
    o = handle()
    n, rank, rows, cols = 700, 128, 25000, 25000
    a, b = (torch.zeros(n, *s, dtype=BF, device="cuda") for s in ((rank, cols), (rows, rank)))
    p, q, _ = make(1, rank, rows, cols)
    a[-1], b[-1] = p[0], q[0]
    x, y = torch.randn(2, cols, device="cuda").to(BF), torch.randn(2, rows, device="cuda")
    w, out = moe.moe_lora_of(a, b), torch.empty_like(y)
    moe.moe_lora(o, w, i32([n - 1, 0]), x, y, out)
    want, bound = reference(p, q, None, [0, -1], x, y, F32)
    assert ((out.double() - want).abs() <= bound).all()


def test_repeats_a_graph_and_another_stream():
    """The same bits every time; captured, replayed with another assignment; behind a projection, in place."""
    o = handle()
    w = moe.moe_lora_of(*make(6, 64, 512, 1024))
    index, x, y = i32([0, 5, 3, 3, -1, 2, 1]), torch.randn(7, 1024, device="cuda").to(BF), torch.randn(7, 512, device="cuda")
    want, out = torch.empty_like(y), torch.empty_like(y)
    moe.moe_lora(o, w, index, x, y, want)
    for _ in range(3):
        moe.moe_lora(o, w, index, x, y, out)
        assert torch.equal(out, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_lora(o, w, index, x, y, out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_lora(o, w, index, x, y, out)
        moe.moe_lora(o, w, index, x, out)                                          # once more on top
    index.copy_(i32([1, 1, 1, 1, 1, -1, 0]))
    graph.replay()
    moe.moe_lora(o, w, index, x, y, want)
    moe.moe_lora(o, w, index, x, want)
    assert torch.equal(out, want)
