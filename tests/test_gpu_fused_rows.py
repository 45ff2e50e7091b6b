"""Projections and adapters whose input and output are columns of one buffer: the same bits as apart, and nothing else is written."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import handle, i32, ok  # noqa: E402


@pytest.mark.parametrize("M", [1, 7, 33, 64])
@pytest.mark.parametrize("first", [True, False])
def test_input_and_output_in_one_buffer(M, first):
    o, cols, rows = handle(), 256, 199
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g, device="cuda")
    w = moe.moe_linear_of(codes, torch.randint(118, 122, (rows, cols // 32), dtype=torch.uint8, generator=g, device="cuda"), None,
                          moe.MOE_FMT_MXFP4, 32)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    lw = moe.moe_lora_of(r(3, 16, cols), r(3, rows, 16))
    at = (torch.arange(M, device="cuda") % 4 - 1).int()
    both = r(M, cols + 208)
    x, out = (both[:, :cols], both[:, cols + 5:cols + 5 + rows]) if first else (both[:, 208:], both[:, 3:3 + rows])
    before, x0, out0 = both.clone(), x.clone(), torch.empty(M, rows, dtype=torch.bfloat16, device="cuda")
    for a, b in ((x0, out0), (x, out)):
        moe.moe_linear(o, w, a, b)
        moe.moe_lora(o, lw, at, a, b)
    ok(o)
    assert torch.equal(out, out0)
    out.copy_(before[:, cols + 5:cols + 5 + rows] if first else before[:, 3:3 + rows])
    assert torch.equal(both, before)
