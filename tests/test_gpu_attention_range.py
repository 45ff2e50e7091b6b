"""Attention over values near both ends of the cache's range: a weighted mean is finite where the values are, however many keys
it is of and however their parts are joined."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from kv4_testlib import Cache4  # noqa: E402
from ops_testlib import Cache, attention, handle, ok  # noqa: E402

FMTS = [moe.MOE_KV_E4M3, moe.MOE_KV_INT8, moe.MOE_KV_MXFP4]


def cache(fmt, lens, kv, D, blk, power):
    """Positive V's with scales around 2^power (E4M3's and INT8's codes reach 2^7 above, E2M1's 6), K's as ever."""
    if fmt == moe.MOE_KV_MXFP4:
        c = Cache4(lens, kv, D, blk).fill(seed=5)
        code, scale = c.unpacked(slice(None), 1)
        c.repack(slice(None), 1, code & 7, torch.where(scale == 0, 0, scale - 125 + 127 + power))
    else:
        c = Cache(lens, kv, D, blk, fmt).fill(seed=5)
        v = c.codes[:, :, 1]
        v.copy_(v & 127 if fmt == moe.MOE_KV_E4M3 else v.view(torch.int8).abs().view(torch.uint8))
        c.scales[:, :, 1] = (torch.rand(c.scales.shape[:2], device="cuda") if fmt == moe.MOE_KV_INT8 else
                             torch.randint(0, 2, c.scales.shape[:2], device="cuda").float()) * 2.0 ** (power - 1) + 2.0 ** (power - 1)
    return c


def check(c, new, lens, heads, qscale):
    """The bound that every format's tests use (`attention`: f16 probabilities and one rounding to bf16), without its smallest term,
    which is above the smallest values here.  A part's values are held at least at 2^-13 of themselves: one of 2^-107 keeps all of fp32's
    bits there, one of 2^-112 its 24."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q = (torch.randn(sum(new), heads, c.D, generator=g, device="cuda") * qscale).bfloat16()
    out = torch.empty_like(q)
    moe.moe_attention(handle(), c.desc, c.batch(new, lens), q, out)
    ok(handle())
    want, _, bound = attention(c, new, lens, q, c.D ** -0.5)
    assert torch.isfinite(out).all()
    err, bound = (out.double() - want).abs(), bound - 1e-30
    assert (err <= bound).all(), (err / bound).max().item()


def powers(fmt):
    return (123, -112) if fmt == moe.MOE_KV_MXFP4 else (119, -107)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk,D", [(32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("end", [0, 1])
@pytest.mark.parametrize("qscale", [0.0, 0.05, 1.0])
def test_prompts_in_parts_and_whole(fmt, blk, D, end, qscale):
    power = powers(fmt)[end]
    for heads, kv, new, lens in ((16, 2, [40], [4000]), (32, 4, [16, 1, 40], [1100, 2049, 3000]), (32, 16, [600], [1500])):
        check(cache(fmt, lens, kv, D, blk, power), new, lens, heads, qscale)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk,D", [(32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("end", [0, 1])
@pytest.mark.parametrize("qscale", [0.0, 0.05, 1.0])
def test_single_tokens(fmt, blk, D, end, qscale):
    """Items of 8 and 16 rows; one that all CTAs share, several that end within a CTA and within a group's run."""
    power = powers(fmt)[end]
    for heads, kv, new, lens in ((8, 1, [1], [9000]), (16, 1, [1], [9000]), (8, 2, [1] * 5, [4000, 70, 1, 1300, 700]),
                                 (4, 4, [1] * 60, [300, 90, 500] * 20), (40, 4, [2] * 3, [900, 2000, 150])):
        check(cache(fmt, lens, kv, D, blk, power), new, lens, heads, qscale)
