"""What moe_rope and its tables refuse beside what tests/test_more_ops_host.py has, and what the binding hands to the library; no
GPU is needed.  The handle and the pointers here are never followed."""
import ctypes

import pytest

import bit_moe_decode_02_gb300 as moe
from test_more_ops_host import A, INV, L, lora, o, rope  # noqa: F401
from test_more_ops_host import test_turns as check_turns


@pytest.mark.parametrize("kw,word", [
    (dict(position=9 * A), "q_out overlaps position"), (dict(position=9 * A - 8), "q_out overlaps position"),
    (dict(position=9 * A + 512 * 2 * 3 - 4), "q_out overlaps position"), (dict(turns=9 * A + 1024), "q_out overlaps turns"),
    (dict(turns=10 * A - 248), "k_out overlaps turns"), (dict(position=10 * A + 4), "k_out overlaps position"),
    (dict(qos=520, position=9 * A + 1032), "q_out overlaps position"),                                # from the gap into the next row
    (dict(q=9 * A, qs=512, position=9 * A + 512), "q_out overlaps position"),                         # in place
    (dict(qos=512 + 128, turns=9 * A + 1280 + 1024 + 8), "q_out overlaps turns")])
def test_rope_outputs_over_positions_or_the_table(L, o, kw, word):  # noqa: F811
    """Another token's row would overwrite a position or a speed before it is read."""
    assert rope(L, o, **kw) == INV and word in moe.moe_last_error()


def test_rope_positions_beside_the_outputs(L, o):  # noqa: F811
    """What ends where an output begins, begins where it ends, or lies between two of its rows is no overlap: the check after it,
    of the outputs' own, is what refuses these."""
    for kw in (dict(position=9 * A - 12), dict(position=9 * A + 512 * 2 * 3), dict(turns=9 * A - 256), dict(qos=520, position=9 * A + 1024),
               dict(qos=512 + 128, turns=9 * A + 1024), dict(qos=512 + 128, turns=9 * A + 1280 + 1024)):
        assert rope(L, o, ko=9 * A + 16, kos=kw.get("qos", 512), **kw) == INV and "q_out overlaps k_out" in moe.moe_last_error()


class Fake:
    """Stands for a CUDA tensor: what the binding looks at."""

    def __init__(self, kind, *shape, at=A):
        self.dtype, self.shape, self.is_cuda, self.at, self.device = kind, shape, True, at, "cuda"

    def data_ptr(self):
        return self.at

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]


def calls(handle, bad):
    """Each call that hands its arguments over as words, with something that the library refuses where `bad`."""
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    cache = moe.moe_kv_cache(A, A, 10, 2, 64, 16 if bad else 64, moe.MOE_KV_E4M3)
    batch, rows = moe.moe_kv_batch(A, A, A, 2, 3, 4), Fake(bf, 3, 2, 64)
    ints = [Fake(i32, 2, at=k * A) for k in range(1, 6)]
    return {
        "moe_kv_write": lambda: moe.moe_kv_write(handle, cache, batch, rows, rows, stream=1),
        "moe_kv_read": lambda: moe.moe_kv_read(handle, cache, batch, rows, rows, stream=1),
        "moe_rope": lambda: moe.moe_rope(handle, moe.moe_rope_table(A, 66 if bad else 64, 0, 1.0), Fake(i32, 3), rows, stream=1),
        "moe_kv_plan": lambda: moe.moe_kv_plan(handle, moe.moe_kv_pool(A, A, 10, 2, 4, 16 if bad else 64), *ints[:3], Fake(i32, 3), *ints[3:],
                                               n_tokens=5, stream=1),
        "moe_lora": lambda: moe.moe_lora(handle, moe.moe_lora_weights(A, A, None, 1, 12 if bad else 8, 64, 64), Fake(i32, 3), Fake(bf, 3, 64),
                                         Fake(bf, 3, 64, at=2 * A), stream=1)}


@pytest.mark.parametrize("name", ["moe_kv_write", "moe_kv_read", "moe_rope", "moe_kv_plan", "moe_lora"])
def test_the_library_sees_every_handle(L, o, name):  # noqa: F811
    """None is refused by the library, in its words; a ctypes.c_void_p is a handle as an address is: the check after the handle's is
    the one that speaks."""
    for none in (None, ctypes.c_void_p()):
        with pytest.raises(moe.MoeError, match=f"{name}: .*(handle|may be NULL)") as e:
            calls(none, False)[name]()
        assert e.value.status == INV
    for handle in (o, ctypes.c_void_p(o)):
        with pytest.raises(moe.MoeError, match=f"{name}: .*(block=16|rot_dim=66|rank=12)"):
            calls(handle, True)[name]()


def test_rope_without_a_table(L, o):  # noqa: F811
    torch = pytest.importorskip("torch")
    with pytest.raises(moe.MoeError, match="moe_rope: the handle, the table"):
        moe.moe_rope(o, None, Fake(torch.int32, 3), Fake(torch.bfloat16, 3, 2, 64), stream=1)


def test_adapters_without_an_output(o):  # noqa: F811
    torch = pytest.importorskip("torch")
    w = moe.moe_lora_weights(A, A, None, 1, 8, 64, 64)
    with pytest.raises(ValueError, match="moe_lora: out"):
        moe.moe_lora(o, w, Fake(torch.int32, 3), Fake(torch.bfloat16, 3, 64), None, stream=1)


@pytest.mark.parametrize("kind", [moe.MOE_ROPE_LINEAR, moe.MOE_ROPE_PARTS, moe.MOE_ROPE_WAVELENGTH])
def test_factors_that_leave_no_fraction(L, kind):  # noqa: F811
    """A speed above 2^53 has no fraction of a turn in a double: such factors are refused, and down to 2^-32 the table holds what
    tests/test_more_ops_host.py asks of every table."""
    par = dict(length=4096.0, low=1.0, high=32.0)
    for factor in (1e-300, 2.0 ** -33):
        with pytest.raises(moe.MoeError, match="factor"):
            moe.moe_rope_turns(64, 10000.0, kind, factor, **par)
    check_turns(64, 10000.0, kind, (2.0 ** -32, *par.values()))


def test_adapters_beside_their_input(L, o):  # noqa: F811
    """x and out as columns of one buffer share no byte: the check after theirs, of y and out, is what refuses these; a row more to the
    left, a row too wide, or another pitch, and they do."""
    w = dict(rows=100, cols=256)
    for kw in (dict(x=8 * A, xs=512, out=8 * A + 512, os=512), dict(x=8 * A + 256, xs=512, out=8 * A, os=512),
               dict(x=8 * A, xs=512, out=8 * A + 512, os=256, type=0)):
        size = 4 if kw.get("type") == 0 else 2
        assert lora(L, o, w, y=kw["out"] + size, ys=kw["os"], **kw) == INV and "y overlaps out" in moe.moe_last_error()
    for kw in (dict(x=8 * A, xs=512, out=8 * A + 510, os=512), dict(x=8 * A + 192, xs=512, out=8 * A, os=512),
               dict(x=8 * A, xs=512, out=8 * A + 512, os=520), dict(x=8 * A, xs=512, out=8 * A + 512, os=512, type=0)):
        assert lora(L, o, w, y=None, ys=0, **kw) == INV and "x overlaps out" in moe.moe_last_error()
