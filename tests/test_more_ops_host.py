"""Rotary tables, and what the operators around the cache refuse before any CUDA call; no GPU is needed.  The handle
and the pointers here are never followed."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import bit_moe_decode_02_gb300 as moe
from bit_moe_decode_02_gb300 import build_ext

A = 1 << 20      # an aligned address
INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


@pytest.fixture(scope="module")
def L():
    build_ext.build()
    return moe.lib()


@pytest.fixture(scope="module")
def o():
    buf = ctypes.create_string_buffer(1024)       # stands for a handle: refusals come before its use
    yield ctypes.addressof(buf)
    del buf


def _speeds(rot, base, kind, factor, length, low, high):
    """f_i in doubles, from the definition."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = np.power(float(base), -2.0 * i / rot)
    if kind == moe.MOE_ROPE_LINEAR:
        return f / factor
    if kind == moe.MOE_ROPE_PARTS:
        at = lambda n: rot * np.log(length / (2 * np.pi * n)) / (2 * np.log(base))  # noqa: E731
        a, b = max(at(high), 0.0), min(at(low), rot / 2 - 1)
        x = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        return f * (1 - x) + f / factor * x
    if kind == moe.MOE_ROPE_WAVELENGTH:
        x = np.clip((length * f / (2 * np.pi) - low) / (high - low), 0, 1)
        return f * x + f / factor * (1 - x)
    return f


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (54, 500000.0), (64, 150000.0), (128, 10000.0), (512, 1e6), (64, 1.5)])
@pytest.mark.parametrize("kind,par", [(moe.MOE_ROPE_PLAIN, (1.0, 0, 0, 0)), (moe.MOE_ROPE_LINEAR, (4.0, 0, 0, 0)), (moe.MOE_ROPE_LINEAR, (0.01, 0, 0, 0)),
                                      (moe.MOE_ROPE_PARTS, (32.0, 4096, 1.0, 32.0)), (moe.MOE_ROPE_WAVELENGTH, (8.0, 8192, 1.0, 4.0))])
def test_turns(rot, base, kind, par):
    """Within a few units of the double's last place (pow, log and the blends round a handful of times) of f / 2 pi mod 1."""
    got = moe.moe_rope_turns(rot, base, kind, *par)
    assert got.dtype == np.uint64 and got.shape == (rot // 2,)
    for g, f in zip(got.tolist(), _speeds(rot, base, kind, *par)):
        want = Fraction(float(f)) / (2 * PI)
        off = (Fraction(g, 2 ** 64) - want) % 1
        off = min(off, 1 - off)
        assert off <= want * 8 * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 62), (float(off), float(want))


def test_turns_of_plain_frequencies_are_exact_to_the_double():
    """f = 1 (pair 0): 1 / 2 pi to within a unit of 2^-62, far below the double's own 2^-55."""
    assert abs(Fraction(int(moe.moe_rope_turns(64, 10000.0)[0]), 2 ** 64) - 1 / (2 * PI)) < Fraction(1, 2 ** 62)


@pytest.mark.parametrize("kw,word", [
    (dict(rot_dim=0), "rot_dim"), (dict(rot_dim=3), "rot_dim"), (dict(rot_dim=514), "rot_dim"), (dict(scaling=4), "scaling"),
    (dict(scaling=-1), "scaling"), (dict(base=1.0), "base"), (dict(base=float("nan")), "base"), (dict(base=float("inf")), "base"),
    (dict(scaling=1, factor=0.0), "factor"), (dict(scaling=1, factor=float("inf")), "factor"), (dict(scaling=2, length=0.0), "length"),
    (dict(scaling=2, low=0.0), "low"), (dict(scaling=3, high=1.0), "high"), (dict(scaling=3, high=float("nan")), "high")])
def test_turns_refusals(L, kw, word):
    d = dict(rot_dim=64, scaling=0, base=1e4, factor=2.0, length=100.0, low=1.0, high=4.0)
    d.update(kw)
    c = moe.moe_rope_config(*[d[f] for f, _ in moe.moe_rope_config._fields_])
    out = (ctypes.c_ulonglong * 256)()
    assert L.moe_rope_turns(ctypes.byref(c), out) == INV and word in moe.moe_last_error()
    assert L.moe_rope_turns(None, out) == INV
    assert L.moe_rope_turns(ctypes.byref(c), None) == INV


def rope(L, o, **kw):
    d = dict(turns=A, rot=64, layout=0, mscale=1.0, position=A, T=3, D=64, type=1, q=8 * A, qs=640, qh=8, qo=9 * A, qos=512, k=8 * A + 1024,
             ks=640, kh=2, ko=10 * A, kos=128)
    d.update(kw)
    t = moe.moe_rope_table(d["turns"], d["rot"], d["layout"], d["mscale"])
    return L.moe_rope(o, t, d["position"], d["T"], d["D"], d["type"], d["q"], d["qs"], d["qh"], d["qo"], d["qos"], d["k"], d["ks"], d["kh"],
                      d["ko"], d["kos"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(turns=None), "NULL"), (dict(position=None), "NULL"), (dict(type=2), "type"), (dict(layout=2), "layout"), (dict(D=60), "head_dim"),
    (dict(D=520), "head_dim"), (dict(rot=66), "rot_dim"), (dict(rot=0), "rot_dim"), (dict(rot=31), "rot_dim"),
    (dict(mscale=float("nan")), "mscale"), (dict(T=0), "n_tokens"), (dict(T=(1 << 20) + 1), "n_tokens"), (dict(qh=0), "q_heads"),
    (dict(kh=-1), "k_heads"), (dict(kh=1025), "k_heads"), (dict(turns=A + 4), "aligned"), (dict(position=A + 2), "aligned"),
    (dict(q=None), "q must"), (dict(k=None), "k must"), (dict(qo=None), "q_out must"), (dict(ko=None), "k_out must"),
    (dict(q=8 * A + 8), "aligned"), (dict(qs=644), "multiple"), (dict(qs=504), "less than"), (dict(kos=120), "less than"),
    (dict(qo=8 * A + 16, qos=640), "overlaps"), (dict(qo=8 * A, qos=648), "overlaps"), (dict(ko=9 * A + 512), "overlaps"),
    (dict(qo=8 * A + 256, qos=640, q=7 * A), "overlaps"), (dict(type=0, qs=642), "multiple")])
def test_rope_refusals(L, o, kw, word):
    assert rope(L, o, **kw) == INV and word in moe.moe_last_error() and "moe_rope" in moe.moe_last_error()


def test_rope_needs_a_handle_and_a_table(L, o):
    assert rope(L, None) == INV
    assert L.moe_rope(o, None, A, 1, 64, 1, A, 64, 1, A, 64, None, 0, 0, None, 0, None) == INV


def plan(L, o, pool={}, **kw):
    p = dict(ring=A, table=2 * A, ring_size=100, n_seqs=5, table_stride=10, block=64)
    p.update(pool)
    d = dict(n_new=3 * A, kv_len=4 * A, state=5 * A, n_tokens=50, cu=6 * A, kv_len_out=7 * A, state_out=8 * A, admitted=9 * A, seq=10 * A,
             position=11 * A, slot=12 * A)
    d.update(kw)
    return L.moe_kv_plan(o, moe.moe_kv_pool(*[p[f] for f, _ in moe.moe_kv_pool._fields_]), *d.values(), None)


@pytest.mark.parametrize("pool,kw,code,word", [
    (dict(ring=None), {}, INV, "NULL"), (dict(table=None), {}, INV, "NULL"), (dict(ring_size=0), {}, INV, "ring_size"),
    (dict(n_seqs=0), {}, INV, "n_seqs"), (dict(n_seqs=1025), {}, INV, "n_seqs"), (dict(table_stride=0), {}, INV, "table_stride"),
    (dict(block=48), {}, UNS, "block"), ({}, dict(n_new=None), INV, "NULL"), ({}, dict(kv_len=None), INV, "NULL"),
    ({}, dict(state=None), INV, "NULL"), ({}, dict(cu=None), INV, "NULL"), ({}, dict(kv_len_out=None), INV, "NULL"),
    ({}, dict(state_out=None), INV, "NULL"), ({}, dict(n_tokens=0), INV, "n_tokens"), ({}, dict(n_tokens=(1 << 20) + 1), INV, "n_tokens"),
    ({}, dict(cu=6 * A + 2), INV, "aligned"), ({}, dict(slot=12 * A + 4), INV, "slot"), ({}, dict(seq=11 * A), INV, "overlaps"),
    ({}, dict(cu=4 * A + 4), INV, "overlaps"), ({}, dict(kv_len_out=4 * A + 4), INV, "overlaps"), ({}, dict(kv_len_out=3 * A), INV, "overlaps"),
    ({}, dict(state_out=5 * A + 4), INV, "overlaps"), ({}, dict(position=2 * A + 100), INV, "overlaps"), ({}, dict(admitted=8 * A), INV, "overlaps"),
    (dict(table=A + 200), {}, INV, "overlaps")])
def test_plan_refusals(L, o, pool, kw, code, word):
    assert plan(L, o, pool, **kw) == code and word in moe.moe_last_error() and "moe_kv_plan" in moe.moe_last_error()
    assert plan(L, None) == INV
    assert L.moe_kv_plan(o, None, A, A, A, 1, A, A, A, None, None, None, None, None) == INV


def lora(L, o, w={}, **kw):
    d = dict(a=A, b=2 * A, scale=None, n_adapters=4, rank=16, rows=100, cols=256)
    d.update(w)
    e = dict(index=A, x=8 * A, xs=256, M=2, y=9 * A, ys=100, out=10 * A, os=100, type=1)
    e.update(kw)
    return L.moe_lora(o, moe.moe_lora_weights(*[d[f] for f, _ in moe.moe_lora_weights._fields_]), *e.values(), None)


@pytest.mark.parametrize("w,kw,word", [
    (dict(a=None), {}, "NULL"), (dict(b=None), {}, "NULL"), (dict(a=A + 8), {}, "aligned"), (dict(scale=A + 2), {}, "aligned"),
    (dict(n_adapters=0), {}, "n_adapters"), (dict(n_adapters=65537), {}, "n_adapters"), (dict(rank=0), {}, "rank"), (dict(rank=12), {}, "rank"),
    (dict(rank=136), {}, "rank"), (dict(rows=0), {}, "rows"), (dict(cols=100), {}, "cols"), (dict(cols=32776), {}, "cols"),
    ({}, dict(index=None), "NULL"), ({}, dict(index=A + 1), "aligned"), ({}, dict(M=0), "M="), ({}, dict(M=65), "M="),
    ({}, dict(x=None), "x must"), ({}, dict(x=8 * A + 2), "aligned"), ({}, dict(xs=248), "less than"), ({}, dict(xs=257), "multiple"),
    ({}, dict(type=2), "type"), ({}, dict(out=None), "out"), ({}, dict(out=10 * A + 1), "aligned"), ({}, dict(y=9 * A + 1), "aligned"),
    ({}, dict(os=99), "stride"), ({}, dict(ys=99), "stride"), ({}, dict(out=8 * A + 512), "overlaps"), ({}, dict(out=9 * A + 2), "overlaps"),
    ({}, dict(out=9 * A, os=101), "overlaps")])
def test_lora_refusals(L, o, w, kw, word):
    assert lora(L, o, w, **kw) == INV and word in moe.moe_last_error() and "moe_lora" in moe.moe_last_error()
    assert lora(L, None) == INV
    assert L.moe_lora(o, None, A, A, 256, 1, A, 100, A, 100, 1, None) == INV


def test_binding_refuses_tensors_of_another_form(o):
    """The C call sees only an address: the binding checks what the tensor is."""
    torch = pytest.importorskip("torch")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="ring"):
        moe.moe_kv_pool_of(i, i.reshape(2, 2), 64)
    with pytest.raises(ValueError, match="a:"):
        moe.moe_lora_of(torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="position"):
        moe.moe_rope(o, None, i, torch.zeros(4, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="index"):
        moe.moe_lora(o, moe.moe_lora_weights(A, A, None, 1, 8, 4, 64), i, torch.zeros(4, 64), torch.zeros(4, 4))
    with pytest.raises(ValueError, match="n_tokens"):
        moe.moe_kv_plan(o, moe.moe_kv_pool(A, A, 4, 2, 2, 64), i, i, i, i, i, i)


@pytest.mark.parametrize("kw,code,word", [
    (dict(scales=A), INV, "scales must be NULL"), (dict(codes=None), INV, "NULL"), (dict(codes=A + 8), INV, "aligned"), (dict(block=16), UNS, "block"),
    (dict(head_dim=96), UNS, "head_dim"), (dict(format=3), INV, "format"), (dict(format=5), INV, "format"), (dict(kv_heads=0), INV, "kv_heads")])
def test_mxfp4_cache_refusals(L, o, kw, code, word):
    d = dict(codes=A, scales=None, num_blocks=10, kv_heads=2, head_dim=64, block=64, format=moe.MOE_KV_MXFP4)
    d.update(kw)
    c = moe.moe_kv_cache(*[d[f] for f, _ in moe.moe_kv_cache._fields_])
    b = moe.moe_kv_batch(A, A, A, 2, 3, 4)
    if d["format"] in (3, 5):
        c.scales = A
    for name, call in (("moe_kv_write", lambda: L.moe_kv_write(o, c, b, A, 128, A, 128, None)),
                       ("moe_kv_read", lambda: L.moe_kv_read(o, c, b, A, 128, A, 128, None)),
                       ("moe_attention", lambda: L.moe_attention(o, c, b, A, 256, 4 if c.kv_heads else 1, 0.1, 0, None, 2 * A, None, None))):
        assert call() == code, name
        assert word in moe.moe_last_error() and name in moe.moe_last_error()
