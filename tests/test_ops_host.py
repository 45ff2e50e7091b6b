"""The operators around the expert block refuse bad arguments before any CUDA
call; no GPU is needed.  The handle and the pointers here are never followed."""
import ctypes

import pytest

import bit_moe_decode_02_gb300 as moe
from bit_moe_decode_02_gb300 import build_ext

A = 1 << 20      # an aligned address


@pytest.fixture(scope="module")
def L():
    build_ext.build()
    return moe.lib()


@pytest.fixture(scope="module")
def o():
    buf = ctypes.create_string_buffer(1024)       # stands for a handle: refusals come before its use
    yield ctypes.addressof(buf)
    del buf


def cache(**kw):
    d = dict(codes=A, scales=A, num_blocks=10, kv_heads=2, head_dim=64, block=64, format=moe.MOE_KV_E4M3)
    d.update(kw)
    return moe.moe_kv_cache(*[d[f] for f, _ in moe.moe_kv_cache._fields_])


def batch(**kw):
    d = dict(cu=A, kv_len=A, table=A, n_seqs=2, n_tokens=3, table_stride=4)
    d.update(kw)
    return moe.moe_kv_batch(*[d[f] for f, _ in moe.moe_kv_batch._fields_])


INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
BAD_CACHE = [(dict(codes=None), {}, INV, "NULL"), (dict(scales=None), {}, INV, "NULL"), (dict(format=3), {}, INV, "format"),
             (dict(block=48), {}, UNS, "block"), (dict(block=0), {}, UNS, "block"), (dict(head_dim=96), {}, UNS, "head_dim"),
             (dict(kv_heads=0), {}, INV, "kv_heads"), (dict(kv_heads=300), {}, INV, "kv_heads"),
             (dict(num_blocks=0), {}, INV, "num_blocks"), (dict(codes=A + 8), {}, INV, "aligned"),
             (dict(scales=A + 4), {}, INV, "aligned"), ({}, dict(cu=None), INV, "NULL"), ({}, dict(kv_len=None), INV, "NULL"),
             ({}, dict(table=None), INV, "NULL"), ({}, dict(cu=A + 2), INV, "aligned"), ({}, dict(n_seqs=0), INV, "n_seqs"),
             ({}, dict(n_seqs=1025), INV, "n_seqs"), ({}, dict(n_tokens=0), INV, "n_tokens"),
             ({}, dict(n_tokens=(1 << 20) + 1), INV, "n_tokens"), ({}, dict(table_stride=0), INV, "table_stride")]


@pytest.mark.parametrize("c,b,code,word", BAD_CACHE)
def test_cache_and_batch(L, o, c, b, code, word):
    c, b = cache(**c), batch(**b)
    calls = (("moe_kv_write", lambda: L.moe_kv_write(o, c, b, A, 128, A, 128, None)),
             ("moe_kv_read", lambda: L.moe_kv_read(o, c, b, A, 128, A, 128, None)),
             ("moe_attention", lambda: L.moe_attention(o, c, b, A, 256, 4 if c.kv_heads else 1, 0.1, 0, None, 2 * A, None, None)))
    for name, call in calls:
        assert call() == code, name
        assert word in moe.moe_last_error() and name in moe.moe_last_error()


def test_rows(L, o):
    c, b = cache(), batch()
    for f in (L.moe_kv_write, L.moe_kv_read):
        for k, ks, v, vs, word in ((None, 128, A, 128, "k must"), (A, 128, None, 128, "v must"), (A + 2, 128, A, 128, "k must"),
                                   (A, 132, A, 128, "multiple of 8"), (A, 120, A, 128, "less than a row"), (A, 128, A, 64, "less than")):
            assert f(o, c, b, k, ks, v, vs, None) == INV and word in moe.moe_last_error()
        assert f(None, c, b, A, 128, A, 128, None) == INV
        assert f(o, None, b, A, 128, A, 128, None) == INV
        assert f(o, c, None, A, 128, A, 128, None) == INV


def test_attention(L, o):
    c, b = cache(), batch()
    nan = float("nan")
    for q, qs, heads, scale, window, sinks, out, lse, word in (
            (None, 256, 4, 0.1, 0, None, 2 * A, None, "q must"), (A + 4, 256, 4, 0.1, 0, None, 2 * A, None, "aligned"),
            (A, 250, 4, 0.1, 0, None, 2 * A, None, "multiple of 8"), (A, 128, 4, 0.1, 0, None, 2 * A, None, "less than a row"),
            (A, 256, 3, 0.1, 0, None, 2 * A, None, "q_heads"), (A, 256, 0, 0.1, 0, None, 2 * A, None, "q_heads"),
            (A, 1 << 20, 1026, 0.1, 0, None, 2 * A, None, "q_heads"), (A, 256, 4, nan, 0, None, 2 * A, None, "scale"),
            (A, 256, 4, 0.1, -1, None, 2 * A, None, "window"), (A, 256, 4, 0.1, 0, None, None, None, "out"),
            (A, 256, 4, 0.1, 0, None, 2 * A + 2, None, "out"), (A, 256, 4, 0.1, 0, A + 1, 2 * A, None, "sinks"),
            (A, 256, 4, 0.1, 0, None, 2 * A, A + 2, "lse"), (A, 256, 4, 0.1, 0, None, A + 512, None, "overlaps"),
            (A, 256, 4, 0.1, 0, None, A - 16, None, "overlaps")):
        assert L.moe_attention(o, c, b, q, qs, heads, scale, window, sinks, out, lse, None) == INV
        assert word in moe.moe_last_error()


def weights(**kw):
    d = dict(codes=A, scales=A, bias=None, rows=100, cols=256, format=moe.MOE_FMT_INT4, group=64)
    d.update(kw)
    return moe.moe_linear_weights(*[d[f] for f, _ in moe.moe_linear_weights._fields_])


@pytest.mark.parametrize("kw,word", [
    (dict(codes=None), "NULL"), (dict(scales=None), "NULL"), (dict(codes=A + 8), "aligned"), (dict(scales=A + 2), "aligned"),
    (dict(bias=A + 1), "bias"), (dict(rows=0), "rows"), (dict(rows=(1 << 24) + 1), "rows"), (dict(cols=0), "cols"),
    (dict(cols=96), "cols"), (dict(cols=32768 + 64), "cols"), (dict(format=3), "format"), (dict(group=48), "group"),
    (dict(group=0), "group"), (dict(format=moe.MOE_FMT_MXFP4), "group"), (dict(format=moe.MOE_FMT_MXFP4, group=32, cols=48), "cols")])
def test_linear_weights(L, o, kw, word):
    assert L.moe_linear(o, weights(**kw), A, 1 << 16, 2, 4 * A, 100, moe.MOE_DT_F32, None) == INV
    assert word in moe.moe_last_error() and "moe_linear" in moe.moe_last_error()


def test_linear(L, o):
    w = weights()
    for x, xs, M, out, os, kind, word in (
            (None, 256, 2, 2 * A, 100, 0, "x must"), (A + 2, 256, 2, 2 * A, 100, 0, "aligned"), (A, 255, 2, 2 * A, 100, 0, "multiple"),
            (A, 248, 2, 2 * A, 100, 0, "less than"), (A, 256, 0, 2 * A, 100, 0, "M="), (A, 256, 65, 2 * A, 100, 0, "M="),
            (A, 256, 2, None, 100, 0, "out"), (A, 256, 2, 2 * A + 2, 100, 0, "out"), (A, 256, 2, 2 * A + 1, 100, 1, "out"),
            (A, 256, 2, 2 * A, 99, 0, "stride of out"), (A, 256, 2, 2 * A, 100, 2, "output type"), (A, 256, 2, A + 64, 100, 0, "overlaps")):
        assert L.moe_linear(o, w, x, xs, M, out, os, kind, None) == INV
        assert word in moe.moe_last_error()
    assert L.moe_linear(None, w, A, 256, 1, 2 * A, 100, 0, None) == INV
    assert L.moe_linear(o, None, A, 256, 1, 2 * A, 100, 0, None) == INV


def test_sample(L, o):
    p = moe.moe_sample_params(None, None, None, None, A)
    for l, kind, stride, M, V, par, tok, lp, word in (
            (None, 0, 100, 2, 100, p, A, None, "NULL"), (A, 2, 100, 2, 100, p, A, None, "type"), (A, 0, 99, 2, 100, p, A, None, "stride"),
            (A, 0, 100, 0, 100, p, A, None, "M="), (A, 0, 100, 65536, 100, p, A, None, "M="), (A, 0, 100, 2, 0, p, A, None, "V="),
            (A, 0, 1 << 20, 2, (1 << 19) + 1, p, A, None, "V="), (A, 0, 100, 2, 100, None, A, None, "NULL"),
            (A, 0, 100, 2, 100, p, None, None, "NULL"), (A + 2, 0, 100, 2, 100, p, A, None, "aligned"), (A, 0, 100, 2, 100, p, A + 2, None, "aligned"),
            (A, 0, 100, 2, 100, p, A, A + 1, "aligned"), (A + 1, 1, 100, 2, 100, p, A, None, "aligned"),
            (A, 0, 100, 2, 100, moe.moe_sample_params(None, None, None, None, None), A, None, "u must"),
            (A, 0, 100, 2, 100, moe.moe_sample_params(A + 2, None, None, None, A), A, None, "aligned")):
        assert L.moe_sample(o, l, kind, stride, M, V, par, tok, lp, None) == INV
        assert word in moe.moe_last_error()
    assert L.moe_sample(None, A, 0, 100, 2, 100, p, A, None, None) == INV


def test_handle(L):
    assert L.moe_ops_create(None) == INV
    assert L.moe_ops_get_status(None, None) == INV
    L.moe_ops_destroy(None)
    import torch
    if not torch.cuda.is_available():
        h = ctypes.c_void_p(123)
        assert L.moe_ops_create(ctypes.byref(h)) == moe.MOE_ERR_CUDA and h.value is None


def test_binding_refuses_tensors_of_another_form():
    """The C call sees only an address: the binding checks what the tensor is."""
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 2, 2, 64 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_kv_cache_of(t, torch.zeros(4, 2, 2), 64, 64, moe.MOE_KV_E4M3)
    with pytest.raises(ValueError, match="cu"):
        moe.moe_kv_batch_of(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="codes"):
        moe.moe_linear_of(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), None, moe.MOE_FMT_MXFP4, 32)
