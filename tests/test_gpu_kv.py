"""The 8-bit paged cache against its definition: every code and scale that
moe_kv_write leaves, and every value that moe_kv_read returns, bit for bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import Cache, block_scale, decode, encode, handle, ok  # noqa: E402

FMTS = [moe.MOE_KV_E4M3, moe.MOE_KV_INT8]


class Model:
    """What the cache has to hold, in numpy."""

    def __init__(self, cache: Cache):
        self.c = cache
        self.codes = cache.codes.cpu().numpy().copy()
        self.scales = cache.scales.cpu().numpy().copy()

    def write(self, new, kv_len, k, v):
        c, at = self.c, 0
        for b, (n, t) in enumerate(zip(new, kv_len)):
            for which, src in ((0, k), (1, v)):
                x = src[at:at + n].float().cpu().numpy()
                for j in range((t - n) // c.blk, (t - 1) // c.blk + 1) if n else ():
                    lo, hi = max(t - n - j * c.blk, 0), min(t - j * c.blk, c.blk)
                    part = x[j * c.blk + lo - (t - n):j * c.blk + hi - (t - n)]
                    for h in range(c.H):
                        self._block(c.table[b, j], h, which, lo, hi, part[:, h])
            at += n

    def _block(self, pid, h, which, lo, hi, x):
        c = self.c
        codes = self.codes[pid, h, which].reshape((c.blk, c.D) if which == 0 else (c.D, c.blk))
        codes = codes if which == 0 else codes.T
        s = block_scale(x, c.fmt)
        old = self.scales[pid, h, which]
        with np.errstate(all="ignore"):
            if lo == 0:
                codes[:] = 0
            elif s > old:
                ratio = np.float32(old * np.float32(np.float32(1) / s))
                codes[:lo] = encode(np.float32(decode(codes[:lo], c.fmt)) * ratio, c.fmt)
            else:
                s = old
            self.scales[pid, h, which] = s
            codes[lo:hi] = encode(x * np.float32(np.float32(1) / s), c.fmt)

    def check(self):
        assert np.array_equal(self.scales, self.c.scales.cpu().numpy())
        got = self.c.codes.cpu().numpy()
        bad = np.argwhere(got != self.codes)
        assert bad.size == 0, (bad[:5], len(bad))


def _values(T, H, D, seed, kind="normal"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, 2, H, D, generator=g, device="cuda")
    if kind == "spread":
        x *= torch.pow(2.0, torch.randint(-30, 30, x.shape, generator=g, device="cuda").float())
    if kind == "odd":
        r = torch.rand(x.shape, generator=g, device="cuda")
        x = torch.where(r < 0.05, float("nan"), torch.where(r < 0.1, float("inf"), torch.where(r < 0.15, -float("inf"), x)))
        x = torch.where((r > 0.2) & (r < 0.4), 0.0, x)
    if kind == "tiny":
        x *= 2.0 ** -125
    if kind == "huge":
        x = torch.clamp(x * 2.0 ** 126, -3.38e38, 3.38e38)
    if kind == "zero":
        x *= 0
    x = x.bfloat16()
    return x[:, 0], x[:, 1]       # rows of a fused tensor: strided


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["normal", "spread", "odd"])
def test_write_is_bit_exact(fmt, blk, D, kind):
    """Fresh blocks, blocks continued with and without a larger scale, sequences without tokens; then tokens one by one
    across a block's end."""
    o, H = handle(), 3
    had, new = [0, 5, blk - 1, blk, 2 * blk + 7, 3, 0], [1, 2 * blk + 3, 2, 1, blk, 0, blk]
    end = [a + b for a, b in zip(had, new)]
    c = Cache([e + 70 for e in end], H, D, blk, fmt, seed=blk + D)
    c.codes.random_(0, 120)                      # stale bytes everywhere
    m = Model(c)
    steps = [(had, had), (new, end)]
    for i in range(35):
        steps.append(([1, 0, 1, 1, 1, 0, 1], [e + (i + 1) * f for e, f in zip(end, [1, 0, 1, 1, 1, 0, 1])]))
    for i, (n, t) in enumerate(steps):
        k, v = _values(sum(n), H, D, 100 * blk + i, kind)
        if i == 1:
            k, v = (k.float() * 3).bfloat16(), v     # the keys' scales grow, the values' mostly do not
        m.write(n, t, k, v)
        moe.moe_kv_write(o, c.desc, c.batch(n, t), k, v)
    ok(o)
    m.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", ["tiny", "huge", "zero"])
def test_write_at_the_ends_of_the_range(fmt, kind):
    o = handle()
    c = Cache([100], 2, 64, 64, fmt)
    m = Model(c)
    for i, (n, t) in enumerate([([70], [70]), ([30], [100])]):
        k, v = _values(n[0], 2, 64, i, kind if i == 0 else "normal")
        m.write(n, t, k, v)
        moe.moe_kv_write(o, c.desc, c.batch(n, t), k, v)
    ok(o)
    m.check()
    assert torch.isfinite(c.scales).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_read_is_bit_exact(fmt, blk, D):
    o, H = handle(), 3
    lens = [1, blk, 3 * blk + 5, 40, 777]
    new = [1, blk - 3, 2 * blk + 7, 0, 600]
    c = Cache(lens, H, D, blk, fmt, seed=3).fill(seed=blk + D)
    T = sum(new)
    fused = torch.full((T, 2, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_read(o, c.desc, c.batch(new, lens), fused[:, 0], fused[:, 1])
    ok(o)
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        k, v = c.values(b, t)
        for i, x in ((0, k), (1, v)):
            want = x[t - n:].float().bfloat16()      # the product has at most 8 + 24 bits: exact in float64, then fp32, bf16
            if fmt == moe.MOE_KV_INT8:               # ... where fp32 rounds first, as the kernel's product does
                want = x[t - n:].to(torch.float32).bfloat16()
            assert torch.equal(fused[at:at + n, i], want)
        at += n


@pytest.mark.parametrize("fmt", FMTS)
def test_round_trip_error(fmt):
    """A value comes back within half a step: of INT8's scale, or 2^-4 of itself (E4M3), and one bf16 rounding."""
    o = handle()
    c = Cache([500], 4, 128, 64, fmt)
    k, v = _values(500, 4, 128, 5)
    b = c.batch([500], [500])
    moe.moe_kv_write(o, c.desc, b, k, v)
    rk, rv = torch.empty_like(k.contiguous()), torch.empty_like(v.contiguous())
    moe.moe_kv_read(o, c.desc, b, rk, rv)
    ok(o)
    for i, (x, r) in enumerate(((k, rk), (v, rv))):
        pos = torch.arange(500, device="cuda") // 64
        s = c.scales[torch.from_numpy(c.table[0].astype(np.int64)).cuda()[pos], :, i][..., None].double()
        x, r = x.double(), r.double()
        step = 0.5 * s if fmt == moe.MOE_KV_INT8 else torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)
        assert ((x - r).abs() <= step * 1.0001 + r.abs() * 2.0 ** -8).all()


def test_blocks_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes, used at its end."""
    o = handle()
    nb = (1 << 32) // (8 * 2 * 128 * 128) + 40
    c = Cache([300, 200], 8, 128, 128, moe.MOE_KV_INT8, num_blocks=nb)
    c.table[0, :3], c.table[1, :2] = [nb - 1, nb - 3, nb - 2], [nb - 5, 2]
    c.dtable = torch.from_numpy(c.table).cuda()
    k, v = _values(500, 8, 128, 9)
    b = c.batch([300, 200], [300, 200])
    moe.moe_kv_write(o, c.desc, b, k, v)
    rk, rv = torch.empty(500, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(500, 8, 128, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_read(o, c.desc, b, rk, rv)
    ok(o)
    assert ((rk.double() - k.double()).abs() <= 6.0 / 254 + 6 * 2.0 ** -8).all()
    assert ((rv.double() - v.double()).abs() <= 6.0 / 254 + 6 * 2.0 ** -8).all()
    del c, k, v, rk, rv
    torch.cuda.empty_cache()


def test_bad_metadata_sets_the_status_and_spares_the_rest():
    o = handle()
    c = Cache([100, 100, 100], 2, 64, 64, moe.MOE_KV_E4M3).fill(1)
    k, v = _values(30, 2, 64, 1)
    good = c.batch([10, 10, 10], [100, 100, 100])
    for cu, lens, spoil in (([0, 10, 5, 30], [100, 100, 100], None),       # not increasing
                            ([0, 10, 20, 31], [100, 100, 100], None),      # past the batch
                            ([0, 10, 20, 30], [100, 9, 100], None),        # fewer cached than new
                            ([0, 10, 20, 30], [100, 1 << 30, 100], None),  # past the table
                            ([0, 10, 20, 30], [100, 100, 100], -1), ([0, 10, 20, 30], [100, 100, 100], c.codes.shape[0])):
        table, before = c.dtable.clone(), c.codes.clone()
        if spoil is not None:
            table[1, 1] = spoil
        bad = moe.moe_kv_batch_of(torch.tensor(cu, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table, 30)
        moe.moe_kv_write(o, c.desc, bad, k, v)
        assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
        ids = torch.from_numpy(c.table[1, :2].astype(np.int64)).cuda()
        if spoil is None and cu[3] == 30:
            assert torch.equal(c.codes[ids], before[ids])
    moe.moe_kv_write(o, c.desc, good, k, v)
    ok(o)


def test_another_stream():
    """Work on a stream of its own, its inputs made there: nothing runs on the default stream."""
    o = handle()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Cache([300], 2, 64, 64, moe.MOE_KV_INT8)
        k, v = _values(300, 2, 64, 2)
        b = c.batch([300], [300])
        rk, rv = torch.empty_like(k.contiguous()), torch.empty_like(v.contiguous())
        moe.moe_kv_write(o, c.desc, b, k, v)
        moe.moe_kv_read(o, c.desc, b, rk, rv)
        assert moe.moe_ops_get_status(o) == 0
        assert ((rk.double() - k.double()).abs() <= 6.0 / 254 + 6 * 2.0 ** -8).all()


@pytest.mark.parametrize("n_seqs,last", [(33, 40), (33, 31), (100, 500), (65, -1)])
def test_bad_metadata_past_the_blocks_of_the_batch(n_seqs, last):
    """The first sequences account for every token of the batch; the metadata of the last one is wrong all the same."""
    o = handle()
    n = n_seqs - 1
    c = Cache([10] * n_seqs, 1, 64, 64, moe.MOE_KV_INT8)
    k, v = _values(n, 1, 64, 1)
    cu = list(range(n)) + [n, last]
    bad = moe.moe_kv_batch_of(torch.tensor(cu, dtype=torch.int32).cuda(), torch.tensor([10] * n_seqs, dtype=torch.int32).cuda(),
                              c.dtable, n)
    moe.moe_kv_write(o, c.desc, bad, k, v)
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    moe.moe_kv_read(o, c.desc, bad, k.contiguous(), v.contiguous())
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
    q = torch.randn(n, 2, 64, device="cuda").bfloat16()
    moe.moe_attention(o, c.desc, bad, q, torch.empty_like(q))
    assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
