"""The 4-bit paged cache against its definition: every byte that moe_kv_write leaves, and every value that moe_kv_read
returns, bit for bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from kv4_testlib import E2M1, Cache4, places, quantise  # noqa: E402
from ops_testlib import handle, i32, ok  # noqa: E402


class Model:
    """What the cache has to hold, in numpy."""

    def __init__(self, c):
        self.c, self.bytes = c, c.codes.cpu().numpy().copy()
        self.where = places(c.blk, c.D)

    def write(self, new, kv_len, k, v):
        c, at = self.c, 0
        for b, (n, t) in enumerate(zip(new, kv_len)):
            for i, src in ((0, k), (1, v)):
                code, scale = quantise(src[at:at + n].double().cpu().numpy())          # [n, H, D], [n, H, D / 32]
                where, nib, z = self.where[i]
                for x in range(n):
                    p = t - n + x
                    rec, o = self.bytes[c.table[b, p // c.blk], :, i], p % c.blk
                    if o == 0:
                        rec[:] = 0
                    for half in (0, 1):
                        m = nib[o] == half
                        rec[:, where[o][m]] = rec[:, where[o][m]] & (0xf0 >> 4 * half) | (code[x][:, m] << 4 * half).astype(np.uint8)
                    rec[:, z[o][::32]] = scale[x]
            at += n

    def check(self):
        got = self.c.codes.cpu().numpy()
        bad = np.argwhere(got != self.bytes)
        assert bad.size == 0, (bad[:5], len(bad))


def values(T, H, D, seed, kind="normal"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, 2, H, D, generator=g, device="cuda")
    if kind == "spread":
        x *= torch.pow(2.0, torch.randint(-30, 30, x.shape, generator=g, device="cuda").float())
    if kind == "odd":
        r = torch.rand(x.shape, generator=g, device="cuda")
        x = torch.where(r < 0.05, float("nan"), torch.where(r < 0.1, float("inf"), torch.where(r < 0.15, -float("inf"), x)))
        x = torch.where((r > 0.2) & (r < 0.4), 0.0, x)
        x[:, :, :, :32] = torch.where(r[..., :32] < 0.5, float("nan"), 0.0)             # a group without a finite value but 0
    if kind == "ties":                                                                  # a group's largest at, above and below 6 of a power of two
        x = torch.randint(-25, 26, x.shape, generator=g, device="cuda") * 0.25
    if kind == "tiny":
        x *= 2.0 ** -101
    if kind == "huge":
        x = torch.clamp(x * 2.0 ** 126, -3.38e38, 3.38e38)
    if kind == "zero":
        x *= 0
    x = x.bfloat16()
    return x[:, 0], x[:, 1]       # rows of a fused tensor: strided


@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 3, 16])
@pytest.mark.parametrize("kind", ["normal", "spread", "odd", "ties"])
def test_write_is_bit_exact(blk, D, H, kind):
    """Fresh blocks and continued ones over random bytes, sequences without tokens; then tokens one by one across a block's end."""
    o = handle()
    had, new = [0, 5, blk - 1, blk, 2 * blk + 7, 3, 0], [1, 2 * blk + 3, 2, 1, blk, 0, blk]
    end = [a + b for a, b in zip(had, new)]
    c = Cache4([n + 40 for n in end], H, D, blk, seed=blk).fill(seed=H)
    m = Model(c)
    k, v = values(sum(new), H, D, blk + D, kind)
    m.write(new, end, k, v)
    moe.moe_kv_write(o, c.desc, c.batch(new, end), k, v)
    ok(o)
    m.check()
    for step in range(36):
        one = [int(step % 3 != b % 3) for b in range(7)]
        end = [a + b for a, b in zip(end, one)]
        k, v = values(sum(one), H, D, step, kind)
        m.write(one, end, k, v)
        moe.moe_kv_write(o, c.desc, c.batch(one, end), k, v)
    ok(o)
    m.check()


@pytest.mark.parametrize("kind", ["tiny", "huge", "zero"])
def test_ends_of_the_range(kind):
    o = handle()
    c = Cache4([130], 2, 64, 64).fill(seed=1)
    m = Model(c)
    k, v = values(130, 2, 64, 5, kind)
    m.write([130], [130], k, v)
    moe.moe_kv_write(o, c.desc, c.batch([130], [130]), k, v)
    ok(o)
    m.check()


@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_read_back(blk, D):
    """Every code and scale, any part of a sequence, into strided rows; the rest of the rows stays."""
    o, H = handle(), 3
    lens = [1, blk, 3 * blk + 5, 200, 0]
    c = Cache4(lens, H, D, blk, seed=4).fill(seed=D, spread=60, centre=200)
    for new in ([1, blk, 3 * blk + 5, 200, 0], [1, 3, blk + 1, 7, 0], [0, 0, 1, 199, 0]):
        T = sum(new)
        out = torch.full((T + 1, 2, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_kv_read(o, c.desc, c.batch(new, lens), out[:T, 0, :H], out[:T, 1, :H])
        ok(o)
        at = 0
        for b, (n, t) in enumerate(zip(new, lens)):
            if n:
                for i, w in enumerate(c.values(b, t)):
                    assert torch.equal(out[at:at + n, i, :H].double(), w[t - n:])
            at += n
        assert (out[T] == 7.0).all() and (out[:, :, H] == 7.0).all()


def test_every_code_comes_back():
    o = handle()
    c = Cache4([64], 1, 64, 64)
    x = torch.tensor(list(E2M1) + list(-E2M1), device="cuda").bfloat16().repeat(64, 4)[:, None] * 2.0 ** 5
    k, v = torch.empty_like(x), torch.empty_like(x)
    moe.moe_kv_write(o, c.desc, c.batch([64], [64]), x, -x)
    moe.moe_kv_read(o, c.desc, c.batch([64], [64]), k, v)
    ok(o)
    assert torch.equal(k, x) and torch.equal(v, -x)


def test_how_tokens_came_does_not_matter():
    """The same tokens at once and one by one leave the same bytes."""
    o = handle()
    k, v = values(150, 2, 128, 3, "spread")
    a, b = Cache4([150], 2, 128, 64), Cache4([150], 2, 128, 64)
    moe.moe_kv_write(o, a.desc, a.batch([150], [150]), k, v)
    for t in range(150):
        moe.moe_kv_write(o, b.desc, b.batch([1], [t + 1]), k[t:t + 1], v[t:t + 1])
    ok(o)
    assert torch.equal(a.codes, b.codes)


@pytest.mark.parametrize("n", [300, 1024])
def test_many_sequences(n):
    o = handle()
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(1, 100, (n,), generator=g).tolist()
    new = [i % 3 for i in range(n)]
    lens = [max(a, b) for a, b in zip(lens, new)]
    c = Cache4(lens, 2, 64, 32).fill(seed=1)
    m = Model(c)
    k, v = values(sum(new), 2, 64, 1)
    m.write(new, lens, k, v)
    moe.moe_kv_write(o, c.desc, c.batch(new, lens), k, v)
    ok(o)
    m.check()


def test_bad_blocks_and_lengths():
    """A block number or a length that cannot be: the status says so, others are written."""
    o = handle()
    for what in ("table", "length"):
        c = Cache4([40, 70], 1, 64, 32, spare=3).fill(seed=2)
        m = Model(c)
        k, v = values(3, 1, 64, 9)
        lens = [40, 70]
        if what == "table":
            c.dtable[0, 1] = c.codes.shape[0]
        else:
            lens[0] = 1 << 30
        moe.moe_kv_write(o, c.desc, c.batch([1, 2], lens), k, v)
        assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
        m.write([0, 2], [40, 70], k[1:], v[1:])
        m.check()
        out = torch.full((3, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_kv_read(o, c.desc, c.batch([1, 2], lens), out, out.clone())
        assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
        assert (out[0] == 9.0).all() and torch.equal(out[1:].double(), c.values(1, 70)[0][68:])


def test_blocks_past_4_gb():
    """Blocks whose bytes lie beyond 2^32."""
    o = handle()
    c = Cache4([100], 16, 128, 128, num_blocks=1 << 15)
    c.table[0, 0] = (1 << 15) - 1
    c.dtable = i32(c.table.tolist())
    m_k, m_v = values(100, 16, 128, 2)
    k, v = torch.empty_like(m_k), torch.empty_like(m_v)
    moe.moe_kv_write(o, c.desc, c.batch([100], [100]), m_k, m_v)
    moe.moe_kv_read(o, c.desc, c.batch([100], [100]), k, v)
    ok(o)
    assert c.codes.numel() > 1 << 32 and int(c.codes[:-1].amax()) == 0
    for got, src in ((k, m_k), (v, m_v)):
        code, scale = quantise(src.double().cpu().numpy())
        want = np.append(E2M1, -E2M1)[code] * np.power(2.0, scale - 127.0).repeat(32, -1)
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_in_a_graph():
    o = handle()
    c = Cache4([90], 2, 64, 64)
    m = Model(c)
    b = c.batch([1], [90])
    k, v = values(1, 2, 64, 7)
    kk, vv = k.clone(), v.clone()
    moe.moe_kv_write(o, c.desc, b, kk, vv)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_kv_write(o, c.desc, b, kk, vv)
    k, v = values(1, 2, 64, 8)
    kk.copy_(k), vv.copy_(v)
    g.replay()
    torch.cuda.synchronize()
    m.write([1], [90], k, v)
    m.check()
