"""The operators of a decode step together: blocks planned on the GPU, a projection with adapters beside it, rotary positions
in place, the cache and attention over it, against the same layer in 64 bits; and the example with all of them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from bit_moe_decode_02_gb300 import build_ext  # noqa: E402
from examples.decode import Model  # noqa: E402
from kv4_testlib import Cache4  # noqa: E402
from ops_testlib import Cache, attention, handle, i32, ok  # noqa: E402


class Layer:
    """A projection to queries, keys and values with adapters, and what a step does with them."""

    def __init__(self, fmt, B=3, H=8, Hk=2, D=64, hidden=256, rank=16, blk=32, blocks=40, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.Hk, self.D, self.blk = B, H, Hk, D, blk
        rows = (H + 2 * Hk) * D
        codes = torch.randint(0, 256, (rows, hidden // 2), dtype=torch.uint8, generator=g, device="cuda")
        scales = torch.randint(119, 122, (rows, hidden // 32), dtype=torch.uint8, generator=g, device="cuda")
        self.w = moe.moe_linear_of(codes, scales, None, moe.MOE_FMT_MXFP4, 32)
        self.lora = moe.moe_lora_of((torch.randn(2, rank, hidden, generator=g, device="cuda") * 0.1).bfloat16(),
                                    (torch.randn(2, rows, rank, generator=g, device="cuda") * 0.1).bfloat16(),
                                    torch.tensor([0.5, 2.0], device="cuda"))
        self.adapter = i32([0, 1, -1][:B])
        self.rope = moe.moe_rope_of(D, 10000.0)
        self.cache = Cache4([1], Hk, D, blk, num_blocks=blocks) if fmt == moe.MOE_KV_MXFP4 else Cache([1], Hk, D, blk, fmt, num_blocks=blocks)
        self.table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
        self.pool = moe.moe_kv_pool_of(torch.randperm(blocks, generator=g, device="cuda").int(), self.table, blk)
        self.kv_len, self.state, self.new = i32([0] * B), i32([5, blocks]), i32([0] * B)
        self.cu, self.admitted = i32([0] * (B + 1)), i32([0])
        self.g = g

    def buffers(self, room, hidden=256):
        e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.qkv, self.out = e(room, hidden), e(room, (self.H + 2 * self.Hk) * self.D), e(room, self.H, self.D)
        self.seq, self.pos = e(room, t=torch.int32), e(room, t=torch.int32)
        self.batch = moe.moe_kv_batch_of(self.cu, self.kv_len, self.table, room)

    def step(self):
        o, H, Hk, D = handle(), self.H, self.Hk, self.D
        moe.moe_kv_plan(o, self.pool, self.new, self.kv_len, self.state, self.cu, self.kv_len, self.state, self.admitted, self.seq, self.pos)
        index = torch.where(self.seq >= 0, self.adapter[self.seq.clamp_min(0).long()], -1)
        moe.moe_linear(o, self.w, self.x, self.qkv)
        moe.moe_lora(o, self.lora, index, self.x, self.qkv)
        self.q, self.k, self.v = (t.unflatten(1, (-1, D)) for t in self.qkv.split((H * D, Hk * D, Hk * D), 1))
        moe.moe_rope(o, self.rope, self.pos, self.q, self.k)
        moe.moe_kv_write(o, self.cache.desc, self.batch, self.k, self.v)
        moe.moe_attention(o, self.cache.desc, self.batch, self.q, self.out)

    def check(self, counts, lens):
        """q, k and v against 64 bits, then attention over what the cache holds, and the cache against k and v.

        Three roundings to bf16, of 2^-8 of the value that is rounded at most: the projection W x, its sum y with the adapter's part,
        and the rotated pair, which is no larger than |u| + |v|; an error of u or v before the rotation reaches both.  W x may be
        larger than y, so it counts by itself.  fp32 sums: 2^-19 of the projection's magnitudes (256 columns) and, as in the adapters'
        own test, (256 / 16 + 32) 2^-23 < 2^-17 of theirs."""
        T, D = sum(counts), self.D
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
        codes, scales, _ = self.w.tensors
        w = torch.stack((value[(codes & 15).long()], value[(codes >> 4).long()]), -1).flatten(1)
        w = w * torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), scales.double() - 127).repeat_interleave(32, 1)
        x = self.x[:T].double()
        y, mag = x @ w.t(), x.abs() @ w.abs().t() * 2.0 ** -19
        mag += y.abs() * 2.0 ** -8
        a, b, s = self.lora.tensors
        seq = torch.repeat_interleave(torch.arange(self.B, device="cuda"), torch.tensor(counts, device="cuda"))
        for m in range(T):
            i = int(self.adapter[seq[m]])
            if i >= 0:
                h = a[i].double() @ x[m]
                y[m] += float(s[i]) * (b[i].double() @ h)
                mag[m] += abs(float(s[i])) * (b[i].double().abs() @ (a[i].double().abs() @ x[m].abs())) * 2.0 ** -17
        mag += 2 * y.abs() * 2.0 ** -8                        # of y, and of the rotated pair
        pos = torch.cat([torch.arange(n - c, n, device="cuda") for c, n in zip(counts, lens)]).double()
        t = (pos[:, None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -2.0 * torch.arange(D // 2, device="cuda") / D))[:, None]
        y, turn = y.unflatten(1, (-1, D)), self.H + self.Hk
        u, v = y[:, :turn, :D // 2], y[:, :turn, D // 2:]
        want = torch.cat((torch.cat((u * t.cos() - v * t.sin(), v * t.cos() + u * t.sin()), -1), y[:, turn:]), 1)
        got = self.qkv[:T].double().unflatten(1, (-1, D))
        bound = 1.01 * mag.unflatten(1, (-1, 2, D // 2)).sum(-2, keepdim=True).expand(-1, -1, 2, -1).flatten(-2)      # of u and of v
        assert ((got - want).abs() <= bound).all()
        c = self.cache
        c.table = self.table.cpu().numpy()
        ref, _, limit = attention(c, counts, lens, self.q[:T], D ** -0.5)
        assert ((self.out[:T].double() - ref).abs() <= limit).all()
        at = 0
        for n, (b, length) in zip(counts, enumerate(lens)):
            if n:
                for have, src in zip(c.values(b, length), (self.k, self.v)):
                    put = src[at:at + n].double()
                    # a code's half step: 2^-4 of the group's or block's largest for 8 bits and more, 1/6 for E2M1 (half of 2 in 6, or of
                    # a scale that is up to twice what the largest needs)
                    worst = put.abs().amax() if n == length else max(put.abs().amax(), have.abs().amax())
                    assert ((have[length - n:] - put).abs() <= worst / (6 if c.fmt == moe.MOE_KV_MXFP4 else 16)).all()
            at += n


@pytest.mark.parametrize("fmt", [moe.MOE_KV_E4M3, moe.MOE_KV_INT8, moe.MOE_KV_MXFP4])
def test_a_captured_step(fmt):
    """Captured once and replayed for prompts, single tokens, an ended and an idle stream: nothing between steps but new inputs."""
    layer, room = Layer(fmt), 60
    layer.buffers(room)
    layer.step()
    ok(handle())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    lens = [0, 0, 0]
    for counts in ([20, 1, 37], [1, 1, 1], [1, 0, 1], [1, 33, -1], [1, 1, 9]):
        layer.new.copy_(i32(counts))
        layer.x.copy_(torch.randn(layer.x.shape, generator=layer.g, device="cuda"))
        graph.replay()
        ok(handle())
        lens = [0 if n < 0 else a + n for a, n in zip(lens, counts)]
        assert layer.kv_len.tolist() == lens and int(layer.admitted) == 3
        layer.check([max(n, 0) for n in counts], lens)


def test_the_example_with_a_4_bit_cache_and_adapters():
    build_ext.build()
    prompts, runs = [[1, 2, 3], [4] * 90, [5]], []
    for adapters in (2, 2, 0):
        model = Model(streams=3, cache_format=moe.MOE_KV_MXFP4, adapters=adapters)
        runs.append(model.generate(prompts, 6))
        assert model.lengths == [3 + 5, 90 + 5, 1 + 5] and model.kv_len.tolist() == model.lengths
        model.close()
    assert runs[0] == runs[1]
    assert runs[0][2] == runs[2][2]                          # the last stream has no adapter
    assert runs[0][:2] != runs[2][:2]
    assert all(len(t) == 6 and all(0 <= x < 1000 for x in t) for t in runs[0])
