"""Block tables, positions and slots of a step against a walk over the requests."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import Cache, attention, handle, i32, ok  # noqa: E402


class Pool:
    """A pool's state in Python lists, and one step of it from the definition."""

    def __init__(self, lens, blk, stride, blocks, seed=0, head=None):
        r = random.Random(seed)
        ids = r.sample(range(blocks), blocks)
        self.blk, self.stride, self.size, self.lens = blk, stride, blocks, list(lens)
        self.table = [[-9] * stride for _ in lens]
        for b, n in enumerate(lens):
            for j in range(-(-n // blk)):
                self.table[b][j] = ids.pop()
        self.head = r.randrange(blocks) if head is None else head
        self.ring = [-5] * blocks
        for i, x in enumerate(ids):
            self.ring[(self.head + i) % blocks] = x
        self.count = len(ids)
        self.d = dict(ring=i32(self.ring), table=i32(self.table), len=i32(self.lens), state=i32([self.head, self.count]))
        self.desc = moe.moe_kv_pool_of(self.d["ring"], self.d["table"], blk)

    def step(self, new, room):
        cu, seq, pos, slot, admitted, back, free = [0], [], [], [], None, [], self.count
        lens = list(self.lens)
        for b, n in enumerate(new):
            if n < 0:
                back += self.table[b][:-(-self.lens[b] // self.blk)]
                lens[b] = 0
            held = -(-self.lens[b] // self.blk)
            need = -(-(self.lens[b] + max(n, 0)) // self.blk) - held
            if admitted is None and (need > free or cu[-1] + max(n, 0) > room):
                admitted = b
            if admitted is not None:
                cu.append(cu[-1])
                continue
            for j in range(held, held + need):
                self.table[b][j] = self.ring[self.head]
                self.head = (self.head + 1) % self.size
                free -= 1
            for i in range(max(n, 0)):
                p = self.lens[b] + i
                seq.append(b), pos.append(p), slot.append(self.table[b][p // self.blk] * self.blk + p % self.blk)
            cu.append(cu[-1] + max(n, 0))
            if n > 0:
                lens[b] += n
        for i, x in enumerate(back):
            self.ring[(self.head + free + i) % self.size] = x
        self.count, self.lens = free + len(back), lens
        pad = [-1] * (room - len(seq))
        return cu, lens, [self.head, self.count], [len(new) if admitted is None else admitted], seq + pad, pos + pad, slot + pad

    def run(self, new, room, in_place=False):
        o = handle()
        e = lambda n, t=torch.int32: torch.full((n,), -77, dtype=t, device="cuda")  # noqa: E731
        n = len(new)
        out = [e(n + 1), self.d["len"] if in_place else e(n), self.d["state"] if in_place else e(2), e(1), e(room), e(room), e(room, torch.int64)]
        moe.moe_kv_plan(o, self.desc, i32(new), self.d["len"], self.d["state"], *out)
        ok(o)
        self.d["len"], self.d["state"] = out[1], out[2]
        want = self.step(new, room)
        for name, w, g in zip(("cu", "kv_len", "state", "admitted", "seq", "position", "slot"), want, out):
            assert g.tolist() == w, name
        assert self.d["table"].tolist() == self.table
        assert self.d["ring"].tolist() == self.ring
        return out


@pytest.mark.parametrize("blk", [32, 64, 128])
@pytest.mark.parametrize("seqs", [1, 2, 31, 33, 256, 1024])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps(blk, seqs, in_place):
    """Prompts, then single tokens, ends and idle requests, with more blocks than needed: every output of every step."""
    r = random.Random(seqs + blk)
    lens = [r.choice([0, 0, 1, blk - 1, blk, blk + 1, r.randrange(5 * blk)]) for _ in range(seqs)]
    p = Pool(lens, blk, 40, sum(-(-n // blk) for n in lens) + seqs * 12 + 3, seed=seqs)
    p.run([r.choice([0, 1, blk, r.randrange(4 * blk)]) for _ in range(seqs)], 4 * blk * seqs + 5, in_place)
    for k in range(4):
        new = [r.choice([-1, 0, 1, 1, 1, 2]) for _ in range(seqs)]
        p.run(new, 2 * seqs + k, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_blocks_and_tokens_that_do_not_fit(in_place):
    """Few free blocks: those before the first that does not fit are served, exactly up to the last block; then the same with
    the room for tokens.  Ended requests give their blocks back all the same."""
    for free in range(0, 12):
        p = Pool([0, 10, 32, 5, 64], 32, 20, 5 + free, seed=free)
        p.run([33, 22, 64, -1, 1], 200, in_place)
        p.run([1, 1, 1, 40, 1], 200, in_place)
    for room in (1, 32, 33, 54, 55, 118, 119, 120, 121):
        p = Pool([0, 10, 32, 5, 64], 32, 20, 30, seed=room)
        p.run([33, 22, 64, -1, 1], room, in_place)


def test_the_ring_wraps():
    p = Pool([0, 0], 32, 8, 9, head=8)
    p.run([100, 60], 160)
    for _ in range(8):
        p.run([-1, 0], 1)
        p.run([70, -1], 70, True)
        p.run([-1, 90], 90)


@pytest.mark.parametrize("in_place", [False, True])
def test_many_tokens(in_place):
    """Enough for every SM, one long request among short ones, tokens up to the largest batch."""
    lens = [3] * 400
    p = Pool(lens, 64, 9000, 400 + 12000)
    new = [5] * 400
    new[200] = 500000
    p.run(new, (1 << 20) if in_place else 502017, in_place)


def test_the_same_inputs_give_the_same_outputs():
    """Not in place: a second call after the first leaves everything as it is."""
    o = handle()
    p = Pool([40, 0, 7], 32, 10, 30)
    new, e = i32([50, -1, 1]), lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = [e(4), e(3), e(2)]
    moe.moe_kv_plan(o, p.desc, new, p.d["len"], p.d["state"], *out, n_tokens=60)
    first = [t.clone() for t in (*out, p.d["table"], p.d["ring"])]
    moe.moe_kv_plan(o, p.desc, new, p.d["len"], p.d["state"], *out, n_tokens=60)
    ok(o)
    assert all(torch.equal(a, b) for a, b in zip(first, (*out, p.d["table"], p.d["ring"])))


def test_bad_lengths_and_states():
    """A length, a count of new tokens or a state that cannot be: the status says so, the sequence keeps what it has, others go on."""
    o = handle()
    e = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(p, new, lens=None, state=None):
        cu, ln, st, adm, pos = e(4), e(3), e(2), e(1), e(50)
        moe.moe_kv_plan(o, p.desc, i32(new), p.d["len"] if lens is None else i32(lens), p.d["state"] if state is None else i32(state), cu, ln, st,
                        adm, position=pos)
        assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
        return cu.tolist(), ln.tolist(), st.tolist(), adm.tolist()
    fresh = lambda: Pool([10, 20, 30], 32, 3, 20, head=0)  # noqa: E731
    assert call(fresh(), [1, -2, 1]) == ([0, 1, 1, 2], [11, 20, 31], [0, 17], [3])
    assert call(fresh(), [1, 77, 1]) == ([0, 1, 1, 2], [11, 20, 31], [0, 17], [3])                # past the row of the table
    assert call(fresh(), [1, 2 ** 31 - 1, 1]) == ([0, 1, 1, 2], [11, 20, 31], [0, 17], [3])
    assert call(fresh(), [1, 1, 1], [10, -3, 30]) == ([0, 1, 1, 2], [11, -3, 31], [0, 17], [3])
    assert call(fresh(), [1, -1, 1], [10, 2 ** 31 - 1, 30]) == ([0, 1, 1, 2], [11, 2 ** 31 - 1, 31], [0, 17], [3])
    for state in ([-1, 5], [20, 5], [0, -1], [0, 21]):
        assert call(fresh(), [1, -1, 1], state=state) == ([0, 0, 0, 0], [10, 20, 30], state, [0])
    # more blocks come back than there are: none does
    assert call(fresh(), [1, -1, 1], state=[0, 20]) == ([0, 1, 1, 2], [11, 20, 31], [0, 20], [3])


def test_block_numbers_out_of_range():
    """Passed on as they are, with a slot of -1, and the status set."""
    o = handle()
    for bad in (-1, 20, 2 ** 31 - 1):
        p = Pool([10, 0], 32, 3, 20, head=0)
        p.d["ring"][0] = bad
        p.d["table"][0, 0] = bad
        cu, ln, st, slot = (torch.empty(n, dtype=t, device="cuda") for n, t in ((3, torch.int32), (2, torch.int32), (2, torch.int32), (4, torch.int64)))
        moe.moe_kv_plan(o, p.desc, i32([1, 2]), p.d["len"], p.d["state"], cu, ln, st, slot=slot)
        assert moe.moe_ops_get_status(o) == moe.MOE_ERR_DEVICE_FAULT
        assert slot.tolist() == [-1] * 4 and int(p.d["table"][1, 0]) == bad and cu.tolist() == [0, 1, 3]


def test_its_batch_goes_through_the_cache():
    """Captured once, replayed for every step, updated in place: plan, write, attention over what was planned."""
    o = handle()
    H, D, blk, B, room = 2, 64, 32, 3, 70
    c = Cache([1], H, D, blk, moe.MOE_KV_E4M3, num_blocks=24)
    p = Pool([0, 0, 0], blk, 8, 24)
    new, g = i32([0, 0, 0]), torch.Generator(device="cuda").manual_seed(3)
    cu, adm, pos = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (B + 1, 1, room))
    k, v = (torch.empty(room, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, out = (torch.empty(room, 4, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    batch = moe.moe_kv_batch_of(cu, p.d["len"], p.d["table"], room)

    def step():
        moe.moe_kv_plan(o, p.desc, new, p.d["len"], p.d["state"], cu, p.d["len"], p.d["state"], adm, position=pos)
        moe.moe_kv_write(o, c.desc, batch, k, v)
        moe.moe_attention(o, c.desc, batch, q, out)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = [0, 0, 0]
    for counts in ([40, 1, 29], [1, 1, 1], [0, 33, 1], [-1, 1, 1], [5, 0, 2]):
        new.copy_(i32(counts))
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        out.fill_(9.0)
        graph.replay()
        ok(o)
        lens = [0 if n < 0 else a + n for a, n in zip(lens, counts)]
        counts = [max(n, 0) for n in counts]
        assert p.d["len"].tolist() == lens and cu.tolist()[-1] == sum(counts)
        c.table = p.d["table"].cpu().numpy()
        T = sum(counts)
        want, _, bound = attention(c, counts, lens, q[:T], D ** -0.5)
        assert ((out[:T].double() - want).abs() <= bound).all()
        assert (out[T:] == 9.0).all()
