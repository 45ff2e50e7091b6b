"""Sampling against its definition in 64 bits.  The kernel's exponential is an
fp32 one, so where the reference's running sums come within its error of a
decision (a filter's end, or u's place) either side of it is right."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import bit_moe_decode_02_gb300 as moe  # noqa: E402
from ops_testlib import handle, ok  # noqa: E402

REL = 2.0 ** -21     # of a weight: an fp32 exponential (2 units in the last place) and the rounding to 2^-31 added below


def f(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda") if v is not None else None


def sample(logits, temperature=None, top_k=None, top_p=None, min_p=None, u=None, logprob=True):
    M = logits.shape[0]
    tok = torch.full((M,), -5, dtype=torch.int32, device="cuda")
    lp = torch.full((M,), 5.0, device="cuda") if logprob else None
    k = torch.tensor(top_k, dtype=torch.int32, device="cuda") if top_k is not None else None
    o = handle()
    moe.moe_sample(o, logits, f(temperature), k, f(top_p), f(min_p), f(u), tok, lp)
    ok(o)
    return tok.cpu().numpy(), lp.cpu().numpy() if logprob else None


def agrees(l, T, k, p, q, u, tok, lp):
    """Whether `tok` is the definition's token for one row, within the exponential's error."""
    l = np.where(np.isnan(l), -np.inf, l).astype(np.float32)
    top = l.max()
    with np.errstate(all="ignore"):
        z = np.where(l == top, np.float32(0), (l - top) * np.float32(np.float32(1) / np.float32(max(T, 1e-30))))
    z = np.where(l == -np.inf, -np.inf, z).astype(np.float64)
    w = np.rint(np.exp(z) * 2.0 ** 31)
    order = np.argsort(-l.astype(np.float64), kind="stable")
    if k and 0 < k < len(l):
        order = order[:k]
    wo = w[order]
    slack = wo.sum() * REL + len(wo)
    sizes = {len(order)}
    if p is not None and p < 1:
        cum = np.cumsum(wo)
        need = [max(1.0, math.ceil(float(np.float32(p)) * cum[-1] + d)) for d in (-slack, 0, slack)]
        first, last = (int(np.searchsorted(cum, n)) + 1 for n in (need[0], need[2]))
        sizes = set(range(max(first, 1), min(last, len(order)) + 1))
        assert len(sizes) < 50
    for size in sizes:
        kept = order[:size]
        least = min(max(float(np.float32(q)) if q else 0.0, 0.0), 1.0) * 2.0 ** 31
        for d in (0, 1, -1):
            keep = kept[w[kept] >= least * (1 + d * REL) + d * (1 if least else 0)]
            if tok not in keep:
                continue
            keep = np.sort(keep)
            cum = np.cumsum(w[keep])
            at = int(np.searchsorted(keep, tok))
            target = min(max(float(np.float32(u)), 0.0), 1 - 2.0 ** -24) * cum[-1]
            if (cum[at - 1] if at else 0.0) - slack <= target <= cum[at] + slack and w[tok] > 0:
                want = z[tok] - math.log(cum[-1] / 2.0 ** 31)
                if lp is None or abs(lp - want) <= 2.0 ** -20 * max(1.0, abs(z[tok])):
                    return True
    return False


def check(logits, T=None, k=None, p=None, q=None, seed=0, u=None):
    M = logits.shape[0]
    rng = np.random.default_rng(seed)
    u = rng.random(M, dtype=np.float32) if u is None else np.asarray(u, np.float32)
    tok, lp = sample(logits, T, k, p, q, u.tolist())
    host = logits.float().cpu().numpy()
    g = lambda a, m, d: d if a is None else a[m]  # noqa: E731
    for m in range(M):
        assert agrees(host[m], g(T, m, 1.0), g(k, m, 0), g(p, m, None), g(q, m, 0.0), u[m], tok[m], lp[m]), (m, tok[m], lp[m])


def rows(M, V, seed=0, sigma=2.5, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, V, generator=g, device="cuda") * sigma).to(dtype)


@pytest.mark.parametrize("V", [1, 2, 31, 100, 1000, 4097, 32000, 151643, 524288])
@pytest.mark.parametrize("M", [1, 7])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_filters(V, M, dtype):
    l = rows(M, V, V + M, dtype=dtype)
    rng = np.random.default_rng(V)
    T = (0.3 + rng.random(M)).tolist()
    k = rng.integers(1, min(V, 300) + 1, M).tolist()
    p = (0.05 + 0.94 * rng.random(M)).tolist()
    q = (0.2 * rng.random(M)).tolist()
    check(l)
    check(l, T)
    check(l, T, k)
    check(l, T, None, p)
    check(l, T, None, None, q)
    check(l, T, k, p, q)
    check(l, None, k, p)
    check(l, T, rng.integers(0, V + 2, M).tolist(), p)


@pytest.mark.parametrize("M", [1, 3, 20, 153, 400])
def test_batches(M):
    l = rows(M, 5003, M)
    rng = np.random.default_rng(M)
    check(l, (0.5 + rng.random(M)).tolist(), rng.integers(-1, 60, M).tolist(), (0.5 + 0.6 * rng.random(M)).tolist(), (0.1 * rng.random(M)).tolist())


def test_rows_apart():
    """Rows of a larger tensor, at odd offsets."""
    big = rows(5, 10011, 3)
    check(big[:, 7:10008], [0.9] * 5, [50] * 5, [0.9] * 5)


def test_ties():
    """Equal logits: lower indexes first, in every filter."""
    V = 3000
    l = torch.zeros(4, V, device="cuda")
    tok, lp = sample(l, None, [1, 10, 0, 0], [1.0, 1.0, 0.25, 1.0], None, [0.999] * 4)
    assert tok.tolist() == [0, 9, 749, 2997]
    assert np.allclose(lp, [0.0, -math.log(10), -math.log(750), -math.log(V)], atol=1e-5)
    l[:, 5::7] = 1.0
    check(l, [1.0] * 4, [100, 429, 430, 0], [1.0, 1.0, 0.9, 0.3], u=[0.99, 0.5, 0.999, 0.2])
    l = -torch.zeros(1, V, device="cuda")
    l[0, ::2] = 0.0                       # -0 and +0 are the same logit
    assert sample(l, None, [3], None, None, [0.999])[0].tolist() == [2]


def test_many_ties_at_the_cut():
    """A bf16 row of few distinct values: the cut falls among thousands of equal ones."""
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randint(0, 6, (6, 40000), generator=g, device="cuda").to(torch.bfloat16)
    check(l, [1.0] * 6, [5000, 6000, 20000, 0, 0, 39999], [1.0, 0.5, 0.999, 0.1, 0.9, 0.77])


def test_greedy():
    l = rows(3, 9999, 5)
    l[0, 77] = l[0, 5000] = 50.0
    tok, lp = sample(l, [0.0, -1.0, float("nan")], [5] * 3, [0.5] * 3, None, [0.9] * 3)
    assert tok[0] == 77 and tok.tolist()[1:] == l.argmax(1).tolist()[1:] and (lp == 0).all()
    tok, _ = sample(l, [1.0] * 3, [1] * 3, None, None, [0.9] * 3)
    assert tok[0] == 77 and tok.tolist()[1:] == l.argmax(1).tolist()[1:]
    tok, _ = sample(l, [1.0] * 3, None, [0.0] * 3, None, [0.9] * 3, logprob=False)
    assert tok[0] == 77 and tok.tolist()[1:] == l.argmax(1).tolist()[1:]
    tok, _ = sample(l, [1e-8] * 3, None, None, None, [0.3, 0.999, 0.999])
    assert tok[0] == 77 and tok.tolist()[1:] == l.argmax(1).tolist()[1:]


def test_values_that_are_not_finite():
    nan, inf = float("nan"), math.inf
    l = torch.full((6, 500), -inf, device="cuda")
    l[1] = nan
    l[2, 40], l[2, 41] = 1.0, nan
    l[3, 9], l[3, 300] = inf, inf
    l[4] = 0.0
    l[4, ::2] = -inf
    l[5] = -3e38
    l[5, 17] = 3e38
    tok, lp = sample(l, [0.7] * 6, [20, 20, 20, 0, 0, 0], [0.9, 0.9, 0.9, 1.0, 1.0, 1.0], None, [0.6] * 6)
    assert tok[0] == 0 and tok[1] == 0 and lp[0] == -inf and lp[1] == -inf
    assert tok[2] == 40 and lp[2] == 0
    assert tok[3] == 300 and abs(lp[3] + math.log(2)) < 1e-6
    assert tok[4] == 301 and abs(lp[4] + math.log(250)) < 1e-5      # the 151st of 250: 0.6 * 250 = 150 are not enough
    assert tok[5] == 17


def test_filters_among_infinities():
    l = rows(3, 5000, 8)
    l[:, 100] = l[:, 4000] = l[:, 4500] = math.inf
    tok, lp = sample(l, None, [1, 2, 0], [1.0, 1.0, 0.5], None, [0.9] * 3)
    assert tok.tolist() == [100, 4000, 4000]
    assert np.allclose(lp, [0.0, -math.log(2), -math.log(2)], atol=1e-6)


def test_ends_of_u_and_of_the_filters():
    l = rows(1, 1000, 2)
    kept = torch.sort(torch.topk(l[0], 10).indices).values.tolist()
    for u, want in ((0.0, kept[0]), (-1.0, kept[0]), (float("nan"), kept[0]), (1.0, kept[-1]), (2.0, kept[-1])):
        assert sample(l, None, [10], None, None, [u])[0][0] == want
    best = int(l.argmax())
    for p, q in ((0.0, None), (-1.0, None), (None, 1.0), (None, 7.0)):
        assert sample(l, None, None, None if p is None else [p], None if q is None else [q], [0.7])[0][0] == best
    for p in (1.0, 3.0, float("nan")):
        check(l, p=None, seed=3)
        a = sample(l, None, None, [p], [-1.0], [0.37])[0][0]
        assert a == sample(l, None, None, None, None, [0.37])[0][0]


def test_frequencies():
    """A grid of u visits each token as often as its probability says."""
    n = 4096
    l = rows(1, 50, 6, sigma=1.5).expand(n, 50).contiguous()
    tok, _ = sample(l, None, None, None, None, ((np.arange(n) + 0.5) / n).tolist())
    p = torch.softmax(l[0].double(), 0).cpu().numpy()
    assert np.abs(np.bincount(tok, minlength=50) - n * p).max() <= 1.01
