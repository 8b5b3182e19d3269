"""Alternatives of rows with many equal logits: as many candidates as a row's kernel counts, picks or
looks for one by one, for rows of one wave, of 256 threads and of 1024.

The logits are small whole numbers and their order is given by (value, index): the indices are compared
for equality with a stable sort. Log-probabilities: l - max is exact; the sum of v exponentials, each off by 2^-22 of
itself at most (the hardware's base 2 exponential and the factor before it, for differences below 16), in any order,
is off by (v 2^-24 + 2^-22) of itself, its logarithm by as much and by 2^-22 of the logarithm, and the result is
rounded twice.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _check(ops, x, m):
    v = x.shape[1]
    s = ops.logits_score(x, None, m)
    l = x.double()
    val, idx = l.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :m], idx[:, :m].to(torch.int32)
    none = val == -float("inf")
    assert torch.equal(s.top_idx, idx.masked_fill(none, -1))
    lse = torch.logsumexp(l - l.amax(1, keepdim=True), 1, keepdim=True)
    ref = (val - l.amax(1, keepdim=True)) - lse
    tol = v * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -22 * lse.abs() + 2.0 ** -22 * ref.abs().masked_fill(none, 0.0)
    off = (s.top_logprob.double() - ref).abs()
    assert bool((off <= tol)[~none].all()) and bool((s.top_logprob == -float("inf"))[none].all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,v", [(300, 64), (300, 130), (300, 256), (300, 1000), (20, 5000), (300, 20000), (5, 40009)])
@pytest.mark.parametrize("m", [1, 2, 5, 16])
def test_equal_logits(ops, n, v, m, dtype):
    print(f"# equal logits n={n} v={v} m={m} {dtype}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(n + v + m)
    m = min(m, v)
    x = torch.randint(-8, 4, (n, v), generator=g, device=DEV).float()
    order = torch.rand(n, v, generator=g, device=DEV).argsort(1)
    # each row has its own number of best logits; every third a second value of as many
    rows = torch.arange(n, device=DEV)
    count = torch.tensor([1, 2, 3, 5, 6, 15, 16, 17, 25, 26, 63, 64, 65, 80, 81, 128, 255, 256, 257, v],
                         device=DEV).clamp(max=v)[rows % 20]
    place = order.argsort(1)  # of a column in its row's random order
    x = torch.where(place < count[:, None], 6.0, x)
    twice = (rows % 3 == 0)[:, None] & (place >= count[:, None]) & (place < 2 * count[:, None])
    x = torch.where(twice, 5.0, x)
    _check(ops, x.to(dtype), m)
    # fewer codes left than alternatives, the rest masked
    few = torch.where(place < (rows % 18)[:, None] + 1, x, -float("inf"))
    _check(ops, few.to(dtype), m)


def _us(f):
    f()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = float("inf")
    for _ in range(5):
        a.record()
        for _ in range(5):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 5 * 1e3)
    return best


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v", [128, 256])
def test_equal_logits_take_no_multiple_of_the_time(ops, v, dtype):
    # a head before its first step: every logit 0. One wave picks among them in 1.2 to 1.3 times the time of
    # random logits (v = 128); where each of them counted all others it took 4 to 6 times as long
    n = 65536
    g = torch.Generator(device=DEV)
    g.manual_seed(v)
    x = torch.randn(n, v, generator=g, device=DEV).to(dtype)
    zero = torch.zeros_like(x)
    usual, equal = _us(lambda: ops.logits_score(x, None, 1)), _us(lambda: ops.logits_score(zero, None, 1))
    assert equal < 2.5 * usual, (usual, equal)
