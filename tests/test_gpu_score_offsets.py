"""Scores do not change when one number is added to a row's logits.

log p, entropy and the log-sum are functions of l - max l. Here that difference is exact in
fp32 at every offset (grid values below 2^24 of their step), so that the outputs have to be the
same bit for bit. Rows of one value have log sum = log v: the sum of v <= 2^24 ones is exact and
its logarithm is off by one unit of 2^-20 (log v < 16) at most; 2^-19 is allowed at any offset.
The gradient of such a row is g ([v = t] - 1 / v) within 2^-16 of its terms, and a bf16 result
(8 significant bits) is off by 2^-8 of itself.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _grid(n, v, seed, top):
    """Multiples of 1/8 in [-top, 0], their order with ties; int32 targets."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = -torch.randint(0, 8 * top + 1, (n, v), generator=g, device=DEV).float() / 8
    t = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    return x, t


@pytest.mark.parametrize("v", [90, 5000, 16384, 70001])
def test_logits_at_any_offset(ops, v):
    x, t = _grid(7, v, v, 30)
    g = torch.linspace(-1, 1, 7, device=DEV)
    a = ops.logits_score(x, t, 8)
    da = ops.logits_score_backward(x, t, a.norm, a.entropy, g, g)
    for off in (100.0, -1e3, 1e4, -1e5, 1e6, -1e6):
        print(f"# v={v} offset {off}", flush=True)
        y = x + off
        b = ops.logits_score(y, t, 8)
        assert torch.equal(b.norm[:, 0], a.norm[:, 0] + off)
        assert torch.equal(b.norm[:, 1], a.norm[:, 1]), (b.norm[:, 1] - a.norm[:, 1]).abs().max()
        assert torch.equal(b.logprob, a.logprob) and torch.equal(b.entropy, a.entropy)
        assert torch.equal(b.top_idx, a.top_idx) and torch.equal(b.top_logprob, a.top_logprob)
        db = ops.logits_score_backward(y, t, b.norm, b.entropy, g, g)
        assert torch.equal(db, da)


VALUES = [0.0, -1e4, 1e4, -1e8, -1e9, 1e9, -1e10, -1e12, 1e12, -1e30, 1e30, -3e38, 3e38]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [90, 5000, 70001])
def test_logits_of_one_value(ops, dtype, v):
    x = torch.tensor(VALUES, device=DEV)[:, None].expand(-1, v).to(dtype).contiguous()
    t = torch.full((len(VALUES),), v - 1, dtype=torch.int32, device=DEV)
    s = ops.logits_score(x, t, 3)
    assert torch.equal(s.norm[:, 0], x[:, 0].float())
    want = math.log(v)
    for got in (s.norm[:, 1], s.entropy, -s.logprob, -s.top_logprob[:, 0], -s.top_logprob[:, 2]):
        assert (got.double() - want).abs().max() <= 2.0 ** -19, got
    g = torch.ones(len(VALUES), device=DEV)
    dx = ops.logits_score_backward(x, t, s.norm, s.entropy, g).double()
    w = torch.full_like(dx, -1.0 / v)
    w[:, -1] += 1
    rel = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -16
    assert bool(((dx - w).abs() <= rel * w.abs() + 2.0 ** -16 / v).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(4, 300), (70, 1000), (300, 5000), (3, 20000)])
@pytest.mark.parametrize("m", [0, 3])
def test_heads_at_any_offset(ops, dtype, n, v, m):
    # one dim carries the offset: every product and every sum of them is exact
    base, t = _grid(n, v, n + v, 3)
    h = torch.zeros(n, 5, device=DEV)
    w = torch.zeros(v, 5, device=DEV)
    h[:, 0], w[:, 0] = 1.0, base[0]
    h[:, 1], w[:, 1] = torch.arange(n, device=DEV) % 8, torch.arange(v, device=DEV) % 4 / 8
    h[:, 2] = 1.0
    a = ops.head_score(h.to(dtype), w.to(dtype), t, m)
    for off in (2.0 ** 7, -2.0 ** 10, 2.0 ** 14, -2.0 ** 17, 2.0 ** 20, -2.0 ** 20):
        print(f"# {n} x {v} {dtype} m={m} offset {off}", flush=True)
        w[:, 2] = off
        b = ops.head_score(h.to(dtype), w.to(dtype), t, m)
        assert torch.equal(b.norm[:, 0], a.norm[:, 0] + off)
        assert torch.equal(b.norm[:, 1], a.norm[:, 1]), (b.norm[:, 1] - a.norm[:, 1]).abs().max()
        assert torch.equal(b.logprob, a.logprob) and torch.equal(b.entropy, a.entropy)
        if m:
            assert torch.equal(b.top_idx, a.top_idx) and torch.equal(b.top_logprob, a.top_logprob)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [90, 5000])
@pytest.mark.parametrize("m", [0, 2])
def test_heads_of_one_value(ops, dtype, v, m):
    for e in (10, 14, 27, 30, 34, 40, 100, 126):
        for sign in (1.0, -1.0):
            print(f"# v={v} {dtype} m={m} value {sign} * 2^{e}", flush=True)
            h = torch.ones(300, 1, device=DEV, dtype=dtype)
            w = torch.full((v, 1), sign * 2.0 ** e, device=DEV, dtype=dtype)
            t = torch.full((300,), v - 1, dtype=torch.int32, device=DEV)
            s = ops.head_score(h, w, t, m)
            assert torch.equal(s.norm[:, 0], w[0].float().expand(300))
            for got in (s.norm[:, 1], s.entropy, -s.logprob):
                assert (got.double() - math.log(v)).abs().max() <= 2.0 ** -19, got
