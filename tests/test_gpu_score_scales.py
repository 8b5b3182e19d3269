"""Scales that are no power of two: l = scale * x is one fp32 number wherever it is used.

Compared with float64 forms of the rounded l. What is left beside l itself: the rounding of
l - max l where it counts (2^-20 below 32, twice), the exponential's (2^-22) and the
logarithm's: 2^-18 in log p, the log-sum and the alternatives at any size of l. Entropy sums
p |l - max| < 64 p: 2^-15. Gradient: p within 2^-16 of itself, and a bf16 result (8
significant bits) 2^-8 of itself. A logit whose l overflows gives its row NaN.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import nn_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")
SCALES = [0.7, 0.8, 0.9, 0.3, 1.25, 1.0 / 3.0]


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _l(x, scale):
    return (x.float() * torch.tensor(scale, dtype=torch.float32, device=DEV)).double()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [90, 5000, 70001])
@pytest.mark.parametrize("scale", SCALES)
def test_far_offsets(ops, dtype, v, scale):
    g = torch.Generator(device=DEV)
    g.manual_seed(v)
    offsets = torch.tensor([0.0, 50.0, -1e4, 1e5, -1e6, 1e6, -1e9, 1e12], device=DEV)
    n = len(offsets)
    x = (2.5 * torch.randn(n, v, generator=g, device=DEV) + offsets[:, None]).to(dtype)
    x[:, 1::7] = -INF
    t = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    print(f"# v={v} {dtype} scale={scale}", flush=True)
    s = ops.logits_score(x, t, 5, scale)
    l = _l(x, scale)
    lp, ent, norm, idx, top = ref.scores(l, t, 5)
    assert torch.equal(s.top_idx, idx)
    assert torch.equal(s.norm[:, 0].double(), norm[:, 0])
    for got, want, tol in ((s.norm[:, 1], norm[:, 1], 2.0 ** -18), (s.entropy, ent, 2.0 ** -15)):
        assert (got.double() - want).abs().max() <= tol
    near = lp > -32  # beyond, the rounding of l - max l itself passes the tolerance
    assert ((s.logprob.double() - lp)[near].abs() <= 2.0 ** -18).all()
    near = top > -32
    assert ((s.top_logprob.double() - top)[near].abs() <= 2.0 ** -18).all()
    gl, gh = torch.randn(2, n, generator=g, device=DEV)
    dx = ops.logits_score_backward(x, t, s.norm, s.entropy, gl, gh, scale).double()
    want = ref.dlogits(l, t, gl, gh, scale)
    p = torch.softmax(l, 1)
    size = 2.0 ** -16 * p * (gl.abs() + gh.abs() * 64)[:, None].double() + 1e-30
    rel = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -16
    assert bool(((dx - want).abs() <= rel * want.abs() + size).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [90, 5000, 70001])
@pytest.mark.parametrize("scale", SCALES)
def test_a_target_has_its_alternatives_log_probability(ops, dtype, v, scale):
    low = torch.finfo(dtype).min
    values = [-3.0, 1e4, -1e9, 1e9, -1e20, low if scale < 1 else low / 2]
    x = torch.tensor(values, device=DEV)[:, None].expand(-1, v).to(dtype).contiguous()
    x[0, 5] = 1.5
    n = len(values)
    for at in (0, 2, 5):
        t = torch.full((n,), at, dtype=torch.int32, device=DEV)
        s = ops.logits_score(x, t, 6, scale)
        where = s.top_idx == at
        assert bool(where.any(1).all())
        assert torch.equal(s.top_logprob[where], s.logprob)
        assert (s.norm[1:, 1].double() - math.log(v)).abs().max() <= 2.0 ** -19, s.norm
        assert (s.entropy[1:].double() - math.log(v)).abs().max() <= 2.0 ** -19
        assert torch.equal(s.norm[1:, 0].double(), _l(x[1:, 0], scale))
        g = torch.ones(n, device=DEV)
        dx = ops.logits_score_backward(x, t, s.norm, s.entropy, g, None, scale).double()[1:]
        want = torch.full_like(dx, -scale / v)
        want[:, at] += scale
        rel = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -16
        assert bool(((dx - want).abs() <= rel * want.abs() + 2.0 ** -16 * scale / v).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [90, 5000])
@pytest.mark.parametrize("m", [0, 2])
def test_heads_of_one_value(ops, dtype, v, m):
    n = 40
    for scale in SCALES:
        for e in (10, 30, 40, 100, 126):
            for sign in (1.0, -1.0):
                print(f"# v={v} {dtype} m={m} scale={scale} value {sign} * 1.5 * 2^{e}", flush=True)
                h = torch.ones(n, 1, device=DEV, dtype=dtype)
                w = torch.full((v, 1), sign * 1.5 * 2.0 ** e, device=DEV, dtype=dtype)
                t = torch.full((n,), v - 1, dtype=torch.int32, device=DEV)
                s = ops.head_score(h, w, t, m, scale)
                assert torch.equal(s.norm[:, 0].double(), _l(w[0], scale).expand(n))
                for got in (s.norm[:, 1], s.entropy, -s.logprob):
                    assert (got.double() - math.log(v)).abs().max() <= 2.0 ** -19, got
                # every code has 1 / v of the row: dw = sum over rows of scale g ([v = t] - 1 / v)
                g = torch.full((n,), 1.0 / n, device=DEV)
                _, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, g, None, scale)
                want = torch.full((v,), -scale / v, dtype=torch.float64, device=DEV)
                want[-1] += scale
                rel = 2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -15
                assert bool(((dw[:, 0].double() - want).abs() <= rel * want.abs()).all())


@pytest.mark.parametrize("v", [90, 5000, 70001])
def test_logits_whose_scaled_value_overflows(ops, v):
    x = torch.zeros(6, v, device=DEV)
    x[1, 3] = 3e38       # 1.25 * 3e38 is beyond fp32
    x[2] = 3e38
    x[3] = -3e38         # l = -inf: nothing left
    x[4, 7] = 2.5e38     # within
    x[5, v - 1] = -3e38  # one code masked
    t = torch.tensor([0, 0, 1, 2, 7, 4], dtype=torch.int32, device=DEV)
    for m in (0, 4):
        s = ops.logits_score(x, t, m, 1.25)
        for r in (1, 2):
            assert torch.isnan(s.norm[r]).all() and torch.isnan(s.entropy[r]) and torch.isnan(s.logprob[r])
        assert s.norm[3].tolist() == [-INF, 0.0] and s.logprob[3] == -INF and s.entropy[3] == 0
        assert s.logprob[4] == 0 and s.norm[4, 1] == 0
        for r, k in ((0, v), (5, v - 1)):
            assert abs(float(s.norm[r, 1]) - math.log(k)) <= 2.0 ** -19
    g = torch.ones(6, device=DEV)
    dx = ops.logits_score_backward(x, t, s.norm, s.entropy, g, g, 1.25)
    assert torch.isnan(dx[1]).all() and torch.isnan(dx[2]).all() and dx[3].eq(0).all()
    assert torch.isfinite(dx[[0, 4, 5]]).all() and dx[5, v - 1] == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0, 700, 4999])  # in a whole tile of codes and in the last one
def test_heads_whose_scaled_logit_overflows(ops, dtype, at):
    v = 5000
    w = torch.zeros(v, 2, device=DEV)
    w[:, 1] = torch.arange(v, device=DEV) % 5 / 4
    w[at, 0] = 2.0 ** 100
    h = torch.zeros(300, 2, device=DEV)
    h[:, 1] = 1.0
    h[7, 0] = 1.75 * 2.0 ** 27   # x = 1.75 * 2^127, 1.25 of which is beyond fp32
    h[290, 0] = 1.25 * 2.0 ** 27
    h, w = h.to(dtype), w.to(dtype)
    t = torch.full((300,), 3, dtype=torch.int32, device=DEV)
    for m in (0, 2):
        s = ops.head_score(h, w, t, m, 1.25)
        assert torch.isnan(s.norm[7]).all() and torch.isnan(s.entropy[7]) and torch.isnan(s.logprob[7])
        assert s.norm[290, 1] == 0 and s.entropy[290] == 0
        rest = torch.arange(300, device=DEV)
        rest = rest[(rest != 7) & (rest != 290)]
        assert torch.equal(s.norm[rest], s.norm[:1].expand(298, 2)) and torch.isfinite(s.norm[0]).all()
