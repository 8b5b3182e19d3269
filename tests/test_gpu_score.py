"""Scores from logits and their gradient against plain float64 forms.

Tolerances, set before the first run. Forward, absolute: log p is a
difference of logits of size L = max |l| (each rounded to 2^-24 L a few
times) and a log of a sum whose terms are within 2^-22 of theirs: 2^-20 + 2^-21 L.
Entropy sums p |l - max| with |l - max| < 64 wherever p counts: 64 (2^-22 + 64 2^-24)
< 2^-11 in the worst case, and 2^-15 for the logits here (|l - max| < 20 where p > e-8).
Gradient: p is within 2^-16 of itself (|log p| 2^-23 for |log p| < 88, and the exponential),
and a bf16 result is rounded by 2^-9 of itself: 2^-8 is allowed.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import nn_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _logits(n, v, dtype, seed, masked=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = 2.5 * torch.randn(n, v, generator=g, device=DEV)
    if masked:
        x[torch.rand(n, v, generator=g, device=DEV) < 0.4] = -INF
        x[::5] = -INF
    t = torch.randint(-1, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    return x.to(dtype), t


def _check(ops, x, t, m, scale, label):
    print(f"# {label}: {tuple(x.shape)} {x.dtype} m={m}", flush=True)
    got = ops.logits_score(x, t, m, scale)
    torch.cuda.synchronize()
    # l is rounded to fp32 once; the order is that of the rounded values
    l = (x.float() * scale).double()
    lp, ent, norm, idx, top = ref.scores(l, t, m)
    fin = torch.where(torch.isfinite(l), l.abs(), 0.0)
    fin = torch.where(fin > 1e30, 0.0, fin)
    tol = 2.0 ** -20 + 2.0 ** -21 * float(fin.max())

    def close(a, b, tol):
        a = a.double()
        same = (a == b) | (torch.isnan(a) & torch.isnan(b))
        assert bool((same | ((a - b).abs() <= tol)).all()), (label, (a - b).abs()[~same].max())

    close(got.logprob, lp, tol)
    close(got.entropy, ent, 2.0 ** -15)
    close(got.norm, norm, tol)
    if m:
        assert torch.equal(got.top_idx, idx), label
        close(got.top_logprob, top, tol)
    else:
        assert got.top_idx is None and got.top_logprob is None
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,m", [
    (1, 1, 1), (1, 2, 0), (3, 7, 7), (5, 100, 16), (70, 129, 3), (2, 2047, 4), (3, 2049, 16),
    (300, 777, 2), (7, 5000, 5), (600, 4099, 16), (1, 16384, 4), (2, 70001, 8), (1, 200003, 16),
    (255, 33000, 1),
])
@pytest.mark.parametrize("masked", [False, True])
def test_scores(ops, n, v, m, dtype, masked):
    x, t = _logits(n, v, dtype, 7 * n + v, masked)
    _check(ops, x, t, m, 1.25, f"masked={masked}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_of_any_alignment(ops, dtype):
    big, t = _logits(33, 1111, dtype, 5)
    for lo, v in ((0, 1000), (1, 1000), (3, 777), (6, 1105), (1110, 1)):
        x = big[:, lo:lo + v]
        outside = big.clone()
        outside[:, lo:lo + v] = 0
        outside[outside != 0] = float("nan")  # nothing outside the view is used
        outside[:, lo:lo + v] = x
        _check(ops, outside[:, lo:lo + v], t.clamp(max=v - 1), min(4, v), 0.5, f"columns {lo}+{v}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v,m", [(50, 16), (3000, 16), (20000, 8), (70001, 16)])
def test_ties_go_to_the_lower_index(ops, dtype, v, m):
    g = torch.Generator(device=DEV)
    g.manual_seed(v)
    x = torch.randint(-2, 3, (9, v), generator=g, device=DEV).to(dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2, ::2] = -0.0  # zeros of both signs are equal
    t = torch.zeros(9, dtype=torch.int32, device=DEV)
    _check(ops, x, t, m, 1.0, "ties")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [90, 5000, 70001])
def test_masked_infinite_and_nan_places(ops, dtype, v):
    low = torch.finfo(dtype).min
    x, t = _logits(12, v, dtype, v)
    t.clamp_(min=0)
    x[0] = -INF                       # nothing left
    x[1] = low                        # every value the lowest: uniform
    x[2, 1:] = low                    # one code left
    x[3, 3:] = -INF                   # fewer left than alternatives
    x[4, v // 2] = float("nan")
    x[5, v - 1] = INF
    x[6, 5] = INF
    x[6, 6] = INF
    x[7] = float("nan")
    x[8, :-1] = -INF                  # the last code alone
    t[9], t[10] = -1, v
    t[11] = v + 5
    for scale in (1.0, 2.0):          # 2 x the lowest value is -inf
        got = _check(ops, x, t, 16, scale, f"v={v} scale={scale}")
        assert got.entropy[0] == 0 and got.logprob[0] == -INF and got.top_idx[0].eq(-1).all()
        assert got.norm[0, 0] == -INF and got.norm[0, 1] == 0
    g = torch.full((12,), 0.5, device=DEV)
    for scale in (1.0, 2.0):
        got = ops.logits_score(x, t, 0, scale)
        dx = ops.logits_score_backward(x, t, got.norm, got.entropy, g, g, scale)
        torch.cuda.synchronize()
        rows = torch.tensor([0, 1, 2, 3, 8, 9], device=DEV)
        l = (x.float() * scale).double()[rows]
        want = ref.dlogits(l, t[rows], g[rows], g[rows], scale)
        err = (dx[rows].double() - want).abs()
        assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -16).all())
        assert dx[0].eq(0).all()
        for r in (4, 5, 6, 7, 10, 11):
            assert torch.isnan(dx[r]).all(), r


def test_without_targets_and_empty_input(ops):
    x, t = _logits(4, 300, torch.float32, 3)
    a, b = ops.logits_score(x, t, 3), ops.logits_score(x, None, 3)
    assert b.logprob is None and torch.equal(a.entropy, b.entropy) and torch.equal(a.top_idx, b.top_idx)
    e = ops.logits_score(x[:0], t[:0], 3)
    assert e.logprob.shape == (0,) and e.top_idx.shape == (0, 3)
    assert ops.logits_score_backward(x[:0], t[:0], e.norm, e.entropy, e.logprob).shape == (0, 300)


def test_offsets_beyond_32_bits(ops):
    n, v = 33000, 70000  # 2.3e9 values
    x = torch.zeros((n, v), dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 30677, 30678, 32999], device=DEV)
    small, _ = _logits(4, v, torch.bfloat16, 11)
    x[rows] = small
    t = torch.full((n,), 69999, dtype=torch.int32, device=DEV)
    got = ops.logits_score(x, t, 2)
    lp, ent, norm, idx, top = ref.scores(small.double(), t[:4], 2)
    assert (got.logprob[rows].double() - lp).abs().max() < 1e-5
    assert torch.equal(got.top_idx[rows], idx)
    assert abs(float(got.entropy[1]) - np.log(v)) < 1e-4
    g = torch.ones(n, device=DEV)
    ops.logits_score_backward(x, t, got.norm, None, g, None, out=x)
    want = ref.dlogits(small.double(), t[:4], g[:4], torch.zeros(4, device=DEV), 1.0)
    assert bool(((x[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-9).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 8), (5, 101), (300, 777), (2, 8193), (1, 70001)])
@pytest.mark.parametrize("masked", [False, True])
def test_gradient(ops, n, v, dtype, masked):
    x, t = _logits(n, v, dtype, n + v, masked)
    print(f"# gradient {n}x{v} {dtype} masked={masked}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    gl, gh = torch.randn(2, n, generator=g, device=DEV)
    s = ops.logits_score(x, t, 0, 1.25)
    dx = ops.logits_score_backward(x, t, s.norm, s.entropy, gl, gh, 1.25)
    want = ref.dlogits((x.float() * 1.25).double(), t, gl, gh, 1.25)
    size = 2.0 ** -16 * (gl.abs() + gh.abs() * 20)[:, None].double()
    rel = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -16
    assert bool(((dx.double() - want).abs() <= rel * want.abs() + size).all())
    # parts: each gradient alone, none, strided and in place
    d0 = ops.logits_score_backward(x, t, s.norm, None, gl, None, 1.25)
    w0 = ref.dlogits((x.float() * 1.25).double(), t, gl, torch.zeros_like(gh), 1.25)
    assert bool(((d0.double() - w0).abs() <= rel * w0.abs() + size).all())
    assert ops.logits_score_backward(x, None, s.norm, s.entropy, None, None).eq(0).all()
    wide = torch.full((n, v + 3), 7.0, dtype=dtype, device=DEV)
    ops.logits_score_backward(x, t, s.norm, s.entropy, gl, gh, 1.25, out=wide[:, 1:v + 1])
    assert torch.equal(wide[:, 1:v + 1], dx) and wide[:, 0].eq(7).all() and wide[:, v + 1:].eq(7).all()
    ops.logits_score_backward(x, t, s.norm, s.entropy, gl, gh, 1.25, out=x)
    assert torch.equal(x, dx)


def test_gradient_against_differences(ops):
    # f = sum g_lp logprob + g_H entropy, in float64; a step of 1e-5 leaves 1e-10 of
    # curvature and 1e-11 / 1e-5 of rounding; the fp32 gradient adds 2^-16 of its size
    n, v = 6, 37
    x, t = _logits(n, v, torch.float32, 17)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    gl, gh = torch.randn(2, n, generator=g, device=DEV)
    s = ops.logits_score(x, t, 0, 0.75)
    dx = ops.logits_score_backward(x, t, s.norm, s.entropy, gl, gh, 0.75).double()

    def f(y):
        lp, ent, _, _, _ = ref.scores(y * 0.75, t, 0)
        return (gl.double() * lp + gh.double() * ent).sum()

    for k in range(4):
        u = torch.randn(n, v, generator=g, device=DEV).double()
        num = (f(x.double() + 1e-5 * u) - f(x.double() - 1e-5 * u)) / 2e-5
        assert abs(float(num - (dx * u).sum())) <= 1e-4 * float((dx * u).abs().sum()) + 1e-6


def test_another_stream_and_repeatable(ops):
    x, t = _logits(50, 70001, torch.bfloat16, 23)
    a = ops.logits_score(x, t, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = ops.logits_score(x, t, 8)
    side.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_refusals(ops):
    x, t = _logits(4, 40, torch.float32, 1)
    with pytest.raises(TypeError):
        ops.logits_score(x.double(), t)
    with pytest.raises(ValueError):
        ops.logits_score(x.cpu(), t)
    with pytest.raises(ValueError):
        ops.logits_score(x.t(), t)
    with pytest.raises(ValueError):
        ops.logits_score(x[:1].expand(4, 40), t)
    with pytest.raises(ValueError):
        ops.logits_score(x, t.long())
    with pytest.raises(ValueError):
        ops.logits_score(x, t[:3])
    for m in (-1, 17, 41):
        with pytest.raises(ops.GmmError):
            ops.logits_score(x, t, m)
    for scale in (0.0, -1.0, float("nan"), INF):
        with pytest.raises(ops.GmmError):
            ops.logits_score(x, t, 0, scale)
    with pytest.raises(ops.GmmError):
        ops.logits_score(x, t, ws=torch.empty(8, dtype=torch.uint8, device=DEV))
    s = ops.logits_score(x, t)
    with pytest.raises(ValueError):
        ops.logits_score_backward(x, t, s.norm[:, :1], s.entropy, s.logprob)
    with pytest.raises(ops.GmmError):
        ops.logits_score_backward(x, None, s.norm, s.entropy, s.logprob)
    with pytest.raises(ops.GmmError):
        ops.logits_score_backward(x, t, s.norm, None, s.logprob, s.logprob)
    with pytest.raises(ValueError):
        ops.logits_score_backward(x, t, s.norm, s.entropy, s.logprob, out=x.bfloat16())
