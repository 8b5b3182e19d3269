"""Scores of a head without its logits, and their gradients, against float64.

Tolerances, set before the first run. With S = scale * max sum_k |h_k w_k|, a logit
is off by at most E = 2^-24 (d / 4 + 16) S: fp32 sums of blocks of 32 products,
six plane products each for fp32 data, and the terms left out (2^-23 of each).
log p and norm: 2 E + 2^-20 + 2^-21 max |l|. Entropy is sum p |l - max| at
|l - max| < 20 where p counts: 2^-15 + 40 E. Gradients: dx is off by
(4 E + 2^-16) of p g, and for bf16 data rounded to fp16 by 2^-11 (2^-10 allowed);
dh and dw are compared by that share of their sums of magnitudes, 2^-20 of them for
the fp32 sums, and a bf16 result (8 significant bits) adds 2^-8 of itself.
"""
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


def _inputs(n, d, v, dtype, seed, grid=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.randn(n, d, generator=g, device=DEV)
    w = torch.randn(v, d, generator=g, device=DEV) * 2 / d ** 0.5
    if grid:  # every sum of products is exact: ties are ties, the order is one
        h = (h * 4).round().clamp(-15, 15) / 4
        w = (w * d ** 0.5).round().clamp(-7, 7) / 16
    t = torch.randint(-1, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    return h.to(dtype), w.to(dtype), t


def _errors(h, w, scale):
    d = h.shape[1]
    s = scale * float((h.double().abs() @ w.double().abs().t()).max())
    return 2.0 ** -24 * (d / 4 + 16) * s


def _check(ops, h, w, t, m, scale, label):
    print(f"# {label}: {tuple(h.shape)} x {tuple(w.shape)} {h.dtype} m={m}", flush=True)
    got = ops.head_score(h, w, t, m, scale)
    torch.cuda.synchronize()
    l = h.double() @ w.double().t() * scale
    lp, ent, norm, idx, top = ref.scores(l, t, m)
    e = _errors(h, w, scale)
    tol = 2 * e + 2.0 ** -20 + 2.0 ** -21 * float(l.abs().max())
    assert (got.logprob.double() - lp).abs().max() <= tol, label
    assert (got.entropy.double() - ent).abs().max() <= 2.0 ** -15 + 40 * e, label
    assert (got.norm.double() - norm).abs().max() <= tol, label
    if m:
        assert torch.equal(got.top_idx, idx), label
        assert (got.top_logprob.double() - top).abs().max() <= tol, label
    return got


SHAPES = [
    (1, 1, 1), (1, 3, 2), (2, 64, 64), (5, 100, 333), (16, 768, 1000), (17, 96, 1024),
    (64, 128, 4096), (65, 200, 129), (130, 7, 257), (300, 65, 128), (257, 320, 5000),
    (1000, 96, 1024),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,v", SHAPES + [(3700, 128, 3841)])
def test_scores(ops, n, d, v, dtype):
    h, w, t = _inputs(n, d, v, dtype, n + d + v)
    _check(ops, h, w, t, 0, 1.25, "scores")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,v", SHAPES)
def test_alternatives(ops, n, d, v, dtype):
    h, w, t = _inputs(n, d, v, dtype, n + d + v, grid=True)
    _check(ops, h, w, t, min(v, 5), 2.0, "alternatives")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_any_stride(ops, dtype):
    for off, d in ((0, 64), (1, 64), (8, 64), (3, 61), (0, 128)):
        h, w, t = _inputs(40, 150, 300, dtype, off + d, grid=True)
        for a in (h, w):
            keep = a[:, off:off + d].clone()
            a.fill_(float("nan"))
            a[:, off:off + d] = keep
        _check(ops, h[:, off:off + d], w[:, off:off + d], t, 3, 1.0, f"columns {off}+{d}")
        _check(ops, h[::2, off:off + d], w[:, off:off + d], t[::2].contiguous(), 0, 1.0, "every other row")
        hs, ws = h[::2, off:off + d], w[::3, off:off + d]
        _grad(ops, hs, ws, t[::2].clamp(max=99).contiguous(), 1.0)


def test_chunks_of_rows(ops):
    # many rows; then more rows than one chunk holds: statistics (5,376 rows of
    # 65,536 codes in 64 MiB), logits (1,024 in 256 MiB)
    h, w, t = _inputs(200_003, 64, 130, torch.bfloat16, 4)
    _check(ops, h, w, t, 0, 1.0, "chunks")
    h, w, t = _inputs(5700, 64, 65_536, torch.bfloat16, 14)
    _check(ops, h, w, t, 0, 1.0, "chunks of statistics")
    h, w, t = _inputs(2500, 64, 65_536, torch.bfloat16, 5, grid=True)
    _check(ops, h, w, t, 2, 1.0, "chunks of logits")


def test_extremes(ops):
    h, w, t = _inputs(20, 64, 200, torch.float32, 6)
    t[:3] = torch.tensor([-1, 200, 5], dtype=torch.int32)
    h[7], h[8, 3], h[9] = 0.0, float("nan"), 30.0 * h[9]
    t[7], t[8] = 3, 3
    got = ops.head_score(h, w, t, 2)
    assert got.logprob[0] == 0 and torch.isnan(got.logprob[1]) and torch.isnan(got.logprob[8])
    v = torch.tensor(200.0, dtype=torch.float64)
    assert abs(float(got.entropy[7] - v.log())) < 1e-5 and abs(float(got.logprob[7] + v.log())) < 1e-5
    assert got.top_idx[7].tolist() == [0, 1]  # all equal: the lowest indices
    lp, ent, _, _, _ = ref.scores(h.double() @ w.double().t(), t, 2)
    ok = torch.tensor([r for r in range(20) if r not in (1, 8)], device=DEV)
    e = _errors(h[ok], w, 1.0)
    assert (got.logprob.double() - lp)[ok].abs().max() <= 2 * e + 2.0 ** -12
    a = ops.head_score(h, w, t, 0)
    assert torch.isnan(a.logprob[1]) and torch.isnan(a.logprob[8]) and torch.isnan(a.entropy[8])
    assert (a.logprob.double() - lp)[ok].abs().max() <= 2 * e + 2.0 ** -12
    dh, dw = ops.head_score_backward(h, w, t, a.norm, a.entropy, torch.ones(20, device=DEV))
    assert torch.isnan(dh[1]).all() and torch.isnan(dh[8]).all() and torch.isnan(dw).all()
    assert dh[0].eq(0).all()  # no target, no entropy: no gradient
    e0 = ops.head_score(h[:0], w, t[:0], 2)
    assert e0.logprob.shape == (0,) and e0.top_idx.shape == (0, 2)
    dh, dw = ops.head_score_backward(h[:0], w, t[:0], e0.norm, e0.entropy, e0.logprob)
    assert dh.shape == (0, 64) and dw.eq(0).all()


def _grad(ops, h, w, t, scale):
    n, d = h.shape
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    gl, gh = torch.randn(2, n, generator=g, device=DEV)
    s = ops.head_score(h, w, t, 0, scale)
    dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, gl, gh, scale)
    torch.cuda.synchronize()
    hd, wd = h.double(), w.double()
    l = hd @ wd.t() * scale
    dx = ref.dlogits(l, t, gl, gh, scale)
    e = _errors(h, w, scale)
    low = h.dtype == torch.bfloat16
    # what dx may be off by, place by place
    p = torch.softmax(l, 1)
    size = scale * p * (gl.abs() + gh.abs() * (l.amax(1) - l.amin(1) + 20))[:, None].double()
    off = (4 * e + 2.0 ** -16) * size + (2.0 ** -10 if low else 2.0 ** -22) * dx.abs()
    sums = 2.0 ** -20
    th = off @ wd.abs() + sums * (dx.abs() @ wd.abs())
    tw = off.t() @ hd.abs() + sums * (dx.abs().t() @ hd.abs())
    wh, ww = dx @ wd, dx.t() @ hd
    if low:
        th, tw = th + 2.0 ** -8 * wh.abs(), tw + 2.0 ** -8 * ww.abs()
    assert bool(((dh.double() - wh).abs() <= 1.01 * th + 1e-12).all()), ((dh.double() - wh).abs() / th).max()
    assert bool(((dw.double() - ww).abs() <= 1.01 * tw + 1e-12).all()), ((dw.double() - ww).abs() / tw).max()
    return dh, dw


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,v", SHAPES)
def test_gradient(ops, n, d, v, dtype):
    h, w, t = _inputs(n, d, v, dtype, n + d + v)
    print(f"# gradient {n} x {d} x {v} {dtype}", flush=True)
    _grad(ops, h, w, t, 1.25)


def test_gradient_of_several_chunks(ops):
    # 512 MiB of dx: 4,096 rows of 65,536 codes in bf16, 1,280 in fp32
    h, w, t = _inputs(4500, 64, 65_536, torch.bfloat16, 8)
    _grad(ops, h, w, t, 1.0)
    h, w, t = _inputs(1500, 32, 65_536, torch.float32, 9)
    _grad(ops, h, w, t, 1.0)


def test_gradient_of_rows_with_nothing_left(ops):
    # a row whose norm says that nothing is left has no gradient, whatever arrives
    for dtype in (torch.float32, torch.bfloat16):
        h, w, t = _inputs(6, 64, 90, dtype, 16)
        t.clamp_(min=0)
        s = ops.head_score(h, w, t)
        g = torch.ones(6, device=DEV)
        a = ops.head_score_backward(h[:5], w, t[:5].contiguous(), s.norm[:5], s.entropy[:5].contiguous(),
                                    g[:5].contiguous(), g[:5].contiguous())
        s.norm[5, 0], s.norm[5, 1], s.entropy[5] = -INF, 0.0, 0.0
        dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, g, g)
        assert dh[5].eq(0).all() and torch.equal(dh[:5], a[0])
        # its row adds nothing to dw (the sums may be cut elsewhere: 2^-7 of the largest)
        assert (dw.float() - a[1].float()).abs().max() <= 2.0 ** -7 * a[1].float().abs().max()


def test_gradient_of_far_apart_magnitudes(ops):
    # rows whose gradients differ by 2^40, operands by 2^30: small rows of dh keep
    # their digits, and what dw loses is small beside its largest contributions
    h, w, t = _inputs(60, 64, 300, torch.bfloat16, 13)
    t.clamp_(min=0)
    h, w = h * 2.0 ** 20, w * 2.0 ** -22
    gl = 2.0 ** -torch.linspace(0, 40, 60, device=DEV)
    s = ops.head_score(h, w, t)
    dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, gl)
    dx = ref.dlogits(h.double() @ w.double().t(), t, gl, torch.zeros_like(gl), 1.0)
    wh, ww = dx @ w.double(), dx.t() @ h.double()
    th = 2.0 ** -10 * (dx.abs() @ w.double().abs()) + 2.0 ** -8 * wh.abs()
    assert bool(((dh.double() - wh).abs() <= 1.1 * th).all())
    tw = 2.0 ** -10 * (dx.abs().t() @ h.double().abs()) + 2.0 ** -8 * ww.abs()
    # what is dropped: 2^-39 of the largest dx, times h, in each of 60 rows
    tw += 60 * 2.0 ** -39 * float(dx.abs().max()) * float(h.abs().max())
    assert bool(((dw.double() - ww).abs() <= 1.1 * tw).all())


@pytest.mark.parametrize("e", [-115, 115])
def test_gradient_of_tiny_and_huge_operands(ops, e):
    # operands at the ends of the range whose products are ordinary; some codes and
    # rows are 0 (0 times the largest power of two stays 0)
    h, w, t = _inputs(33, 64, 100, torch.bfloat16, 15)
    t.clamp_(min=0)
    h, w = h * 2.0 ** e, w * 2.0 ** -e
    h[3], w[7] = 0.0, 0.0
    gl = torch.linspace(-1, 1, 33, device=DEV)
    gl[5] = 0.0
    s = ops.head_score(h, w, t)
    dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, gl)
    dx = ref.dlogits(h.double() @ w.double().t(), t, gl, torch.zeros_like(gl), 1.0)
    wh, ww = dx @ w.double(), dx.t() @ h.double()
    th = 2.0 ** -10 * (dx.abs() @ w.double().abs()) + 2.0 ** -8 * wh.abs()
    tw = 2.0 ** -10 * (dx.abs().t() @ h.double().abs()) + 2.0 ** -8 * ww.abs()
    assert dh[5].eq(0).all()
    assert bool(((dh.double() - wh).abs() <= 1.1 * th).all())
    assert bool(((dw.double() - ww).abs() <= 1.1 * tw).all())


def test_gradient_against_differences(ops):
    # float64 differences with a step of 1e-5: 1e-10 of curvature, 1e-6 of rounding
    h, w, t = _inputs(9, 20, 31, torch.float32, 10)
    dh, dw = _grad(ops, h, w, t, 0.75)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    gl, gh = torch.randn(2, 9, generator=g, device=DEV).double()

    def f(a, b):
        lp, ent, _, _, _ = ref.scores(a @ b.t() * 0.75, t, 0)
        return (gl * lp + gh * ent).sum()

    for k in range(3):
        u = torch.randn(9, 20, generator=g, device=DEV).double()
        z = torch.randn(31, 20, generator=g, device=DEV).double()
        e = 1e-5
        num = (f(h.double() + e * u, w.double() + e * z) - f(h.double() - e * u, w.double() - e * z)) / (2 * e)
        got = (dh.double() * u).sum() + (dw.double() * z).sum()
        size = (dh.double() * u).abs().sum() + (dw.double() * z).abs().sum()
        assert abs(float(num - got)) <= 1e-4 * float(size)


def test_another_stream_and_repeatable(ops):
    h, w, t = _inputs(500, 96, 3000, torch.bfloat16, 12)
    a = ops.head_score(h, w, t, 4)
    ga = ops.head_score_backward(h, w, t, a.norm, a.entropy, a.logprob, a.entropy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = ops.head_score(h, w, t, 4)
        gb = ops.head_score_backward(h, w, t, b.norm, b.entropy, b.logprob, b.entropy)
    side.synchronize()
    for p, q in zip(tuple(a) + ga, tuple(b) + gb):
        assert torch.equal(p, q)


def test_refusals(ops):
    h, w, t = _inputs(4, 32, 40, torch.float32, 1)
    with pytest.raises(ValueError):
        ops.head_score(h, w[:, :31], t)
    with pytest.raises(ValueError):
        ops.head_score(h, w.bfloat16(), t)
    with pytest.raises(ValueError):
        ops.head_score(h, w.cpu(), t)
    with pytest.raises(TypeError):
        ops.head_score(h.half(), w.half(), t)
    with pytest.raises(ValueError):
        ops.head_score(h, w, t.float())
    for m in (-1, 17):
        with pytest.raises(ops.GmmError):
            ops.head_score(h, w, t, m)
    with pytest.raises(ops.GmmError):
        ops.head_score(h, w, t, 0, 0.0)
    with pytest.raises(ops.GmmError):
        ops.head_score(h, w, t, ws=torch.empty(8, dtype=torch.uint8, device=DEV))
    s = ops.head_score(h, w, t)
    with pytest.raises(ops.GmmError):
        ops.head_score_backward(h, w, t, s.norm, None, s.logprob, s.logprob)
    with pytest.raises(ValueError):
        ops.head_score_backward(h, w, t, s.norm.t(), s.entropy, s.logprob)
