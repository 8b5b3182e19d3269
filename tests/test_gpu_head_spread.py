"""Gradients of bf16 heads whose dims, rows and gradients are far apart in magnitude.

fp16 holds the operands of the gradients' products, with powers of two that are taken out of
the sums again: for W one per dim, for h one per dim after the rows' gradients are multiplied
in, for dx one per row. So dims may lie anywhere, and rows of h may be as large as
their gradients are small. Allowed, as for ordinary magnitudes: the logits' E = 2^-24 (d / 4 + 16)
max sum |h w| and 2^-16 in p, dx to 2^-10, place by place, a bf16 result's 2^-8 of itself, and 2^-39 of
the largest |W| of the dim, |h| g of the dim and g of the row, which is where fp16 ends.
"""
import pytest

torch = pytest.importorskip("torch")

from tests import nn_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _inputs(n, d, v, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.randn(n, d, generator=g, device=DEV)
    w = torch.randn(v, d, generator=g, device=DEV) * 2 / d ** 0.5
    t = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    return h, w, t


def _check(ops, h, w, t, gl, rows=None):
    """rows: those that have a gradient (all)."""
    h, w = h.bfloat16(), w.bfloat16()
    s = ops.head_score(h, w, t)
    dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, gl)
    rows = slice(None) if rows is None else rows
    hd, wd = h.double()[rows], w.double()
    # from the kernel's own norm, whose error is the scores' matter
    lp = hd @ wd.t() - s.norm[rows].double().sum(1)[:, None]
    hot = torch.zeros_like(lp)
    hot.scatter_(1, t[rows].long()[:, None], 1.0)
    gd = gl[rows].double().abs()[:, None]
    dx = gl[rows].double()[:, None] * (hot - lp.exp())
    wh, ww = dx @ wd, dx.t() @ hd
    e = 2.0 ** -24 * (h.shape[1] / 4 + 16) * float((hd.abs() @ wd.abs().t()).max())
    off = 2.0 ** -10 * dx.abs() + (2 * e + 2.0 ** -16) * lp.exp() * gd
    th = (off + 2.0 ** -39 * gd) @ wd.abs() + 2.0 ** -8 * wh.abs()
    th += 2.0 ** -39 * dx.abs().sum(1, keepdim=True) * wd.abs().amax(0)
    tw = (off + 2.0 ** -39 * gd).t() @ hd.abs() + 2.0 ** -8 * ww.abs()
    tw += 2.0 ** -39 * (hot + lp.exp()).sum(0)[:, None] * (gd * hd.abs()).amax(0)
    tiny = 2.0 ** -126  # below it a bf16 result has fewer digits
    assert bool(((dh[rows].double() - wh).abs() <= 1.1 * th + tiny).all()), ((dh[rows].double() - wh).abs() / th).max()
    assert bool(((dw.double() - ww).abs() <= 1.1 * tw + tiny).all()), ((dw.double() - ww).abs() / tw).max()
    return dh, dw


@pytest.mark.parametrize("n,d,v", [(33, 64, 100), (70, 100, 333), (257, 256, 1000), (5, 8, 70)])
def test_dims_far_apart(ops, n, d, v):
    h, w, t = _inputs(n, d, v, n)
    e = torch.linspace(-60, 0, d, device=DEV).round()
    print(f"# {n} x {d} x {v}", flush=True)
    gl = torch.linspace(-1, 1, n, device=DEV) + 0.01
    _check(ops, h, w * 2.0 ** e, t, gl)               # columns of W
    _check(ops, h * 2.0 ** e, w, t, gl)               # columns of h
    _check(ops, h * 2.0 ** -e, w * 2.0 ** e, t, gl)   # both, with ordinary logits
    w[:, d // 2] = 0.0
    h[:, d // 3] = 0.0
    dh, dw = _check(ops, h, w, t, gl)
    assert dh[:, d // 2].eq(0).all() and dw[:, d // 3].eq(0).all()


@pytest.mark.parametrize("n,d,v", [(33, 64, 100), (300, 100, 333)])
def test_large_rows_of_small_gradients(ops, n, d, v):
    h, w, t = _inputs(n, d, v, n)
    e = (torch.arange(n, device=DEV) % 46).float()
    # rows up to 2^45 with logits of ordinary size: what they multiply in W is small
    h[:, d // 2:] *= 2.0 ** e[:, None]
    w[:, d // 2:] *= 2.0 ** -50
    print(f"# {n} x {d} x {v}", flush=True)
    _check(ops, h, w, t, 2.0 ** -e)


def test_rows_without_gradient_do_not_count(ops):
    # padding: no target, no gradient, and whatever the memory held
    h, w, t = _inputs(40, 64, 200, 3)
    gl = torch.ones(40, device=DEV)
    pad = torch.arange(40, device=DEV) % 3 == 0
    h[pad] *= 2.0 ** 90
    t[pad] = -1
    dh, _ = _check(ops, h, w, t, gl, ~pad)
    assert dh[pad].eq(0).all()
