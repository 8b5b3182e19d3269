"""Balance loss of a router and its gradient against plain float64 forms.

Tolerances, set before the first run, relative to p: an exponential of d < 0 is off by
2^-24 (1.5 |d| + 4), the row's sum by 2^-24 (E / 16 + 16), its reciprocal or logarithm by a few 2^-24
more (the logarithm's own size times 2^-24 in the gradient): r = 2^-24 (2.5 D + E / 8 + 32) with D the
largest |d| of a row. Sums over rows add 2^-24 (n / 64 + 64); the loss, a product of
exact counts and prob, 2^-24 E / 16 + 16 more. The gradient is g E / N p (f - s): r on p, r s + 2^-22 on s
and f, and its own rounding.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _plain(z, idx):
    """(loss, counts, totals, prob, p, f, live) in float64."""
    z = z.double()
    e = z.shape[1]
    ok = (idx >= 0) & (idx < e)
    live = ok.any(1)
    counts = torch.bincount(idx[ok].long(), minlength=e)
    empty = (z == -INF).all(1)
    p = torch.softmax(z, 1)
    p[empty] = 0.0
    p[~live] = 0.0
    rows, picks = int(live.sum()), int(counts.sum())
    prob = p.sum(0) / max(rows, 1)
    f = counts.double() / max(picks, 1)
    return e * (f * prob).sum(), counts, (rows, picks), prob, p, f, live


def _check(ops, z, idx, g=0.7, out=None):
    n, e = z.shape
    r = ops.balance_loss(z, idx)
    loss, counts, totals, prob, p, f, live = _plain(z, idx)
    assert torch.equal(r.counts, counts.to(torch.int32)) and tuple(r.totals.tolist()) == totals
    zd = z.double()
    d = (zd.amax(1, keepdim=True) - zd)
    d = d[torch.isfinite(d) & (p > 0)]
    far = float(d.max()) if d.numel() else 0.0
    rel = 2.0 ** -24 * (2.5 * min(far, 104.0) + e / 8 + 32)
    rows = rel + 2.0 ** -24 * (n / 64 + 64)
    assert bool(((r.prob.double() - prob).abs() <= rows * prob + 1e-37).all())
    assert abs(r.loss.double() - loss) <= (rows + 2.0 ** -24 * (e / 16 + 16)) * loss + 1e-37
    gl = torch.tensor(g, device=DEV)
    dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm, gl, out=out)
    by = abs(float(gl.double())) * e / max(totals[0], 1)
    s = p @ f[:, None]
    ref = float(gl.double()) * e / max(totals[0], 1) * p * (f - s)
    tol = by * p * (rel * (f - s).abs() + (rel + 2.0 ** -22) * (s + f)) + 2.0 ** -22 * ref.abs() + 1e-37
    if z.dtype == BF16:
        tol += 2.0 ** -8 * ref.abs()
    assert dz.dtype == z.dtype and bool(((dz.double() - ref).abs() <= tol).all()), \
        ((dz.double() - ref).abs() / tol).max()
    assert dz[~live].eq(0).all()
    return r, dz


def _inputs(n, e, m, dtype, seed):
    g = _gen(seed)
    z = (2 * torch.randn(n, e, generator=g, device=DEV) + torch.randn(e, generator=g, device=DEV)).to(dtype)
    idx = z.float().topk(m, 1).indices.to(torch.int32)
    idx[torch.rand(n, generator=g, device=DEV) < 0.2] = -1
    return z, idx


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,e,m", [(1, 1, 1), (2, 3, 2), (5, 64, 4), (100, 65, 2), (333, 60, 2), (17, 128, 16),
                                   (70, 129, 3), (1000, 256, 8), (40, 257, 1), (33, 513, 5), (300, 1000, 2),
                                   (20, 1025, 2), (9, 4096, 16), (50_001, 16, 2), (8200, 60, 9), (8301, 100, 2),
                                   (8200, 200, 3), (8203, 400, 2), (8200, 1500, 2), (1_000_001, 8, 1)])
def test_loss_and_gradient(ops, n, e, m, dtype):
    print(f"# balance n={n} e={e} m={m} {dtype}", flush=True)
    z, idx = _inputs(n, e, min(m, e), dtype, n + e + m)
    a, da = _check(ops, z, idx)
    b = ops.balance_loss(z, idx)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(da, ops.balance_loss_backward(z, b.counts, b.totals, b.norm, torch.tensor(0.7, device=DEV)))


def test_balanced_is_one(ops):
    z = torch.zeros(64, 8, device=DEV)
    idx = torch.arange(64, device=DEV, dtype=torch.int32)[:, None] % 8
    r = ops.balance_loss(z, idx.contiguous())
    assert abs(float(r.loss) - 1.0) < 1e-6
    d = ops.balance_loss_backward(z, r.counts, r.totals, r.norm)
    assert d.abs().max() <= 2.0 ** -22 / 64


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masks(ops, dtype):
    z, idx = _inputs(60, 70, 3, dtype, 3)
    z[torch.rand(60, 70, generator=_gen(4), device=DEV) < 0.5] = -INF
    z[5] = -INF                        # a live row without a number
    idx[5] = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)
    z[6] = torch.finfo(dtype).min      # masked with the lowest value: even shares
    idx[6, 0] = 9
    z[7, 1:] = -INF                    # one expert left
    idx[8] = torch.tensor([70, -5, 2 ** 31 - 1], dtype=torch.int32, device=DEV)  # none of them an expert
    idx[9] = torch.tensor([4, -1, 4], dtype=torch.int32, device=DEV)             # the same one twice
    z[10], idx[10] = float("nan"), -1  # padding may hold anything
    z[11, 3], idx[11] = INF, -1
    keep = torch.ones(60, dtype=torch.bool, device=DEV)
    keep[10:12] = False
    r = ops.balance_loss(z, idx)
    want = ops.balance_loss(z[keep].contiguous(), idx[keep].contiguous())
    assert torch.equal(r.counts, want.counts) and torch.equal(r.totals, want.totals)
    assert torch.isfinite(r.loss) and abs(float(r.loss - want.loss)) <= 1e-5
    z2 = z.clone()
    z2[10:12] = 0
    _check(ops, z2, idx)
    dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm)
    assert dz[10:12].eq(0).all() and dz[5].eq(0).all() and torch.isfinite(dz).all()
    assert r.norm[10].tolist() == [INF, 0.0] and r.norm[5].tolist() == [-INF, 0.0]
    z[20, 1], idx[20] = float("nan"), 0
    r = ops.balance_loss(z, idx)
    assert torch.isnan(r.loss) and torch.isnan(r.prob).all()
    dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm)
    assert torch.isnan(dz[20]).all() and torch.isfinite(dz[:20]).all() and torch.isfinite(dz[21:]).all()


def test_nothing_routed(ops):
    z, idx = _inputs(30, 9, 2, F32, 5)
    idx[:] = -1
    for rows in (30, 0):
        r = ops.balance_loss(z[:rows], idx[:rows])
        assert r.loss == 0 and r.counts.eq(0).all() and r.prob.eq(0).all() and r.totals.tolist() == [0, 0]
        assert ops.balance_loss_backward(z[:rows], r.counts, r.totals, r.norm).eq(0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("e", [5, 37, 300])
def test_strides_and_in_place(ops, e, dtype):
    z, idx = _inputs(44, e, 2, dtype, 6)
    wide = torch.full((44, e + 9), float("nan"), dtype=dtype, device=DEV)
    wide[:, 3:3 + e] = z
    a, da = _check(ops, z, idx)
    out = torch.full((44, e + 5), 3.0, dtype=dtype, device=DEV)
    b, db = _check(ops, wide[:, 3:3 + e], idx, out=out[:, 1:1 + e])
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(da, db)
    assert out[:, 0].eq(3).all() and out[:, 1 + e:].eq(3).all()
    ops.balance_loss_backward(wide[:, 3:3 + e], a.counts, a.totals, a.norm, torch.tensor(0.7, device=DEV),
                              out=wide[:, 3:3 + e])
    assert torch.equal(wide[:, 3:3 + e], da)
    assert torch.isnan(wide[:, :3]).all() and torch.isnan(wide[:, 3 + e:]).all()


def test_gradient_against_differences(ops):
    z, idx = _inputs(50, 12, 2, F32, 7)
    turn = torch.randn(50, 12, generator=_gen(8), device=DEV).double()
    r = ops.balance_loss(z, idx)
    dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm).double()
    h = 1e-5
    change = (_plain(z.double() + h * turn, idx)[0] - _plain(z.double() - h * turn, idx)[0]) / (2 * h)
    # h^2 times a third derivative below E per unit step, and the kernel's 2^-18 of the terms
    assert abs(change - (dz * turn).sum()) <= 1e-8 + 2.0 ** -18 * (dz * turn).abs().sum()


def test_picks_of_the_library(ops):
    # the layer's own picks, with its gate's logits
    g = _gen(9)
    x = torch.randn(40, 32, generator=g, device=DEV)
    gate = torch.randn(7, 32, generator=g, device=DEV)
    w_in = torch.randn(7, 16, 32, generator=g, device=DEV)
    w_out = torch.randn(7, 32, 8, generator=g, device=DEV)
    _, idx, _ = ops.moe_layer(x, w_in, w_out, gate, 2)
    _check(ops, x @ gate.t(), idx)


def test_another_stream(ops):
    z, idx = _inputs(3000, 64, 4, BF16, 10)
    a = ops.balance_loss(z, idx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = ops.balance_loss(z, idx)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(ops):
    z, idx = _inputs(10, 6, 2, F32, 11)
    for bad in (idx.long(), idx[:9], idx[:, 0], idx.t(), idx.cpu()):
        with pytest.raises(ValueError):
            ops.balance_loss(z, bad)
    with pytest.raises(TypeError):
        ops.balance_loss(z.double(), idx)
    for m in (0, 17):
        with pytest.raises(ops.GmmError):
            ops.balance_loss(z, torch.zeros(10, m, dtype=torch.int32, device=DEV))
    with pytest.raises(ops.GmmError):
        ops.balance_loss(torch.zeros(1, 4097, device=DEV), idx[:1].contiguous())
    with pytest.raises(ops.GmmError):
        ops.balance_loss(z, idx, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
    r = ops.balance_loss(z, idx)
    for kw in (dict(counts=r.counts[:5]), dict(totals=r.totals.int()), dict(norm=r.norm[:9]),
               dict(g_loss=torch.ones(2, device=DEV)), dict(g_loss=torch.ones((), device=DEV).double()),
               dict(out=z.bfloat16())):
        a = dict(counts=r.counts, totals=r.totals, norm=r.norm) | kw
        with pytest.raises(ValueError):
            ops.balance_loss_backward(z, **a)
