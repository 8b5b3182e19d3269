"""Mixture-of-experts layer against a plain float64 form.

Rows and gates lie on a grid, so that the gate's sums are exact and the picks and
their order have to be the same, ties included. Tolerances, set before the first run:
shares within 2^-20 (|z| < 32: 2^-24 of it, and the exponential). y: the fp32 sums of the
first product are off by 2^-24 (d / 4 + 16) of their sums of magnitudes and pass
through silu(a) b, whose slope is below 1.1 |b| and |a| + 1; the features are then held to 2^-16 (bf16) or
2^-24 (fp32), and summed with 2^-24 (f / 4 + 16); a bf16 result adds 2^-8 of itself.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _inputs(n, d, f, e, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device=DEV)

    x = (normal(n, d) * 8).round().clamp(-31, 31) / 8
    gate = (normal(e, d) * 4).round().clamp(-15, 15) / 4 / 2.0 ** max(0, (d.bit_length() - 1) // 2)
    return (x.to(dtype), gate.to(dtype), (normal(e, 2 * f, d) / d ** 0.5).to(dtype),
            (normal(e, d, f) / f ** 0.5).to(dtype))


def _reference(x, w_in, w_out, idx, resp):
    """y and what it may be off by, for the given picks."""
    n, d = x.shape
    e, _, f = w_out.shape
    low = x.dtype == torch.bfloat16
    xd = x.double()
    y = torch.zeros(n, d, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(y)
    for c in range(e):
        for j in range(idx.shape[1]):
            t = (idx[:, j] == c).nonzero()[:, 0]
            if not len(t):
                continue
            wi, wo, r = w_in[c].double(), w_out[c].double(), resp[t, j].double()[:, None]
            h = xd[t] @ wi.t()
            size = xd[t].abs() @ wi.abs().t() * 2.0 ** -24 * (d / 4 + 16)
            a, b = h[:, :f], h[:, f:]
            act = a * torch.sigmoid(a) * b
            off = size[:, :f] * 1.1 * b.abs() + size[:, f:] * (a.abs() + 1)
            off += act.abs() * (2.0 ** -16 if low else 2.0 ** -21)
            y[t] += r * (act @ wo.t())
            tol[t] += r.abs() * (off @ wo.abs().t() + act.abs() @ wo.abs().t() * 2.0 ** -24 * (f / 4 + 16))
    return y, tol + (2.0 ** -8 if low else 2.0 ** -22) * y.abs()


def _check(ops, n, d, f, e, m, dtype, share_all=False, seed=0):
    print(f"# moe n={n} d={d} f={f} e={e} m={m} {dtype}", flush=True)
    x, gate, w_in, w_out = _inputs(n, d, f, e, dtype, seed + n + d + f + e)
    y, idx, resp = ops.moe_layer(x, w_in, w_out, gate, m, share_all)
    torch.cuda.synchronize()
    z = x.double() @ gate.double().t()
    val, want = z.sort(dim=1, descending=True, stable=True)
    assert torch.equal(idx, want[:, :m].to(torch.int32))
    share = torch.softmax(z, 1).gather(1, want)[:, :m] if share_all else torch.softmax(val[:, :m], 1)
    assert (resp.double() - share).abs().max() <= 2.0 ** -20
    ref, tol = _reference(x, w_in, w_out, idx, resp)
    assert bool(((y.double() - ref).abs() <= tol + 1e-12).all()), ((y.double() - ref).abs() / tol).max()
    return x, gate, w_in, w_out, y, idx, resp


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,f,e,m", [
    (1, 1, 1, 1, 1), (1, 768, 256, 64, 2), (2, 96, 128, 8, 8), (3, 33, 17, 5, 3), (5, 100, 200, 7, 1),
    (16, 128, 64, 4, 2), (17, 64, 100, 2, 1), (40, 96, 33, 3, 2), (64, 256, 96, 16, 4),
    (130, 65, 48, 2, 2), (700, 32, 16, 5, 4), (9, 1030, 70, 300, 16),
])
def test_layer(ops, n, d, f, e, m, dtype):
    _check(ops, n, d, f, e, m, dtype)
    _check(ops, n, d, f, e, m, dtype, share_all=True, seed=1)


def test_many_pairs(ops):
    # more pairs than one window holds, and many rows of one expert
    _check(ops, 3000, 16, 32, 3, 3, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_given_picks(ops, dtype):
    x, gate, w_in, w_out = _inputs(20, 48, 40, 6, dtype, 3)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    idx = torch.randint(0, 6, (20, 3), generator=g, device=DEV, dtype=torch.int32)  # repeats among them
    resp = torch.randn(20, 3, generator=g, device=DEV)
    idx[2] = -1                       # nothing picked
    idx[3, 1], idx[4, 0] = 6, -5      # outside
    for rows in (20, 1, 5):
        y, i2, r2 = ops.moe_layer(x[:rows], w_in, w_out, idx=idx[:rows], resp=resp[:rows])
        assert torch.equal(i2, idx[:rows]) and torch.equal(r2, resp[:rows])
        ref, tol = _reference(x[:rows], w_in, w_out, idx[:rows], resp[:rows])
        assert bool(((y.double() - ref).abs() <= tol + 1e-12).all())
        if rows > 2:
            assert y[2].eq(0).all()


def test_ties_nan_and_strides(ops):
    x, gate, w_in, w_out = _inputs(12, 40, 24, 9, torch.float32, 5)
    gate[:] = gate[0]                  # all gates equal: the lowest indices
    gate[7] = gate[7] + 0.0
    y, idx, resp = ops.moe_layer(x, w_in, w_out, gate, 3)
    assert torch.equal(idx, torch.arange(3, device=DEV, dtype=torch.int32).expand(12, 3))
    assert (resp - 1 / 3).abs().max() < 1e-6
    x[4, 2] = float("nan")
    y2, idx2, resp2 = ops.moe_layer(x, w_in, w_out, gate, 3)
    assert torch.isnan(y2[4]).all() and torch.isnan(resp2[4]).all()
    keep = torch.arange(12, device=DEV) != 4
    assert torch.equal(y2[keep], y[keep])
    wide = torch.full((12, 45), float("nan"), device=DEV)
    wide[:, 3:43] = x
    y3, _, _ = ops.moe_layer(wide[:, 3:43], w_in, w_out, gate, 3)
    assert torch.equal(y3[keep], y[keep])
    e = ops.moe_layer(x[:0], w_in, w_out, gate, 3)
    assert e[0].shape == (0, 40) and e[1].shape == (0, 3)


def test_another_stream_and_repeatable(ops):
    x, gate, w_in, w_out = _inputs(50, 256, 200, 16, torch.bfloat16, 6)
    a = ops.moe_layer(x, w_in, w_out, gate, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = ops.moe_layer(x, w_in, w_out, gate, 4)
    side.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_refusals(ops):
    x, gate, w_in, w_out = _inputs(4, 32, 16, 5, torch.float32, 7)
    idx = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    resp = torch.ones((4, 2), device=DEV)
    for bad in (dict(gate=None), dict(gate=gate, idx=idx, resp=resp), dict(gate=None, idx=idx),
                dict(gate=gate[:, :31]), dict(gate=gate.bfloat16()), dict(gate=None, idx=idx.long(), resp=resp),
                dict(gate=None, idx=idx[:3], resp=resp[:3])):
        with pytest.raises(ValueError):
            ops.moe_layer(x, w_in, w_out, **bad)
    for m in (0, 6, 17):
        with pytest.raises(ops.GmmError):
            ops.moe_layer(x, w_in, w_out, gate, m)
    with pytest.raises(ValueError):
        ops.moe_layer(x, w_in[:, :31], w_out, gate, 2)
    with pytest.raises(ValueError):
        ops.moe_layer(x, w_in, w_out.transpose(1, 2).contiguous().transpose(1, 2), gate, 2)
    with pytest.raises(TypeError):
        ops.moe_layer(x.half(), w_in, w_out, gate, 2)
    with pytest.raises(ops.GmmError):
        ops.moe_layer(x, w_in, w_out, gate, 2, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
