"""Logits of -inf in a head: masked codes, wherever they lie and however they are scored.

They come from a weight of -inf or from a product beyond fp32. Such a code has probability
0: the scores are those of the other codes (float64 of them; logits here are below 8, so
that log p is within 2^-18 and the entropy within 2^-15), and no gradient passes. A row of
nothing else has norm (-inf, 0). NaN and +inf give NaN, an infinity in an fp32 operand counts as NaN.
"""
import pytest

torch = pytest.importorskip("torch")

from tests import nn_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")
V = 5000
PLACES = [0, 700, 4607, 4999]  # in whole tiles of codes, and in the last one


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _inputs(n, dtype, seed):
    """Grid values whose sums are exact; dim 0 of h is 1 and of w is 0."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.randint(-2, 3, (n, 4), generator=g, device=DEV).float() / 2
    w = torch.randint(-8, 9, (V, 4), generator=g, device=DEV).float() / 8
    h[:, 0], w[:, 0] = 1.0, 0.0
    t = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    return h.to(dtype), w.to(dtype), t


def _check(ops, h, w, t, l, m):
    s = ops.head_score(h, w, t, m)
    lp, ent, norm, idx, top = ref.scores(l, t, m)

    def close(a, b, tol):
        a = a.double()
        same = (a == b) | (torch.isnan(a) & torch.isnan(b))
        assert bool((same | ((a - b).abs() <= tol)).all()), (a, b)

    close(s.logprob, lp, 2.0 ** -18)
    close(s.entropy, ent, 2.0 ** -15)
    close(s.norm, norm, 2.0 ** -18)
    if m:
        keep = ~torch.isnan(norm[:, 0])
        assert torch.equal(s.top_idx[keep], idx[keep])
        close(s.top_logprob[keep], top[keep], 2.0 ** -18)
    return s


@pytest.mark.parametrize("n", [4, 70, 300])
@pytest.mark.parametrize("m", [0, 3])
@pytest.mark.parametrize("at", PLACES)
def test_weights_of_minus_infinity(ops, n, m, at):
    h, w, t = _inputs(n, torch.bfloat16, n + at)
    w[at, 0] = -INF
    t[1] = at
    print(f"# n={n} m={m} at={at}", flush=True)
    l = h[:, 1:].double() @ w[:, 1:].double().t()
    l[:, at] = -INF
    s = _check(ops, h, w, t, l, m)
    assert s.logprob[1] == -INF
    # +inf and NaN: the whole row
    for bad in (INF, float("nan")):
        w[at, 0] = bad
        l[:, at] = bad
        _check(ops, h, w, t, l, m)


@pytest.mark.parametrize("at", PLACES)
def test_infinite_fp32_weights(ops, at):
    # with and without low bits in the row that meets the infinity
    h, w, t = _inputs(70, torch.float32, at)
    h[::2, 0] = 1 + 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -18 + 2.0 ** -21
    h[1::6, 0] = -h[0, 0]
    print(f"# at={at}", flush=True)
    for bad in (INF, -INF, float("nan")):
        w[at, 0] = bad
        for m in (0, 3):
            s = ops.head_score(h, w, t, m)
            assert torch.isnan(s.norm).all() and torch.isnan(s.entropy).all()
            assert torch.isnan(s.logprob).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [4, 70, 300])
@pytest.mark.parametrize("at", PLACES)
def test_products_beyond_the_range(ops, dtype, n, at):
    h, w, t = _inputs(n, dtype, n + at)
    h[2, 0] = 2.0 ** 100   # only this row's product with the code overflows
    h[0, 0] = 0.0
    w[at, 0] = -2.0 ** 100
    t[2], t[3], t[0] = at, at, at
    print(f"# n={n} {dtype} at={at}", flush=True)
    l = h.double() @ w.double().t()
    l[2, at] = -INF
    for m in (0, 3):
        s = _check(ops, h, w, t, l, m)
        assert s.logprob[2] == -INF
    g = torch.ones(n, device=DEV)
    for gh in (None, 0.5 * g):
        dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, g, gh)
        assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
        if dtype == torch.float32:
            dx = ref.dlogits(l, t, g, torch.zeros_like(g) if gh is None else gh, 1.0)
            # logits and dx to 2^-16 of dx's parts, fp32 sums
            size = 2.0 ** -15 * (dx.abs() + torch.softmax(l, 1) * 16)
            assert bool(((dh.double() - dx @ w.double()).abs() <= size @ w.double().abs()).all())
            assert bool(((dw.double() - dx.t() @ h.double()).abs() <= size.t() @ h.double().abs()).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [4, 70, 300])
def test_rows_that_are_masked_whole(ops, dtype, n):
    h, w, t = _inputs(n, dtype, n)
    w[:, 0] = -2.0 ** 100
    h[:, 0] = 0.0
    h[2, 0] = 2.0 ** 100
    print(f"# n={n} {dtype}", flush=True)
    l = h.double() @ w.double().t()
    l[2] = -INF
    for m in (0, 3):
        s = _check(ops, h, w, t, l, m)
        assert s.norm[2].tolist() == [-INF, 0.0] and s.logprob[2] == -INF and s.entropy[2] == 0
        if m:
            assert s.top_idx[2].eq(-1).all()
    g = torch.ones(n, device=DEV)
    for gh in (None, g):
        dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, g, gh)
        assert dh[2].eq(0).all() and torch.isfinite(dh).all() and torch.isfinite(dw).all()
