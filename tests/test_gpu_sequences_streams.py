"""The operators for sequences of codes run on the caller's stream, in its order.

On a stream of its own a long operation is queued, then a copy that overwrites an operand, then the call:
launched anywhere else it would read what was there before. The result must be that of the
new operand, bit for bit, and another one than that of the old.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for t in r if isinstance(t, torch.Tensor)]


def _check(old, new, call):
    """call(x) with an x that holds old, and new once the stream has got there."""
    want_old, want = (_flat(call(t.clone())) for t in (old, new))  # a call may write its operand
    assert any(not torch.equal(a, b) for a, b in zip(want_old, want))
    ballast = torch.zeros(1 << 28, device=DEV)  # 1 GB
    side = torch.cuda.Stream()
    done = torch.cuda.Event()
    late = False
    for _ in range(3):  # an allocation may have made the host wait
        x = old.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                ballast.add_(1.0)
            x.copy_(new)
            got = _flat(call(x))
            done.record()
        late = not done.query()  # the call was made while the copy was still to come
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        if late:
            break
    assert late


def test_embed(ops):
    g = _gen(1)
    codes = torch.randint(-1, 50, (3000,), generator=g, device=DEV, dtype=torch.int32)
    table = torch.randn(50, 96, generator=g, device=DEV)
    _check(table, -table, lambda t: ops.embed(t, codes))


@pytest.mark.parametrize("n", [0, 500, 3000, 20_000])
def test_embed_backward(ops, n):
    g = _gen(2)
    codes = torch.randint(-1, 50, (n,), generator=g, device=DEV, dtype=torch.int32)
    grad = torch.randn(n, 96, generator=g, device=DEV)
    if n:
        _check(grad, grad + 1.0, lambda t: ops.embed_backward(t, codes, 50))
        return
    # nothing to read: the zeros come after what was written before
    _check(torch.zeros(50, 96, device=DEV), torch.ones(50, 96, device=DEV),
           lambda t: [t.clone(), ops.embed_backward(grad, codes, 50, out=t).clone()])


def test_quantize_rows(ops):
    x = torch.randn(300, 200, generator=_gen(3), device=DEV)
    _check(x, 2.0 * x, ops.quantize_rows)


@pytest.mark.parametrize("n,d,v", [(5, 200, 500), (40, 4999, 200), (300, 203, 500), (300, 256, 500), (128, 8192, 4096)])
def test_quantized_product(ops, n, d, v):
    g = _gen(4)
    q = torch.randint(-127, 128, (n, d), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (v, d), generator=g, device=DEV, dtype=torch.int8)
    one_q, one_w = torch.ones(n, device=DEV), torch.ones(v, device=DEV)
    _check(q, -q, lambda t: ops.quantized_product(t, one_q, w, one_w))
    _check(w, -w, lambda t: ops.quantized_product(q, one_q, t, one_w))


@pytest.mark.parametrize("b,w,v", [(7, 5, 1000), (4, 1, 1000), (2, 1, 200_000)])
def test_beam_step(ops, b, w, v):
    g = _gen(5)
    logits = torch.randn(b * w, v, generator=g, device=DEV)
    scores = -torch.rand(b, w, generator=g, device=DEV)
    last = torch.full((b, w), 3, dtype=torch.int32, device=DEV)
    _check(logits, -logits, lambda t: ops.beam_step(t, scores, last, 1, 4))


def test_beam_reorder(ops):
    g = _gen(6)
    state = torch.randn(20, 333, generator=g, device=DEV)
    parent = torch.randint(0, 4, (5, 4), generator=g, device=DEV, dtype=torch.int32)
    _check(state, -state, lambda t: ops.beam_reorder(t, parent, 4))
    _check(parent, (parent + 1) % 4, lambda t: ops.beam_reorder(state, t, 4))
    _check(state, -state, lambda t: ops.beam_reorder(t, parent, 4, out=t))  # in place


def test_balance(ops):
    g = _gen(7)
    z = torch.randn(5000, 60, generator=g, device=DEV)
    idx = torch.randint(0, 60, (5000, 2), generator=g, device=DEV, dtype=torch.int32)
    _check(z, -z, lambda t: ops.balance_loss(t, idx))
    r = ops.balance_loss(z, idx)
    dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm)
    assert dz.abs().sum() > 0
    one = torch.ones((), device=DEV)
    _check(one, 3.0 * one, lambda t: ops.balance_loss_backward(z, r.counts, r.totals, r.norm, t))
