"""Single products of fp32 operands in a head, where their low bits are largest.

Three bf16 planes carry an fp32 operand. Rounded to nearest, the second is at most 2^-8 and the
third 2^-17 of an operand in [1, 2): the products left out (second by third, third by third)
are below 2^-24 of the product. The six that are kept are added in fp32, smallest
first: 2^-24 for each of the last additions. 2^-22 is allowed in all.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def test_single_products(ops):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    step = 2.0 ** -23
    worst = [1 + 2.0 ** -7 - step, 1 + 2.0 ** -8 - step, 1 + 2.0 ** -8 + step, 1 + 2.0 ** -8,
             1 + 2.0 ** -7 - 2.0 ** -15 - step, 1 + 2.0 ** -8 + 2.0 ** -16 - step, 2 - step, 1 + step,
             -1 - 2.0 ** -7 + step, 1e-30 * (1 + 2.0 ** -7), 3.4e38, -3.4e38]
    h = 1 + torch.rand(4096, generator=g, device=DEV)
    h[:len(worst)] = torch.tensor(worst, device=DEV)
    for y in worst[:9]:
        w = torch.tensor([[y]], device=DEV) * 0.5  # keeps 3.4e38 within the range
        got = ops.head_score(h[:, None], w).norm[:, 0].double()
        want = h.double() * w.double()[0, 0]
        err = ((got - want).abs() / want.abs()).max()
        assert err <= 2.0 ** -22, (y, float(err.log2()))


def test_products_of_gradients(ops):
    # one row, two codes: dx is one number and its negative, dh = dx w, dw = dx h
    step = 2.0 ** -23
    values = torch.tensor([1 + 2.0 ** -7 - step, 1 + 2.0 ** -8 - step, 2 - step, 1 + 2.0 ** -8 + step],
                          device=DEV)
    t = torch.zeros(1, dtype=torch.int32, device=DEV)
    norm = torch.tensor([[0.0, 0.0]], device=DEV)
    for a in values.tolist():
        # logits 0 and a norm of 0 make p = 1 for code 1; its dx is exactly -a
        h = torch.zeros(1, 5, device=DEV)
        w = torch.zeros(2, 5, device=DEV)
        w[1, :4] = values
        gl = torch.tensor([a], device=DEV)
        dh, _ = ops.head_score_backward(h, w, t, norm, None, gl)
        want = -a * values.double()
        assert ((dh[0, :4].double() - want).abs() <= 2.0 ** -22 * want.abs()).all()
