"""Sizes beyond 32 bits are refused by the softmax-over-codes calls, not cut to their low 32 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
WIDE = (1 << 32) + 5


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def test_rows_of_more_than_32_bits(ops):
    x = torch.empty((1, WIDE), dtype=torch.bfloat16, device=DEV)  # 8 GiB, never read
    t = torch.zeros(1, dtype=torch.int32, device=DEV)
    norm, one = torch.zeros(1, 2, device=DEV), torch.zeros(1, device=DEV)
    print("# logits, head, experts", flush=True)
    for call in (lambda: ops.logits_score(x, t),
                 lambda: ops.logits_score_backward(x, t, norm, one, one, out=x),
                 lambda: ops.head_score(x, x, t),
                 lambda: ops.head_score_backward(x, x, t, norm, one, one)):
        with pytest.raises((ops.GmmError, ValueError)):
            call()
    with pytest.raises((ops.GmmError, ValueError)):
        ops.head_score(x[:, :1], x.view(WIDE, 1), t)  # as many codes


@pytest.mark.parametrize("m", [(1 << 32) + 1, 1 << 32, -(1 << 32) + 2])
def test_alternatives_of_more_than_32_bits(ops, m):
    x, t = torch.zeros(4, 40, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    w = torch.zeros(3, 2 * 40, 40, device=DEV)
    for call in (lambda: ops.logits_score(x, t, m), lambda: ops.head_score(x, x, t, m),
                 lambda: ops.moe_layer(x, w, torch.zeros(3, 40, 40, device=DEV), x[:3], m)):
        with pytest.raises((ops.GmmError, ValueError)):
            call()
