"""Embedding gradient at numbers of rows where the searches for codes without rows end after
different numbers of steps in one wave, into tables of one, two and three digits.

Gradients are whole numbers below 2^7 and at most 2^17 rows are summed: every sum is exact in fp32, and the
results are compared for equality. What the probes read is checked on the host (test_embed_search.py).
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


@pytest.mark.parametrize("v", [1, 15, 1000, 1025, (1 << 20) + 1])
@pytest.mark.parametrize("n", [15624, 15625, 16384, 16406, 17000, 19530, 19531, 78125, 90000, 97655])
def test_codes_without_rows(ops, n, v):
    print(f"# embed gradient n={n} v={v}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(n + v)
    d = 5
    grad = torch.randint(-100, 101, (n, d), generator=g, device=DEV).float()
    rand = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    for codes in ((v * rand).to(torch.int32),                      # met evenly
                  (v * rand ** 3).to(torch.int32),                 # unevenly
                  (v // 2 + (v - v // 2) * rand).to(torch.int32),  # the first ones not at all
                  (v // 2 * rand).to(torch.int32)):                # nor the last ones
        codes = codes.clamp(max=v - 1)
        codes[rand < 0.01] = -1
        keep = codes >= 0
        ref = torch.zeros(v, d, dtype=torch.float64, device=DEV)
        ref.index_add_(0, codes[keep].long(), grad[keep].double())
        out = torch.full((v, d), 7.0, device=DEV)
        ops.embed_backward(grad, codes, v, out=out)
        assert torch.equal(out.double(), ref)
