"""Few long rows, which are scored in parts that a second kernel joins.

Tolerances: log p and the log-sum 2^-18 (differences from the maximum below 32, rounded twice
to 2^-20, the exponential and the logarithm), entropy 2^-15; whole numbers are equal.
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


def _check(ops, x, t, m, scale=1.25):
    print(f"# {tuple(x.shape)} {x.dtype} m={m} scale={scale}", flush=True)
    s = ops.logits_score(x, t, m, scale)
    l = (x.float() * scale).double()
    lp, ent, norm, idx, top = ref.scores(l, t, m)

    def close(a, b, tol):
        a = a.double()
        same = (a == b) | (torch.isnan(a) & torch.isnan(b))
        assert bool((same | ((a - b).abs() <= tol)).all()), (a, b)

    close(s.logprob, lp, 2.0 ** -18)
    close(s.entropy, ent, 2.0 ** -15)
    close(s.norm, norm, 2.0 ** -18)
    if m:
        assert torch.equal(s.top_idx, idx)
        close(s.top_logprob, top, 2.0 ** -18)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 98303), (1, 98304), (3, 131072), (85, 98311), (86, 98311),
                                 (2, 2_200_001), (17, 300_007)])
@pytest.mark.parametrize("m", [0, 1, 16])
def test_parts(ops, n, v, m, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(n + v)
    x = 2.5 * torch.randn(n, v, generator=g, device=DEV)
    t = torch.randint(-1, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    _check(ops, x.to(dtype), t, m)
    x[torch.rand(n, v, generator=g, device=DEV) < 0.4] = -INF
    _check(ops, x.to(dtype), t, m)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_parts_with_nothing_ties_and_nan(ops, dtype):
    v = 131_099
    g = torch.Generator(device=DEV)
    g.manual_seed(v)
    x = torch.randint(-2, 3, (12, v), generator=g, device=DEV).to(dtype)
    low = torch.finfo(dtype).min
    x[0] = -INF                    # nothing left
    x[1] = low                     # uniform
    x[2, 1:] = low                 # one code left
    x[3, 3:] = -INF                # fewer left than alternatives
    x[4, v // 2] = float("nan")
    x[5, v - 1], x[5, 7] = INF, INF
    x[6, :-1] = -INF               # the last part alone
    x[7, 40000:] = -INF            # the first parts alone
    x[8] = 0.0                     # all equal
    x[9, ::2] = -0.0
    t = torch.full((12,), 1, dtype=torch.int32, device=DEV)
    t[10], t[11] = -1, v
    _check(ops, x, t, 16, 1.0)
    _check(ops, x, t, 16, 0.75)
