"""Gate logits of -inf and NaN: experts are ranked by z, and NaN comes after every number."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [6, 100, 600, 4096])  # ranked in registers, and by counting
def test_nan_ranks_last(ops, dtype, e):
    n, d, f, m = 3, 2, 1, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(e)
    x = torch.ones(n, d, device=DEV)
    z = torch.randint(-20, 20, (e,), generator=g, device=DEV).float()
    low = torch.finfo(dtype).min
    z[0], z[1], z[2], z[e - 1] = float("nan"), -INF, low, -INF
    if e > 6:
        z[6:-1] = float("nan")  # fewer numbers than picks but for the infinities
    gate = torch.zeros(e, d, device=DEV)
    gate[:, 0] = z
    w_in, w_out = torch.zeros(e, 2 * f, d, device=DEV), torch.zeros(e, d, f, device=DEV)
    print(f"# e={e} {dtype}", flush=True)
    _, idx, _ = ops.moe_layer(x.to(dtype), w_in.to(dtype), w_out.to(dtype), gate.to(dtype), m)
    zs = z.tolist()
    rank = sorted(range(e), key=lambda i: (zs[i] != zs[i], -zs[i] if zs[i] == zs[i] else 0.0, i))
    assert idx.tolist() == [rank[:m]] * n
    _, one, share = ops.moe_layer(x.to(dtype), w_in.to(dtype), w_out.to(dtype), gate.to(dtype), 1)
    assert one.tolist() == [rank[:1]] * n and share.eq(1).all()
