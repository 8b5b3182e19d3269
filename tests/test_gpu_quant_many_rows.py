"""More long rows in 8-bit integers than a launch has workgroups for: 2^22 + 5 rows of 16385 bf16 values."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_more_long_rows_than_workgroups():
    from gmm_em_amd import ops

    n, d = (1 << 22) + 5, 16385
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 3 * n * d + (8 << 30):
        pytest.skip("needs 214 GB of device memory")
    x = torch.ones(n, d, dtype=torch.bfloat16, device=DEV)
    top = (2 + torch.arange(n, device=DEV) % 125).float()  # whole numbers that bf16 holds
    x[:, d - 1] = -top.to(torch.bfloat16)
    q, scale = ops.quantize_rows(x)
    want = (top.double() / 127.0).float()
    assert torch.equal(scale, want)
    assert q[:, d - 1].eq(-127).all()
    one = torch.round(1.0 / want.double()).to(torch.int8)
    for k in (0, d // 2, d - 2):
        assert torch.equal(q[:, k], one)
    for r in (0, (1 << 20) - 1, 1 << 20, (1 << 22) - 1, 1 << 22, n - 1):
        assert q[r, :-1].eq(one[r]).all()
    del x, q
    torch.cuda.empty_cache()
