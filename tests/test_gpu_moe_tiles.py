"""The experts' second product in each of its shapes: by tiles of 16 features over (experts or
pairs), with full and ragged last tiles. Inputs, reference and tolerances are test_gpu_moe's.
"""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_moe import _check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,f,e,m", [
    (30, 496, 40, 16, 2), (30, 512, 40, 16, 2), (5, 1009, 33, 32, 3),    # 496, 512, 960 tiles
    (30, 1008, 40, 16, 2), (30, 1024, 40, 16, 2), (70, 1041, 70, 16, 2),  # 1008, 1024, 1056
    (40, 2032, 24, 64, 1), (150, 1030, 24, 40, 4),
])
def test_shapes_of_the_second_product(ops, n, d, f, e, m, dtype):
    _check(ops, n, d, f, e, m, dtype)
