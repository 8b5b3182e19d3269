"""States that are views of other memory's negated values: their bytes are not their values."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_negated_views_are_refused():
    from gmm_em_amd import ops

    z = torch.complex(torch.zeros(4, device=DEV), torch.arange(4.0, device=DEV))
    state = z.conj().imag  # 0, -1, -2, -3 in memory that holds 0, 1, 2, 3
    parent = torch.tensor([[1, 0], [0, 1]], dtype=torch.int32, device=DEV)
    assert state.is_neg()
    with pytest.raises(TypeError):
        ops.beam_reorder(state, parent, 2)
    moved = ops.beam_reorder(state.resolve_neg(), parent, 2)
    assert moved.tolist() == [-1.0, 0.0, -2.0, -3.0]
    with pytest.raises(ValueError):
        ops.beam_reorder(moved, parent, 2, out=state)
