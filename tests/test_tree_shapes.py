"""Shapes that hold the right number of elements in the wrong places are refused."""
import pytest
import torch

from test_tree_refusals import i32, rmm  # noqa: F401 (a fixture)


@pytest.mark.parametrize("shape", [(3, 2, 50), (1, 5, 50), (7, 1, 50)])
@pytest.mark.parametrize("which", ["P", "Qd"])
def test_verification_rows_of_another_batch(rmm, shape, which):  # noqa: F811
    """[T, B, V] rows in place of [B, T, V] would be read as other nodes'."""
    B, T, V = 2, 3, 50
    kw = dict(P=torch.zeros(B, T, V), Qd=torch.zeros(B, T, V))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):  # the right shapes
        rmm.rmm_tree_verify(kw["P"], i32(B, T), i32(B, T), torch.zeros(B, T), Qd=kw["Qd"])
    kw[which] = torch.zeros(shape)
    with pytest.raises(ValueError, match=which + " has shape"):
        rmm.rmm_tree_verify(kw["P"], i32(B, T), i32(B, T), torch.zeros(B, T), Qd=kw["Qd"])
