"""Decoding with drafts refuses on the host what it cannot do, before any cache is touched."""
import pytest
import torch


class Layer:
    """Stands for a decoder layer: remembers whether it was run."""

    def __init__(self, pos):
        self.pos, self.runs = pos, 0

    def forward_tree(self, x, parents, lens):
        self.runs += 1
        return x


@pytest.mark.parametrize("pos", [(3, 5), (5, 3), (4, 4, 9)])
def test_decode_tree_refuses_layers_of_different_lengths_before_it_runs_any(pos):
    """A layer that is ahead of the first would have its cached keys overwritten by the nodes."""
    from input_adaptive_reduced_rmm_b200.layer import decode_tree

    layers = [Layer(p) for p in pos]
    tokens, parents = torch.zeros(2, dtype=torch.int32), torch.tensor([-1, 0], dtype=torch.int32)
    with pytest.raises(ValueError, match="different numbers"):
        decode_tree(layers, None, torch.zeros(4, 8, dtype=torch.bfloat16), tokens, parents, torch.zeros(2))
    assert [layer.runs for layer in layers] == [0] * len(pos)
