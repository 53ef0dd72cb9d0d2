"""What the torch layer takes as a workspace (no GPU needed): the kernels use its bytes from front to back, so a view
with gaps or repeated elements is refused."""
import pytest
import torch

from decode_context_attention_gb300 import binding


@pytest.mark.parametrize("view", [
    lambda t: t[::2],                      # gaps: the kernels would write between its elements
    lambda t: t[:1].expand(4096),          # one byte that claims to be many
    lambda t: t.view(64, 64).t(),
    lambda t: t.view(64, 64)[:, :32],
])
def test_views_that_are_not_contiguous_are_refused(view):
    with pytest.raises(ValueError, match="contiguous"):
        binding._workspace_args(view(torch.zeros(4096, dtype=torch.uint8)))


def test_contiguous_ones_are_taken_whatever_their_type():
    t = torch.zeros(4096, dtype=torch.uint8)
    assert binding._workspace_args(t) == (t.data_ptr(), 4096)
    assert binding._workspace_args(t[16:]) == (t.data_ptr() + 16, 4080)
    f = torch.zeros((8, 8))
    assert binding._workspace_args(f) == (f.data_ptr(), 256)
