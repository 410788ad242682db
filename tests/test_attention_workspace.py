"""Workspaces that the caller passes to the attention calls."""
import pytest


@pytest.mark.parametrize("view", [lambda t: t[:1].expand(4096), lambda t: t[::2], lambda t: t.view(64, 64).t()])
def test_a_workspace_whose_elements_do_not_lie_side_by_side_is_refused(view):
    """An expanded one has the bytes of one element only."""
    import torch

    from byte_level_lm_amd import ops
    buf = torch.zeros(4096)
    with pytest.raises(ValueError, match="contiguous"):
        ops._scratch(64, view(buf), buf)


def test_a_workspace_of_the_size_is_taken_as_it_is():
    import torch

    from byte_level_lm_amd import ops
    buf = torch.zeros(4096)
    ws, size = ops._scratch(16384, buf, buf)
    assert ws is buf and size == 16384
    with pytest.raises(ValueError, match="workspace too small"):
        ops._scratch(16385, buf, buf)
