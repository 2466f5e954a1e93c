"""Host side of the long-context operators' edge calls (CPU only)."""
import pytest
import torch

import mla_paged_decode_04_b200 as mla


@pytest.mark.parametrize("make", [
    lambda: mla.MlaDecoder(2, 4, 32, 1000, "fp8", "cpu", window=100, sinks=4),
    lambda: mla.MlaPrefill(2, 9, 32, 1000, "bf16", "cpu"),
])
def test_problems_are_reported_in_the_workspace_of_the_moment(make):
    """Two objects may share a workspace: what key_weights reports goes where status() looks."""
    a, b = make(), make()
    assert a._status.data_ptr() == a.workspace.data_ptr() and a._status.numel() == 1
    a.workspace = b.workspace
    assert a.workspace is b.workspace and a._status.data_ptr() == b.workspace.data_ptr()
    a.workspace = b.workspace.view(torch.int32).view(2, -1)
    assert a._status.data_ptr() == b.workspace.data_ptr() and a._status.numel() == 1
    a.workspace = None
    assert a.workspace is None
