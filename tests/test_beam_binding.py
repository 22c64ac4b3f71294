"""The beam wrappers' own checks, on the host."""

import pytest
import torch

from test_pages_host import sv   # noqa: F401


def test_workspace_of_a_type_that_is_refused(sv):   # noqa: F811
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError, match="logits must be"):
            sv.new_beam_workspace(1, 4, 1000, dtype, device="cpu")
    for dtype, flag in ((torch.float32, sv.SPEC_F32), (torch.bfloat16, sv.SPEC_BF16)):
        ws = sv.new_beam_workspace(1, 4, 9000, dtype, device="cpu")
        assert ws.numel() == sv.spec_beam_workspace_bytes(1, 4, 9000, flag)
