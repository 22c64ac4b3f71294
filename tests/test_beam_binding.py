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


def test_states_of_empty_rows(sv):   # noqa: F811
    """Nothing to move, and nothing that needs a device."""
    from speculative_decoding_verification_78_gb300 import _binding as b
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    assert b.spec_beam_reorder([i32(3, 0), i32(3, 2, 0)], i32(4), [i32(4, 0), i32(4, 2, 0)], i32(1)) == sv.SPEC_OK
    with pytest.raises(ValueError, match="device tensor"):   # the others are checked
        b.spec_beam_reorder([i32(3, 0), i32(3, 2)], i32(4), [i32(4, 0), i32(4, 2)], i32(1))
    with pytest.raises(ValueError):
        b.spec_beam_reorder([i32(3, 0)], i32(4), [i32(5, 0)], i32(1))
