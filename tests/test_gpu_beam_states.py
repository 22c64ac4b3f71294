"""GPU test of reordering states some of whose rows have no elements."""

import pytest
import torch

from test_gpu_beam import sv   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [0, 3])
def test_some_states_are_empty(sv, R):   # noqa: F811
    x = torch.arange(R * 5, device="cuda").view(R, 5)
    empty = torch.empty((R, 0, 4), device="cuda")
    parents = torch.tensor([R - 1, -1, 0 if R else -1, R - 1], dtype=torch.int32, device="cuda")
    a, b, c, st = sv.beam_reorder([empty, x, empty], parents)
    assert a.shape == c.shape == (4, 0, 4) and int(st.item()) == 0
    want = torch.zeros(4, 5, dtype=x.dtype, device="cuda")
    for i, p in enumerate(parents.tolist()):
        if p >= 0:
            want[i] = x[p]
    assert torch.equal(b, want)
