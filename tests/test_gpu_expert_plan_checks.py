"""Plans that a caller put together: what the row calls would read has to be there."""
import pytest
import torch

import sparse_selection_primitive_b200 as L

pytestmark = pytest.mark.gpu


def test_plan_without_offsets_is_refused(cuda_device):
    """The number of places in use is the last entry of offsets."""
    plan = L.expert_plan(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 1)
    x, y, w = torch.randn((4, 8), device="cuda"), torch.randn((8, 8), device="cuda"), torch.rand((4, 2), device="cuda")
    L.expert_gather(x, plan)
    for n in (0, 1):
        bad = plan._replace(offsets=plan.offsets[:n])
        with pytest.raises(ValueError, match="offsets"):
            L.expert_gather(x, bad)
        with pytest.raises(ValueError, match="offsets"):
            L.expert_combine(y, w, bad)
