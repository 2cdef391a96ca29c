"""Group norm backward over rows where every channel is a group of its own: 5857 to 6144
such groups need nearly 48 KB of dynamic shared memory beside the kernel's static one.
Bounds as in test_gpu_norm."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from test_gpu_norm import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("C", [5856, 5857, 6000, 6144, 6145])
def test_channels_as_groups(dtype, C):
    check(make(3, 40, C, dtype, False, seed=C), C, dtype, True)


def test_a_refused_call_spoils_no_later_one():
    """Sizes that the library refuses leave no error behind for the next call."""
    x = torch.randn(4, 3, 8200, device="cuda")
    with pytest.raises(G.GdnError):
        G.gdn_group_norm(x, None, None, 4)
    check(make(2, 30, 64, "bf16", True), 4, "bf16", False)
