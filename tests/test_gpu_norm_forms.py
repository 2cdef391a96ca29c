"""Group norm around the limits between its forms: samples too many or too small to be
cut into slabs in one direction or both, and the widest rows.  Bounds as in
test_gpu_norm."""
from __future__ import annotations

import pytest

from test_gpu_norm import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("N,S,C,groups", [
    (151, 20, 64, 4), (152, 20, 64, 4), (200, 3, 36, 3),       # by the number of samples
    (170, 64, 256, 8), (170, 63, 256, 8),                      # backward by their size
    (153, 128, 512, 8), (153, 127, 512, 8), (153, 15, 4400, 4),  # forward by their size
    (2, 40, 8192, 8), (160, 17, 4096, 1)])
def test_limits(dtype, gate, N, S, C, groups):
    check(make(N, S, C, dtype, gate, seed=N + S), groups, dtype, silu=not gate)
