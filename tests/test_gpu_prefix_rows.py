"""A row's results over a shared prefix do not depend on the other rows of its block."""

import math

import pytest
import torch

from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
@pytest.mark.parametrize("members", [20, 70])
@pytest.mark.parametrize("other", [math.nan, 30.0])
def test_prefix_row_beside_another(cp, kv, D, members, other):
    """Another query that is NaN, or whose running maximum moves at every tile,
    takes the whole warp through the exact path: the bits of all others stay."""
    c = Case(cp, 1, [900], [members], 8, 2, D, kv, workers=2)
    o, lse = c.run(out_dtype=torch.float32)
    q = c.q[3, 5].clone()
    c.q[3, 5] = math.nan if math.isnan(other) else q * other
    o2, lse2 = c.run(out_dtype=torch.float32)
    cp.cp_device_error_check()
    if math.isnan(other):
        assert o2[3, 5].isnan().all() and lse2[3, 5].isnan()
    o2[3, 5], lse2[3, 5] = o[3, 5], lse[3, 5]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
