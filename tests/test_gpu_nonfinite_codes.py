"""Values that are no numbers over E4M3 caches: a NaN code of a row that is read
reaches the results, as it does in the other forms of the same calls, and
nothing else."""

import math

import pytest
import torch

from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


def repack(cp, c):
    """The case's values again, where its cache has them."""
    if c.pages:
        cp.cp_kv_shard_pack_paged(c.dplan, c.pages, c.v, None, c.pool[1])
    else:
        c.sv = cp.cp_kv_shard_pack(c.dplan, c.v)[0]


@pytest.mark.parametrize("D", [128, 64])  # the tensor cores, the CUDA cores
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("members", [1, 9, 25, 70])  # blocks of up to 64, 128 and 256 rows
@pytest.mark.parametrize("workers", [1, 7])
def test_prefix_value_code_that_is_nan(cp, D, page, members, workers):
    """The dim of that kv head is NaN for every query of the group; all others
    and the LSE keep their bits.  Tokens at both ends of tiles, whole and cut ones."""
    C, lens = 2, [700, 130]
    c = Case(cp, C, lens, [members, members], 8, 2, D, "fp8", page=page, workers=workers)
    o, lse = c.run(out_dtype=torch.float32)
    codes = c.v.view(torch.uint8)
    at = [(0, 0, 0, 0x7F), (255, 1, D - 1, 0xFF), (256, 0, 17, 0x7F), (699, 1, 16, 0x7F), (698, 0, 63, 0xFF), (700 + 129, 1, 33, 0xFF)]
    want = o.clone()
    for t, g, d, code in at:
        codes[t, g, d] = code
        rows = slice(0, members) if t < 700 else slice(members, None)
        want[rows, 4 * g:4 * g + 4, d] = math.nan
    repack(cp, c)
    o2, lse2 = c.run(out_dtype=torch.float32)
    cp.cp_device_error_check()
    assert torch.equal(lse, lse2)
    assert torch.equal(want.isnan(), o2.isnan())
    assert torch.equal(want.nan_to_num(9.0), o2.nan_to_num(9.0))
