"""Eviction where its inputs are at their edges: pages that are not there in pairs
that keep all or nothing."""

import pytest
import torch

from test_gpu_evict import Pool, i32, shard_rows
from test_gpu_parity import cp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [1, 300, 3000, 9000])  # pairs of up to 1,024 rows, 4,096, more
@pytest.mark.parametrize("bad", [-1, -7, 1 << 30, "num"])
def test_a_page_that_is_not_there(cp, L, bad):
    """Count -1 whatever the request keeps; a page behind the last one in use does not count."""
    p = Pool(cp, 2, [L, L, L], (16,))
    used = -(-shard_rows(L, 2, 0) // 64)
    ident = p.pages.num_pages if bad == "num" else bad
    for keep in (0, 1, L - 1, L, L + 5):
        if keep < 0:
            continue
        p.pages.dev.copy_(torch.from_numpy(p.table))
        p.pages.dev[0, used - 1] = ident
        p.pages.dev[1, 0] = ident
        p.pages.dev[2, used] = ident
        src, dst, count = cp.cp_evict_select(p.pages, 2, i32([L] * 3), i32([keep] * 3), p.w, max(1, L))
        count = count.cpu().tolist()
        assert count[0] == count[1] == -1 and min(count[2:]) >= 0, (keep, count)
        assert (src[:2] == -1).all() and (dst[:2] == -1).all()
    # a request without tokens has no page
    p.pages.dev.fill_(ident)
    assert (cp.cp_evict_select(p.pages, 2, i32([0] * 3), i32([0, 1, 5]), p.w, 3)[2] == 0).all()
