"""Eviction where its inputs are at their edges: pages that are not there in pairs
that keep all or nothing, and positions that nobody has written."""

import numpy as np
import pytest
import torch

from test_gpu_evict import I32, Pool, i32, shard_rows
from test_gpu_parity import DEV, cp  # noqa: F401

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


@pytest.mark.parametrize("C,ctx,keep", [(2, 300, 200), (1, 3000, 100), (1, 9000, 8999), (8, 5000, 512)])
@pytest.mark.parametrize("below", [0, 4])
def test_a_position_that_nobody_has_written(cp, C, ctx, keep, below):
    """Rows of a negative position are protected by neither bound: they stay by their weight."""
    p = Pool(cp, C, [ctx], (16,), seed=ctx)
    rng = np.random.default_rng(3)
    w = rng.random(p.w.numel()).astype(np.float32)
    pos = np.full(w.size, -1, np.int32)
    for r in range(C):
        at = p.rows(0, r)
        known = rng.random(at.size) < 0.5
        pos[at[known]] = (np.arange(at.size) * C + r)[known]
        pos[at[~known]] = rng.choice([-1, -2, -2**31], int((~known).sum()))
    start = ctx - 20
    most = max(1, min(shard_rows(ctx, C, 0), shard_rows(keep, C, 0)))
    src, dst, count = cp.cp_evict_select(p.pages, C, i32([ctx]), i32([keep]), torch.from_numpy(w).to(DEV), most, pos=torch.from_numpy(pos).to(DEV),
                                         keep_below=below, keep_from=i32([start]))
    src, dst, count = (x.cpu().numpy() for x in (src, dst, count))
    for r in range(C):
        at, m = p.rows(0, r), shard_rows(keep, C, r)
        where = pos[at]
        safe = ((where >= 0) & (where < below)) | (where >= start)
        rank = sorted(range(at.size), key=lambda i: (not safe[i], 0.0 if safe[i] else -float(w[at[i]]), i))
        stay = sorted(rank[:m])
        late, holes = [i for i in stay if i >= m], sorted(set(range(m)) - set(stay))
        assert count[r] == len(late)
        assert src[r, :len(late)].tolist() == at[late].tolist() and dst[r, :len(late)].tolist() == at[holes].tolist()


def test_tokens_appended_without_positions(cp):
    """A released row's position is -1: tokens put there compete by weight."""
    p = Pool(cp, 1, [128], (16,))
    pos = torch.full((p.w.numel(),), -1, **I32)
    at = torch.from_numpy(p.rows(0, 0)).to(DEV)
    pos[at[:64]] = torch.arange(64, **I32)
    w = torch.ones_like(p.w)
    w[at[64:]] = 0.5  # new tokens, lighter
    src, dst, count = cp.cp_evict_select(p.pages, 1, i32([128]), i32([64]), w, 64, pos=pos, keep_from=i32([1000]))
    assert count.item() == 0
