"""Eviction of whole requests: one whose choice does not fit on some shard stays as
it is on all of them, and the others go on.  And a captured step of it."""

import numpy as np
import pytest
import torch

from test_gpu_evict import I32, Pool, i32, released, replay, shard_rows
from test_gpu_parity import DEV, cp  # noqa: F401

pytestmark = pytest.mark.gpu
C, CTX, KEEP, MOST = 2, [300, 300, 300, 300, 500, 64], [100, 100, 100, -3, 30, 70], 40


@pytest.fixture
def step(cp):
    """Request 0 fits, 1 has a page that is not there on shard 1, 2 more moves than there
    is room for on shard 0, 3 a negative length, 4 fits, 5 keeps all."""
    p = Pool(cp, C, CTX, (8, 16), seed=5)
    B = len(CTX)
    p.w.fill_(1.0)  # equal weights: the first rows stay, nothing moves
    for b, r, n in ((0, 0, 30), (0, 1, 7), (2, 0, 45), (2, 1, 20), (4, 0, 11)):
        at = p.rows(b, r)
        p.w[torch.from_numpy(at[-n:]).to(DEV)] = 2.0  # the last n rows are the heaviest
    p.table[1 * B + 1, 1] = p.pages.num_pages
    p.pages.dev.copy_(torch.from_numpy(p.table))
    p.pos = torch.arange(p.w.numel(), **I32)
    total = 60
    p.free_ids = torch.cat([torch.full((total,), 7777, **I32), torch.from_numpy(p.free).to(DEV)])
    p.at, p.old, p.new = i32([total]), i32(CTX), i32(KEEP)
    return p


def run(cp, p):
    src, dst, count = cp.cp_evict_select(p.pages, C, p.old, p.new, p.w, MOST)
    cp.cp_cache_move(src, dst, count, p.k, p.v, weights=p.w, pos=p.pos, C=C)
    return count, cp.cp_page_release(p.pages, C, p.old, p.new, p.free_ids, p.at, p.w, p.pos, count=count)


def test_requests_that_do_not_fit_stay(cp, step):
    p, B = step, len(CTX)
    k, v, w, pos, table = (x.clone() for x in (p.k, p.v, p.w, p.pos, p.pages.dev))
    free = p.free_ids.cpu().numpy()
    count, info = run(cp, p)
    assert count.cpu().numpy().reshape(C, B).tolist() == [[30, 0, -1, -1, 11, 0], [7, -1, 20, -1, 0, 0]]
    # as if the three had kept their lengths
    keep = [n if b in (1, 2, 3) else k for b, (n, k) in enumerate(zip(CTX, KEEP))]
    want = released(p, CTX, keep, free, int(p.at))
    assert info.tolist() == want[2][:3] + [3]
    assert np.array_equal(p.free_ids.cpu().numpy(), want[1]) and np.array_equal(p.pages.dev.cpu().numpy(), want[0])
    for b in (1, 2, 3):
        for r in range(C):
            at = p.rows(b, r)
            at = torch.from_numpy(at[(at >= 0) & (at < p.w.numel())]).to(DEV)
            for x, y in ((p.k, k), (p.v, v), (p.w, w), (p.pos, pos)):
                assert torch.equal(x[at], y[at])
    for b in (0, 4):
        for r in range(C):
            at = torch.from_numpy(p.rows(b, r)).to(DEV)
            m = shard_rows(KEEP[b], C, r)
            moved = int(count[r * B + b])
            rank = sorted(range(at.numel()), key=lambda i: (-float(w[at[i]]), i))[:m]
            kept = sorted(rank)
            late, holes = [i for i in kept if i >= m], sorted(set(range(m)) - set(kept))
            assert moved == len(late)
            order = list(range(m))
            for i, j in zip(holes, late):
                order[i] = j
            for x, y in ((p.k, k), (p.w, w), (p.pos, pos)):
                assert torch.equal(x[at[:m]], y[at[order]])
    # request 2 goes with room for its moves, on its own table rows
    rows = torch.tensor([2, B + 2], device=DEV)
    pages = cp.PageTable.on_device(p.pages.dev[rows].contiguous(), p.page, p.pages.num_pages)
    src, dst, count = cp.cp_evict_select(pages, C, i32([300]), i32([100]), p.w, 50)
    assert count.tolist() == [45, 20]


def test_requests_whole_replayed(cp, step):
    p = step
    state = (p.k, p.v, p.w, p.pos, p.pages.dev, p.free_ids)
    keep = [x.clone() for x in state]
    want = [x.clone() for x in (*run(cp, p), *state)]
    for x, y in zip(state, keep):
        x.copy_(y)
    got = [*replay(lambda: run(cp, p), *state), *state]
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("B,shards", [(1, 64), (700, 3), (300, 1)])
def test_all_or_none_of_many_requests(cp, B, shards):
    """Every other request has a pair of -1 on one shard: only the others move and release."""
    ctx, keep = [200] * B, [64] * B
    p = Pool(cp, shards, ctx, (16,), seed=B)
    rng = np.random.default_rng(B)
    count = np.zeros((shards, B), np.int32)
    for b in range(0, B, 2):
        count[rng.integers(shards), b] = -1
    src = np.full((shards * B, 2), -1, np.int32)
    dst = src.copy()
    for r in range(shards):  # one move a pair
        for b in range(B):
            at, m = p.rows(b, r), shard_rows(keep[b], shards, r)
            if count[r, b] == 0 and at.size > m > 0:
                count[r, b], src[r * B + b, 0], dst[r * B + b, 0] = 1, at[-1], at[0]
    k = p.k.clone()
    t = [torch.from_numpy(x).to(DEV) for x in (src, dst, count.reshape(-1))]
    cp.cp_cache_move(*t, p.k, C=shards)
    want = k.clone()
    go = (count >= 0).all(0)
    for r in range(shards):
        for b in np.flatnonzero(go):
            if count[r, b] == 1:
                want[dst[r * B + b, 0]] = k[src[r * B + b, 0]]
    assert torch.equal(p.k, want)
    total = int((p.table >= 0).sum())
    free = np.concatenate([np.full(total, 7777, np.int32), p.free])
    ids = torch.from_numpy(free.copy()).to(DEV)
    info = cp.cp_page_release(p.pages, shards, i32(ctx), i32(keep), ids, i32([total]), p.w, count=t[2])
    out = released(p, ctx, [x if y else 200 for x, y in zip(keep, go)], free, total)
    assert info.tolist() == out[2][:3] + [int((~go).sum())]
    assert np.array_equal(ids.cpu().numpy(), out[1]) and np.array_equal(p.pages.dev.cpu().numpy(), out[0])


def test_whole_requests_refusals(cp):
    p = Pool(cp, 2, [100, 50], (16,))
    t = [torch.full((4, 3), -1, **I32), torch.full((4, 3), -1, **I32), torch.zeros(4, **I32)]
    with pytest.raises(ValueError, match="multiple of C=3"):
        cp.cp_cache_move(*t, p.k, C=3)
    with pytest.raises(ValueError, match="multiple of C=-2"):
        cp.cp_cache_move(*t, p.k, C=-2)
    with pytest.raises(ValueError, match="count"):
        cp.cp_page_release(p.pages, 2, i32([100, 50]), i32([1, 1]), torch.zeros(9, **I32), i32([9]), count=torch.zeros(3, **I32))
    with pytest.raises(TypeError, match="count"):
        cp.cp_page_release(p.pages, 2, i32([100, 50]), i32([1, 1]), torch.zeros(9, **I32), i32([9]), count=torch.zeros(4, device=DEV))
