"""Pages, slots and appended rows of a paged cache, and a latent-attention
step through all of them.

Slots, tables and copied rows are exact.  An E4M3 row is checked against the
rule itself in fp32 (scale = amax / 448, code = rn(x / scale)), code by code.
"""

import math
import threading

import numpy as np
import pytest
import torch

import cp_workloads as W
import oracle
from test_gpu_mla import close, randn, weights
from test_gpu_parity import DEV, cp, np64  # noqa: F401

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def held_table(C, ctx, page, max_pages, num_pages, seed):
    """(table, unused page ids): distinct random ids for the pages that the
    cached tokens hold, -1 elsewhere."""
    rng = np.random.default_rng(seed)
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((C * len(ctx), max_pages), -1, np.int32)
    k = 0
    for r in range(C):
        for b, L in enumerate(ctx):
            n = -(-len(range(r, max(L, 0), C)) // page)
            table[r * len(ctx) + b, :n] = ids[k:k + n]
            k += n
    return table, ids[k:]


def step(cp, C, ctx, new, page, max_pages, num_pages, max_tokens, seed=0, free=None, pos=0):
    table, unused = held_table(C, ctx, page, max_pages, max(num_pages, 1), seed)
    free = unused if free is None else np.asarray(free, np.int32)
    pages = cp.PageTable.on_device(dev(table), page, num_pages)
    got = cp.cp_page_slots(pages, C, dev(ctx), dev(new), dev(free), dev([pos]), max_tokens)
    torch.cuda.synchronize()
    want = oracle.page_slots(C, ctx, new, table, page, num_pages, free, pos, max_tokens)
    for g, w, what in zip([*got, pages.dev], want, ("slots", "cu_new", "info", "table")):
        assert np.array_equal(g.cpu().numpy(), w), f"{what}: {g.cpu().numpy()} != {w}"
    return got, pages, want


@pytest.mark.parametrize("C", [1, 2, 3, 8, 64])
@pytest.mark.parametrize("page", [64, 192])
def test_slots(cp, C, page):
    ctx = [0, 1, page * C - 1, page * C, 5 * page * C + 3, 0, 700, 64]
    new = [1, page * C, 1, 1, 0, 0, 3000, 129]
    step(cp, C, ctx, new, page, max_pages=80, num_pages=4000, max_tokens=sum(new) + 5, seed=C, pos=3)


def test_slots_of_a_decode_step(cp):
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 5000, 300).tolist()
    step(cp, 8, ctx, [1] * 300, 64, max_pages=12, num_pages=30000, max_tokens=300)
    step(cp, 8, ctx, [0] * 300, 64, max_pages=12, num_pages=30000, max_tokens=300)


def test_slots_of_many_requests_and_of_one_long_one(cp):
    n = 8192
    ctx = np.random.default_rng(6).integers(0, 90, n).tolist()
    new = np.random.default_rng(7).integers(0, 3, n).tolist()
    step(cp, 2, ctx, new, 64, max_pages=2, num_pages=40000, max_tokens=2 * n + 3)
    step(cp, 3, [1000001], [123457], 64, max_pages=5860, num_pages=20000, max_tokens=123457)


def test_slots_without_tokens(cp):
    step(cp, 2, [5, 0], [0, 0], 64, 4, 16, max_tokens=0)
    step(cp, 2, [5, 0], [0, 0], 64, 4, 16, max_tokens=9, free=[], pos=0)


@pytest.mark.parametrize("case", ["negative", "sum", "table", "pages", "pos", "pos_past", "tokens", "several"])
def test_slots_of_a_step_that_does_not_fit(cp, case):
    """Nothing is taken and the reason is reported."""
    ctx, new, kw = [10, 20, 30], [100, 200, 300], dict(max_pages=8, num_pages=64, max_tokens=700)
    if case == "negative":
        new = [100, -1, 300]
    elif case == "sum":
        ctx = [10, 2**31 - 100, 30]
        table = np.full((6, 8), 0, np.int32)
        pages = cp.PageTable.on_device(dev(table), 64, 64)
        s, cu, info = cp.cp_page_slots(pages, 2, dev(ctx), dev(new), dev(range(40)), dev([0]), 700)
        assert info.tolist() == [1, 0, 0, 0] and bool((s == -1).all()) and not cu.any()
        assert not pages.dev.any()
        return
    elif case == "table":
        kw["max_pages"] = 2
    elif case == "pages":
        kw["free"] = [7, 8, 9]
    elif case == "pos":
        kw["pos"] = -1
    elif case == "pos_past":
        kw.update(free=[7, 8, 9], pos=4)
    elif case == "tokens":
        kw["max_tokens"] = 599
    else:
        kw.update(free=[], max_tokens=1)
    (_, _, info), _, want = step(cp, 2, ctx, new, 64, **kw)
    assert want[2][0] != 0 and info[0].item() == want[2][0]


def test_slots_of_sums_past_31_bits(cp):
    """Sums of tokens and of pages past 2^31 - 1 are over the largest limits,
    too (the other reasons keep the step from taking anything either way)."""
    table, most = torch.full((128, 2), -1, **I32), 2**31 - 1
    slots, cu, info = cp.cp_page_slots(cp.PageTable.on_device(table[:3], 64, 100), 1, dev([0] * 3), dev([2**30] * 3),
                                       dev(range(50)), dev([0]), most)
    assert info.tolist() == [2 + 4 + 8, 0, 0, 0] and not cu.any()
    assert all(bool((part == -1).all()) for part in slots.split(1 << 28))
    del slots
    free = torch.empty(most, **I32)  # never read
    slots, cu, info = cp.cp_page_slots(cp.PageTable.on_device(table, 64, 100), 1, dev([0] * 128), dev([most] * 128),
                                       free, dev([0]), 5)
    assert info.tolist() == [2 + 4 + 8, 0, 0, 0] and not cu.any() and bool((slots == -1).all())
    assert bool((table == -1).all())


def test_slots_of_bad_page_ids(cp):
    """An id outside the pool gives no row in it."""
    step(cp, 2, [0, 10], [200, 300], 64, max_pages=8, num_pages=20, max_tokens=500, free=[3, 20, -5, 2**31 - 1, 19, 0, 1, 2, 4, 5])


def test_slots_of_batches_of_different_size_at_once(cp):
    """Host threads whose batches need different amounts of shared memory: no
    launch is refused, and each gets its own slots."""
    bad = []

    def work(B, n=4000):
        pages = cp.PageTable.on_device(torch.full((B, 4), -1, **I32), 64, 4 * B)
        ctx, new, free, pos = torch.zeros(B, **I32), torch.ones(B, **I32), torch.arange(4 * B, **I32), torch.zeros(1, **I32)
        slots, cu, info = torch.empty(B, **I32), torch.empty(B + 1, **I32), torch.empty(4, **I32)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        args = (1, B, ctx.data_ptr(), new.data_ptr(), pages.dev.data_ptr(), 4, 64, 4 * B, free.data_ptr(), 4 * B, pos.data_ptr(),
                slots.data_ptr(), B, cu.data_ptr(), info.data_ptr(), stream.cuda_stream)
        for _ in range(n):  # the library's call by itself: the threads meet in it
            status = cp.lib.cp_page_slots(*args)
            if status:
                bad.append((B, status, cp.lib.cp_last_error()))
                break
        stream.synchronize()
        if not torch.equal(slots, torch.arange(B, **I32) * 64):
            bad.append((B, "slots"))

    threads = [threading.Thread(target=work, args=(B,)) for B in (8192, 5200, 8192, 5200, 8192, 100)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_slots_follow_their_lengths_in_a_graph(cp):
    """A captured step, replayed as a decode loop: lengths and the free
    position are advanced on the GPU between replays."""
    C, B, page, num_pages = 3, 5, 64, 60
    ctx = [0, 63, 64 * C - 1, 200, 1000]
    table, unused = held_table(C, ctx, page, 10, num_pages, 1)
    pages = cp.PageTable.on_device(dev(table), page, num_pages)
    L, n, free, pos = dev(ctx), dev([1, 1, 1, 0, 2]), dev(unused), dev([0])
    cp.cp_page_slots(pages, C, L, n, free, pos, 8)  # loads the kernel before the capture; takes the first step's pages
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, cu, info = cp.cp_page_slots(pages, C, L, n, free, pos, 8)
        L += n
        pos.copy_(info[1:2])
    at = 0
    for _ in range(130):
        graph.replay()
        torch.cuda.synchronize()
        ws, wc, wi, table = oracle.page_slots(C, ctx, [1, 1, 1, 0, 2], table, page, num_pages, unused, at, 8)
        assert wi[0] == 0
        assert np.array_equal(slots.cpu().numpy(), ws) and np.array_equal(info.cpu().numpy(), wi)
        assert np.array_equal(pages.dev.cpu().numpy(), table) and np.array_equal(cu.cpu().numpy(), wc)
        at, ctx = int(wi[1]), [a + b for a, b in zip(ctx, [1, 1, 1, 0, 2])]


# ------------------------------------------------------------------ append

def quantised(k, v):
    """Codes and scales by the rule, in fp32, on the host: a division by 448
    there is a division (a CUDA tensor over a Python number is multiplied by
    the number's rounded inverse, up to a unit in the last place off)."""
    k, v = k.cpu().float(), None if v is None else v.cpu().float()
    flat = (k.flatten(1) if v is None else torch.cat([k.flatten(1), v.flatten(1)], 1)).numpy()
    amax = np.abs(flat).max(1)
    scale = np.where(amax > 0, amax / np.float32(448.0), np.float32(1.0)).astype(np.float32)
    q = torch.from_numpy(np.clip(flat / scale[:, None], -448, 448).astype(np.float32))
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    m = k[0].numel()
    vc = None if v is None else codes[:, m:].reshape(k.shape).to(DEV)
    return codes[:, :m].reshape(k.shape).to(DEV), vc, torch.from_numpy(scale).to(DEV)


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,row,with_v", [(1, (576,), False), (130, (576,), False), (33, (1, 64), True), (50, (8, 128), True),
                                          (7, (2, 16), False), (21, (32, 128), True), (5, (3, 208), True), (700, (4, 128), True)])
def test_append_quantised(cp, src, n, row, with_v):
    g = torch.Generator(device=DEV).manual_seed(n)
    size = torch.exp(3 * torch.randn((n,) + (1,) * len(row), generator=g, device=DEV))
    k = (torch.randn((n, *row), generator=g, device=DEV) * size).to(src)
    v = (torch.randn((n, *row), generator=g, device=DEV) * size).to(src) if with_v else None
    k[n // 2] = 0
    if v is not None and n > 10:
        v[n // 2] = 0  # a token of zeros: scale 1
    k.flatten()[0] = 3e38 if n > 40 else 1e-38
    rows = 2 * n + 64
    slots = torch.randperm(rows, generator=g, device=DEV)[:n].to(torch.int32)
    if n > 10:
        slots[3], slots[7] = -1, rows
    fill = torch.randint(0, 100, (rows, *row), generator=g, device=DEV, dtype=torch.uint8)
    kp, vp, sp = fill.clone(), fill.clone() if with_v else None, torch.full((rows,), -7.0, device=DEV)
    cp.cp_cache_append(slots, k, kp.view(torch.float8_e4m3fn), v, vp, sp)
    torch.cuda.synchronize()
    kc, vc, sc = quantised(k, v)
    live = (slots >= 0) & (slots < rows)
    at = slots[live].long()
    assert torch.equal(sp[at], sc[live])
    assert torch.equal(kp[at], kc[live])
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert torch.equal(kp[rest], fill[rest]) and bool((sp[rest] == -7.0).all())
    if with_v:
        assert torch.equal(vp[at], vc[live]) and torch.equal(vp[rest], fill[rest])


def test_append_rounds_ties_and_extremes(cp):
    """Quotients on and beside the borders between two codes, the smallest
    codes, and scales far from 1."""
    rows = []
    for scale_exp in (-140, -126, -100, -60, -3, 0, 4, 60, 119):
        base = np.ldexp(np.float64(448.0), scale_exp)
        vals = [base]
        for c in range(126):
            a, b = oracle.e4m3_to_float(c), oracle.e4m3_to_float(c + 1)
            mid = np.float32(np.ldexp((a + b) / 2, scale_exp))
            vals += [mid, np.nextafter(mid, np.float32(np.inf)), -np.nextafter(mid, np.float32(0))]
        rows.append(np.resize(np.asarray(vals, np.float32), 384))
    k = torch.from_numpy(np.stack(rows)).to(DEV)
    n = k.shape[0]
    kp, sp = torch.zeros((n, 384), dtype=torch.uint8, device=DEV), torch.zeros(n, device=DEV)
    cp.cp_cache_append(torch.arange(n, **I32), k, kp, scale_pool=sp)
    kc, _, sc = quantised(k, None)
    assert torch.equal(sp, sc) and torch.equal(kp, kc)


def test_append_quantises_any_scale(cp):
    """The codes of a division, bit for bit, over random scales."""
    g = torch.Generator(device=DEV).manual_seed(77)
    k = torch.randn((4000, 576), generator=g, device=DEV) * torch.exp(8 * torch.randn((4000, 1), generator=g, device=DEV))
    kp, sp = torch.zeros((4000, 576), dtype=torch.uint8, device=DEV), torch.zeros(4000, device=DEV)
    cp.cp_cache_append(torch.arange(4000, **I32), k, kp, scale_pool=sp)
    kc, _, sc = quantised(k, None)
    assert torch.equal(sp, sc) and torch.equal(kp, kc)


@pytest.mark.parametrize("row,with_v", [((64,), False), ((576,), False), ((8, 128), True), ((2048,), True)])
def test_append_of_the_smallest_rows(cp, row, with_v):
    """fp32 rows whose amax / 448 is no fp32 number, or one of its smallest, with
    zeros of either sign among them: the scale is never 0 and a code never NaN."""
    tiny = np.float32(2.0 ** -149)
    sizes = np.asarray([1, 2, 7, 100, 223, 224, 225, 447, 448, 449, 900, 7000], np.float32) * tiny
    n, m = len(sizes), int(np.prod(row))
    base = np.resize(np.asarray([0.0, 1.0, -0.0, -1.0, 0.5, 0.0, -0.25], np.float32), (2, n, m))
    k, v = (torch.from_numpy((x * sizes[:, None]).astype(np.float32).reshape(n, *row)) for x in base)
    both = torch.cat([k.flatten(1), v.flatten(1)], 1).numpy() if with_v else k.flatten(1).numpy()
    assert (np.abs(both).max(1) == sizes).all()
    scale = np.maximum(sizes / np.float32(448), tiny)
    want = torch.from_numpy(np.clip(both / scale[:, None], -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    kp, sp = torch.full((n, *row), 77, dtype=torch.uint8, device=DEV), torch.zeros(n, device=DEV)
    vp = torch.full_like(kp, 77) if with_v else None
    cp.cp_cache_append(torch.arange(n, **I32), k.to(DEV), kp, v.to(DEV) if with_v else None, vp, sp)
    got = torch.cat([kp.flatten(1), vp.flatten(1)], 1) if with_v else kp.flatten(1)
    assert np.array_equal(sp.cpu().numpy(), scale) and torch.equal(got.cpu(), want)
    assert not bool(((got & 127) == 127).any())


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
def test_append_keeps_the_sign_of_zero(cp, src):
    """Zeros of either sign, in rows of any scale and in a row of zeros."""
    k = torch.tensor([[0.0, -0.0, 1.0, -1.0, 0.0, -1e-30, 1e-30, -0.0] * 8] * 4, device=DEV)
    k[1] *= 1e-4
    k[2] *= 1e30
    k[3] = torch.where(k[3].signbit(), -0.0, 0.0)
    k = k.to(src)
    kp, sp = torch.full((4, 64), 77, dtype=torch.uint8, device=DEV), torch.zeros(4, device=DEV)
    cp.cp_cache_append(torch.arange(4, **I32), k, kp, scale_pool=sp)
    kc, _, sc = quantised(k, None)
    assert torch.equal(sp, sc) and torch.equal(kp, kc)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("n,heads,dim", [(1, 1, 64), (40, 8, 128), (19, 3, 48), (9, 1, 576), (3000, 2, 64)])
def test_append_copies(cp, dtype, n, heads, dim):
    """Rows as they are, from views of a wider projection output."""
    g = torch.Generator(device=DEV).manual_seed(n)
    wide = torch.randint(0, 255, (n, 3 * heads * dim * dtype.itemsize), generator=g, device=DEV, dtype=torch.uint8).view(dtype)
    k = wide[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
    v = wide[:, 2 * heads * dim:].unflatten(1, (heads, dim))
    rows = n + 30
    slots = torch.randperm(rows, generator=g, device=DEV)[:n].to(torch.int32)
    if n > 1:
        slots[n // 2] = -1
    pools = [torch.zeros((rows, heads, dim), dtype=dtype, device=DEV) for _ in range(2)]
    fp8 = dtype == torch.uint8
    ns = torch.rand(n, generator=g, device=DEV) if fp8 else None
    sp = torch.zeros(rows, device=DEV) if fp8 else None
    cp.cp_cache_append(slots, k, pools[0], v, pools[1], sp, ns)
    torch.cuda.synchronize()
    keep = slots >= 0
    at = slots[keep].long()
    for src, pool in zip((k, v), pools):
        want = torch.zeros_like(pool)
        want.view(torch.uint8)[at] = src[keep].contiguous().view(torch.uint8)
        assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))
    if fp8:
        assert torch.equal(sp[at], ns[keep])


def test_append_past_32_bits(cp):
    """Slots whose rows lie past 2^32 bytes of the pool."""
    rows = 8_000_000
    pool, scales = torch.zeros((rows, 576), dtype=torch.uint8, device=DEV), torch.zeros(rows, device=DEV)
    k = randn((5, 576), 1)
    slots = dev([rows - 1, 0, rows - 64, rows // 2, 4_000_001])
    cp.cp_cache_append(slots, k, pool, scale_pool=scales)
    kc, _, sc = quantised(k, None)
    at = slots.long()
    assert torch.equal(pool[at], kc) and torch.equal(scales[at], sc)
    assert int((scales != 0).sum()) == 5
    pool16 = pool.view(torch.bfloat16)[:, :288]
    pool16.zero_()
    cp.cp_cache_append(slots, k[:, :288], pool16)  # a view of a wider row as the source
    assert torch.equal(pool16[at], k[:, :288])


def test_append_nothing(cp):
    pool = torch.ones((64, 576), dtype=torch.bfloat16, device=DEV)
    cp.cp_cache_append(torch.empty(0, **I32), torch.empty((0, 576), dtype=torch.bfloat16, device=DEV), pool)
    cp.cp_cache_append(torch.full((3,), -1, **I32), torch.zeros((3, 576), dtype=torch.bfloat16, device=DEV), pool)
    torch.cuda.synchronize()
    assert bool((pool == 1).all())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fp8", [False, True])
def test_latent_attention_step(cp, fp8):
    """A prompt and three decode steps of a small latent-attention layer: the
    prompt in expanded form, its rows appended to the paged cache, then
    single tokens in absorbed form over that cache.  Every output is checked
    against plain attention in fp64 over the rows that the cache stands for."""
    H, C, page, scale = 8, 2, 64, 1.0 / math.sqrt(192)
    new, B = [150, 1, 333], 3
    w = weights(H, 1)
    nw = np64(w)
    num_pages = 24
    pages = cp.PageTable.on_device(torch.full((C * B, 4), -1, **I32), page, num_pages)
    free, pos = torch.randperm(num_pages, device=DEV).to(torch.int32), torch.zeros(1, **I32)
    pool = torch.zeros((pages.pool_rows, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    spool = torch.zeros(pages.pool_rows, device=DEV) if fp8 else None

    def append(ctx, n, rows):
        nonlocal pos
        slots, _, info = cp.cp_page_slots(pages, C, dev(ctx), dev(n), free, pos, rows.shape[0])
        cp.cp_cache_append(slots, rows, pool, scale_pool=spool)
        pos = info[1:2]
        assert info[0].item() == 0

    def stored(rows):  # what the cache holds for these rows
        if not fp8:
            return np64(rows)
        codes, _, sc = quantised(rows, None)
        return oracle.e4m3_decode(codes.cpu().numpy()) * np64(sc)[:, None]

    lat = randn((sum(new), 576), 2)
    q = randn((sum(new), H, 192), 3)
    kv = cp.cp_mla_expand(lat[:, :512], w)
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, C, new, device=DEV)
    o, lse = cp.cp_mla_prefill_attn(plan, q, kv, lat[:, 512:], scale)
    append([0] * B, new, lat)
    cp.cp_device_error_check()
    K, V = oracle.mla_expanded_qkv(oracle.mla_expand(np64(lat[:, :512]), nw), np64(lat[:, 512:]))
    ref_plan = oracle.zigzag_plan(new, [0] * B, C)
    ref = oracle.prefill_reference(ref_plan, new, [0] * B, np64(q), K, V, scale)
    got = np64(o)
    for r in range(C):
        # keys and values carry a rounding to bf16 that the plain form lacks: a score is off by at most
        # 2^-8 scale sum |q k| (about 0.03 here), O by twice that of its values' mean size and by 2^-8 of it
        assert np.abs(got[plan.rank_off[r]:plan.rank_off[r + 1]] - ref[r][1]).max() <= 8e-2
    rows = [stored(lat[s:e]) for s, e in zip(np.cumsum([0, *new[:-1]]), np.cumsum(new))]
    ctx = list(new)
    for t in range(3):
        x, qd = randn((B, 576), 10 + t), randn((B, H, 192), 20 + t)
        append(ctx, [1] * B, x)
        xs = stored(x)
        rows = [np.concatenate([a, xs[b:b + 1]]) for b, a in enumerate(rows)]
        ctx = [c + 1 for c in ctx]
        dplan = cp.cp_decode_plan(C, ctx, device=DEV)
        ql = cp.cp_mla_absorb(qd, w)
        if t == 0:  # the decode checks the table's host copy, which this one does not have yet
            with pytest.raises(ValueError, match="sync_host"):
                cp.cp_decode_attn_paged(dplan, pages, cp.CP_DECODE_MLA, ql, pool, scale_pool=spool, sm_scale=scale)
        op, lp = cp.cp_decode_attn_paged(dplan, pages.sync_host(), cp.CP_DECODE_MLA, ql, pool, scale_pool=spool, sm_scale=scale)
        ol, _ = cp.cp_lse_merge(op, lp)
        out = cp.cp_mla_project(ol, w)
        cp.cp_device_error_check()
        for b in range(B):
            s = np.einsum("hd,td->ht", np64(ql[b]), rows[b]) * scale
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            lat_out = p @ rows[b][:, :512]
            want = oracle.mla_project(lat_out[None], nw)[0]
            # the decode's bound on a latent dim (2e-2, FP8 6e-2) stands for a row of w, of norm
            # about 1, over independent dims; then the latent output's and the result's roundings
            tol = (6e-2 if fp8 else 2e-2) + 2.0 ** -8 * (np.abs(want) + 2)
            close(out[b], want, tol, f"step {t} request {b}")
