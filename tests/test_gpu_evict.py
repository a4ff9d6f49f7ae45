"""Accumulated attention weights and eviction by them.

Weights: a score is off by at most 2^-20 of the sum of its products' magnitudes
(products exact, sums in fp32; an E4M3 cache's query enters as two E4M3 numbers
that keep 2^-18 of the row's largest element), the given log-sum-exp rounds to 2^-23
of itself in other units, an exponential to 2^-22, and the sum of n terms of one
sign to less than 2^-18 of itself.  Choices and moves are exact.
"""

import math

import numpy as np
import pytest
import torch

from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import gen, randn

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(list(x), **I32)


def shard_rows(L, C, r):
    return len(range(r, max(L, 0), C))


# ------------------------------------------------------------------ weights of prompts

def prompt_weights(plan_rows, new, pre, q, k, lse, scale, window):
    """(weights in 64 bits, relative tolerance): lse rank-major, plan_rows[f] its row."""
    G = q.shape[1] // k.shape[1]
    w, size, q0, k0 = torch.zeros(k.shape[0], dtype=torch.float64, device=DEV), 0.0, 0, 0
    for n, p in zip(new, pre):
        first = max(0, n - window) if window else 0
        K = k[k0:k0 + n + p].double()
        for h in range(q.shape[1]):
            Q = q[q0 + first:q0 + n, h].double()
            x = Q @ K[:, h // G].T * scale
            if x.numel():
                size = max(size, float((Q.abs() @ K[:, h // G].abs().T).max()) * scale)
            l = lse[plan_rows[q0 + first:q0 + n], h].double()[:, None]
            e = torch.where(l == -math.inf, 0.0, (x - l).exp())
            w[k0:k0 + n + p] += torch.tril(e, p + first).sum(0)
        q0, k0 = q0 + n, k0 + n + p
    top = float(lse[lse > -math.inf].abs().max()) if (lse > -math.inf).any() else 0.0
    return w, 2.0**-18 + 2.0**-20 * size + 2.0**-22 * top


def rows_of_plan(plan):
    idx = plan.device_maps()[0].long()
    rows = torch.empty_like(idx)
    rows[idx] = torch.arange(idx.numel(), device=idx.device)
    return rows


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64), (torch.float32, 96)])
@pytest.mark.parametrize("window", [0, 1, 50])
@pytest.mark.parametrize("zigzag,C,new,pre,Hq,Hkv", [
    (True, 1, [1], [0], 1, 1), (True, 4, [300, 1, 0, 7], [0, 500, 40, 129], 8, 2), (False, 3, [129, 257, 5], [1, 0, 333], 6, 2),
    (False, 8, [3, 700], [0, 64], 4, 4), (True, 2, [513], [1000], 12, 1)])
def test_prefill_weights(cp, dtype, D, window, zigzag, C, new, pre, Hq, Hkv):
    g = gen(sum(new) + D)
    T, KV = sum(new), sum(new) + sum(pre)
    q, k, v = randn(g, (T, Hq, D), dtype), randn(g, (KV, Hkv, D), dtype), randn(g, (KV, Hkv, D), dtype)
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG if zigzag else cp.CP_INTERLEAVE, C, new, pre, device=DEV)
    lse = cp.cp_prefill_attn(plan, q, k, v)[1]
    if C == 3:
        lse[5] = -math.inf  # a row that is no query
    got = cp.cp_prefill_weights(plan, q, k, lse, window=window)
    cp.cp_device_error_check()
    want, rel = prompt_weights(rows_of_plan(plan), new, pre, q, k, lse, 1 / math.sqrt(D), window)
    if dtype == torch.float32:
        rel += 2.0**-18  # products rounded, too
    assert ((got.double() - want).abs() <= rel * want + 1e-30).all(), float(((got - want).abs() / want.clamp(min=1e-20)).max())
    if not window and C != 3 and dtype == torch.bfloat16:  # every query spreads a weight of 1 a head
        assert abs(float(got.double().sum()) - T * Hq) <= (rel + 2.0**-10) * T * Hq


def test_prefill_weights_of_a_long_prompt(cp):
    """Work cut over all SMs in the middle of key blocks; the same sums again."""
    g, new, pre, Hq, Hkv, D = gen(3), [5000, 33], [700, 0], 8, 2, 128
    T, KV = sum(new), sum(new) + sum(pre)
    q, k = randn(g, (T, Hq, D)), randn(g, (KV, Hkv, D))
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 8, new, pre, device=DEV)
    lse = cp.cp_prefill_attn(plan, q, k, k)[1]
    got = cp.cp_prefill_weights(plan, q, k, lse)
    again = cp.cp_prefill_weights(plan, q, k, lse)
    cp.cp_device_error_check()
    want, rel = prompt_weights(rows_of_plan(plan), new, pre, q, k, lse, 1 / math.sqrt(D), 0)
    assert ((got.double() - want).abs() <= rel * want).all()
    assert torch.equal(got, again)


@pytest.mark.parametrize("window", [0, 40])
def test_prefill_weights_of_a_request_beside_nan(cp, window):
    """Queries and keys of other requests are not mixed in."""
    g, new, pre = gen(4), [150, 77, 300], [30, 0, 11]
    q, k = randn(g, (sum(new), 8, 64)), randn(g, (sum(new) + sum(pre), 2, 64))
    plan = cp.cp_shard_plan(cp.CP_INTERLEAVE, 3, new, pre, device=DEV)
    lse = cp.cp_prefill_attn(plan, q, k, k)[1]
    want = cp.cp_prefill_weights(plan, q, k, lse, window=window)
    q[150:227], k[180:257] = math.nan, math.nan
    got = cp.cp_prefill_weights(plan, q, k, lse, window=window)
    assert torch.equal(got[:180], want[:180]) and torch.equal(got[257:], want[257:]) and got[180:257].isnan().any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window,at", [(0, 200), (0, 128), (50, 280)])
def test_prefill_weights_of_a_query_that_is_nan(cp, window, at, dtype):
    """A NaN query spoils the keys that it reads (unless the attention itself gave it LSE
    -inf, as its fp32 form does: then it weighs nothing), not the later ones."""
    g, new, pre = gen(5), 300, 20
    q, k = randn(g, (new, 8, 64)).to(dtype), randn(g, (new + pre, 2, 64)).to(dtype)
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [new], [pre], device=DEV)
    lse = cp.cp_prefill_attn(plan, q, k, k)[1]
    want = cp.cp_prefill_weights(plan, q, k, lse, window=window)
    q[at] = math.nan
    lse = cp.cp_prefill_attn(plan, q, k, k)[1]
    got = cp.cp_prefill_weights(plan, q, k, lse, window=window)
    assert lse.isnan().any() or (lse == -math.inf).any()
    reads = got[:pre + at + 1].isnan()
    assert reads.all() if lse.isnan().any() else not reads.any()
    assert torch.equal(got[pre + at + 1:], want[pre + at + 1:])


def test_prefill_weights_of_nothing(cp):
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [0, 0], [70, 0], device=DEV)
    k = randn(gen(1), (70, 2, 64))
    got = cp.cp_prefill_weights(plan, torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV), k, torch.empty((0, 4), device=DEV),
                                out=torch.full((70,), 5.0, device=DEV))
    assert not got.any()


# ------------------------------------------------------------------ weights of decode steps

class Pool:
    """A paged cache of `ctx` tokens a request over C shards, pages shuffled."""

    def __init__(self, cp, C, ctx, row, page=64, dtype=torch.bfloat16, seed=1, spare=6, layout=0, s_q=1):
        self.cp, self.C, self.ctx, self.page = cp, C, ctx, page
        g, rng = gen(seed), np.random.default_rng(seed)
        need = [-(-shard_rows(L, C, r) // page) for r in range(C) for L in ctx]
        ids = rng.permutation(sum(need) + spare).astype(np.int32)
        table = np.full((len(need), max(1, max(need)) + 1), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:]
        self.table = table
        self.pages = cp.PageTable(table, page, len(ids), device=DEV)
        rows = self.pages.pool_rows
        self.scale = None
        if dtype == torch.float8_e4m3fn:
            self.k, self.v = (randn(g, (rows, *row), torch.float32, 20.0).clamp(-448, 448).to(dtype) for _ in range(2))
            self.scale = torch.rand(rows, generator=g, device=DEV) * 0.04 + 0.01
        else:
            self.k, self.v = randn(g, (rows, *row), dtype), randn(g, (rows, *row), dtype)
        self.w = torch.rand(rows, generator=g, device=DEV)
        self.plan = cp.cp_decode_plan_ex(C, ctx, layout=layout, s_q=s_q, device=DEV)

    def rows(self, b, r):
        """Pool rows of request b's pair on shard r."""
        i = np.arange(shard_rows(self.ctx[b], self.C, r))
        return self.table[r * len(self.ctx) + b, i // self.page].astype(np.int64) * self.page + i % self.page


@pytest.mark.parametrize("C,ctx,Hq,Hkv,D,kv,s_q,page", [
    (1, [1], 1, 1, 128, "bf16", 1, 64), (2, [300, 0, 129], 8, 2, 128, "bf16", 1, 64), (3, [64, 700], 8, 2, 64, "bf16", 1, 192),
    (2, [500, 40], 32, 8, 128, "fp8", 1, 64), (8, [1000, 3], 64, 1, 576, "bf16", 1, 64), (2, [700, 129], 64, 1, 576, "fp8", 1, 128),
    (2, [333], 20, 1, 576, "fp8", 3, 64), (2, [200, 9], 8, 2, 128, "bf16", 4, 64), (4, [300], 5, 1, 576, "bf16", 1, 64),
    (2, [300, 7], 8, 8, 96, "bf16", 1, 64), (1, [260], 4, 2, 128, "fp32", 2, 64), (2, [150], 8, 2, 64, "fp8", 1, 64),
    (1, [400], 64, 64, 128, "bf16", 1, 64), (2, [300, 200], 6, 2, 128, "bf16", 1, 64)])
def test_decode_weights(cp, C, ctx, Hq, Hkv, D, kv, s_q, page):
    mla = D == 576
    dtype = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "fp32": torch.float32}[kv]
    p = Pool(cp, C, ctx, (D,) if mla else (Hkv, D), page, dtype, seed=sum(ctx), s_q=s_q)
    g = gen(9)
    lead = (len(ctx), s_q) if s_q > 1 else (len(ctx),)
    q = randn(g, (*lead, Hq, D), torch.float32 if kv == "fp32" else torch.bfloat16, 0.7)
    scale = 1 / math.sqrt(192 if mla else D)
    lse = torch.randn((*lead, Hq), generator=g, device=DEV) + 4
    lse.reshape(-1)[Hq // 2] = -math.inf
    k = p.k.float().double().reshape(p.k.shape[0], Hkv, D)
    if p.scale is not None:
        k = k * p.scale.double()[:, None, None]
    want, size = p.w.double().clone(), 0.0
    named = torch.zeros(want.shape, dtype=torch.bool, device=DEV)
    for b, L in enumerate(ctx):
        for r in range(C):
            at = torch.from_numpy(p.rows(b, r)).to(DEV)
            named[at] = True
            tok = torch.arange(at.numel(), device=DEV) * C + r
            for qi in range(s_q):
                seen = tok <= L - s_q + qi
                qq = q.reshape(len(ctx), s_q, Hq, D)[b, qi].double()
                l = lse.reshape(len(ctx), s_q, Hq)[b, qi].double()
                for h in range(Hq):
                    kk = k[at, h // (Hq // Hkv)]
                    if at.numel():
                        size = max(size, float((kk.abs() @ qq[h].abs()).max()) * scale,
                                   2.0**2 * float(kk.abs().sum(1).max() * qq[h].abs().max()) * scale if kv == "fp8" else 0.0)
                    if l[h] > -math.inf:
                        want[at] += torch.where(seen, (kk @ qq[h] * scale - l[h]).exp(), 0.0)
    before = p.w.clone()
    if kv == "fp8":  # rows that are no request's may hold NaN
        p.k.view(torch.uint8)[~named] = 0x7F
        p.scale[~named] = math.nan
    else:
        p.k[~named] = math.nan
    mode = cp.CP_DECODE_MLA if mla else cp.CP_DECODE_GQA
    got = cp.cp_decode_weights(p.plan, p.pages, mode, q, p.k, lse, p.w, scale_pool=p.scale, sm_scale=scale)
    cp.cp_device_error_check()
    assert got is p.w
    assert torch.equal(got[~named], before[~named])
    rel = 2.0**-18 + 2.0**-20 * size
    assert ((got.double() - want).abs() <= rel * want).all(), float(((got - want).abs() / want).max())


def test_decode_weights_of_the_attention(cp):
    """With the decode's own LSE a step adds a weight of one for each query head."""
    ctx, C, Hq, Hkv, D = [700, 1, 64, 0], 2, 8, 2, 128
    p = Pool(cp, C, ctx, (Hkv, D))
    q = randn(gen(2), (4, Hq, D))
    o, l = cp.cp_decode_attn_paged(p.plan, p.pages, cp.CP_DECODE_GQA, q, p.k, p.v)
    lse = cp.cp_lse_merge(o, l)[1]
    p.w.zero_()
    for steps in (1, 2):  # the second step adds to the first
        cp.cp_decode_weights(p.plan, p.pages, cp.CP_DECODE_GQA, q, p.k, lse, p.w)
        for b, L in enumerate(ctx):
            at = np.concatenate([p.rows(b, r) for r in range(C)])
            assert abs(float(p.w[torch.from_numpy(at).to(DEV)].double().sum()) - (steps * Hq if L else 0)) <= 2.0**-12 * steps * Hq


# ------------------------------------------------------------------ choices and moves

def chosen(p, keep, w, pos, below, start, most):
    """The rule itself, pair by pair: (src, dst, count)."""
    B = len(p.ctx)
    src, dst = (np.full((p.C * B, most), -1, np.int32) for _ in range(2))
    count = np.zeros(p.C * B, np.int32)
    for r in range(p.C):
        for b, L in enumerate(p.ctx):
            at, m = p.rows(b, r), min(shard_rows(L, p.C, r), shard_rows(keep[b], p.C, r))
            where = pos[at] if pos is not None else np.arange(at.size) * p.C + r
            safe = (where < below) | (where >= start[b] if start is not None else False)
            x = w[at].astype(np.float64)  # protected rows come first, by row
            key = [-math.inf if s else math.inf if math.isnan(v) else -v for s, v in zip(safe, x)]  # NaN sorts behind -inf's +inf by the next entry
            rank = sorted(range(at.size), key=lambda i: (not safe[i], not safe[i] and math.isnan(x[i]), key[i], i))
            stay = sorted(rank[:m])
            late, holes = [i for i in stay if i >= m], sorted(set(range(m)) - set(stay))
            pair = r * B + b
            if len(late) > most:
                count[pair] = -1
                continue
            count[pair] = len(late)
            src[pair, :len(late)], dst[pair, :len(late)] = at[late], at[holes]
    return src, dst, count


@pytest.mark.parametrize("kind", ["spread", "ties", "zeros", "special", "negative"])
@pytest.mark.parametrize("C,ctx,keep,page", [
    (1, [1, 2, 70], [1, 1, 64], 64), (2, [300, 0, 129, 64], [100, 5, 200, 0], 64), (3, [2112] * 5, [2048] * 5, 192),
    (8, [5000, 700], [512, 699], 64), (1, [70000], [333], 64), (1, [3000, 1025, 4000], [1000, 1024, 3999], 64),
    (2, [9000, 130], [100, 129], 128)])
def test_evict_select(cp, kind, C, ctx, keep, page):
    p = Pool(cp, C, ctx, (64,), page, seed=C + len(ctx))
    rng = np.random.default_rng(4)
    n = p.w.numel()
    w = np.exp(rng.standard_normal(n) * 4).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, n).astype(np.float32)
    elif kind == "zeros":
        w = np.where(rng.random(n) < 0.9, np.where(rng.random(n) < 0.5, 0.0, -0.0), w).astype(np.float32)
    elif kind == "special":
        w[rng.random(n) < 0.1] = np.inf
        w[rng.random(n) < 0.1] = np.nan
        w[rng.random(n) < 0.1] = -np.inf
        w[rng.random(n) < 0.1] = 1e-42
    elif kind == "negative":
        w = (w - 1).astype(np.float32)
    most = max(1, max(min(shard_rows(k, C, 0), shard_rows(L, C, 0)) for L, k in zip(ctx, keep)))
    for pos, below, start in ((None, 0, None), (None, 4, [max(0, L - 9) for L in ctx]),
                              (rng.permutation(n).astype(np.int32), 20, [n - n // 8] * len(ctx))):
        got = cp.cp_evict_select(p.pages, C, i32(ctx), i32(keep), torch.from_numpy(w).to(DEV), most,
                                 pos=None if pos is None else torch.from_numpy(pos).to(DEV), keep_below=below,
                                 keep_from=None if start is None else i32(start))
        for g, x, what in zip(got, chosen(p, keep, w, pos, below, start, most), ("src", "dst", "count")):
            assert np.array_equal(g.cpu().numpy(), x), what


def test_evict_select_that_does_not_fit(cp):
    p = Pool(cp, 2, [300, 300, 300, 300], (64,))
    w = torch.arange(p.w.numel(), device=DEV).float()
    run = lambda ctx, keep, most=200: [x.cpu().numpy() for x in cp.cp_evict_select(p.pages, 2, i32(ctx), i32(keep), w, most)]  # noqa: E731
    src, dst, count = run([300, -1, 300, 100000], [100, 100, -5, 100])
    assert count[1] == count[2] == count[3] == -1 and count[5] == count[7] == -1 and count[0] >= 0
    assert (src[[1, 2, 3]] == -1).all() and (dst[[1, 2, 3]] == -1).all()
    need = run([300] * 4, [100] * 4)[2]
    few = int(need.min()) if need.min() > 0 else 1
    src, dst, count = run([300] * 4, [100] * 4, few)
    assert all((c == n) if n <= few else c == -1 for c, n in zip(count, need))
    p.pages.dev[0, 1] = p.pages.num_pages  # a page that is not there
    p.pages.dev[1, 0] = -7
    count = run([300] * 4, [100] * 4)[2]
    assert count[0] == count[1] == -1 and (count[2:] >= 0).all()


@pytest.mark.parametrize("row,dtype", [((8, 128), torch.bfloat16), ((576,), torch.float8_e4m3fn), ((2, 64), torch.float32), ((16,), torch.uint8), ((5, 600), torch.bfloat16)])
def test_cache_move(cp, row, dtype):
    rows, pairs, most = 4000, 5, 300
    rng = np.random.default_rng(1)
    ids = rng.permutation(rows)[:2 * pairs * most].astype(np.int32) if rows >= 2 * pairs * most else rng.permutation(rows).astype(np.int32)
    src, dst = ids[0::2][:pairs * most].reshape(pairs, most).copy(), ids[1::2][:pairs * most].reshape(pairs, most).copy()
    count = np.array([300, 0, 7, -1, 129], np.int32)
    src[4, 5], dst[4, 9] = rows, -1  # rows outside the pool
    make = lambda: torch.randint(0, 255, (rows, int(np.prod(row)) * torch.empty(0, dtype=dtype).element_size()), dtype=torch.uint8, generator=gen(3), device=DEV)  # noqa: E731
    k, v, w = make(), make().flip(0), torch.rand(rows, device=DEV)
    pos, sc = torch.arange(rows, **I32), torch.rand(rows, device=DEV)
    view = lambda x: x.view(dtype).reshape(rows, *row)  # noqa: E731
    moves = [(s, d) for i, c in enumerate(count) for s, d in zip(src[i, :max(c, 0)], dst[i, :max(c, 0)]) if 0 <= s < rows and 0 <= d < rows]
    a, b = (torch.tensor([int(m[i]) for m in moves], device=DEV) for i in range(2))
    want = []
    for x in (k, v, sc, w, pos):
        y = x.clone()
        y[b] = x[a]
        want.append(y)
    t = [torch.from_numpy(x).to(DEV) for x in (src, dst, count)]
    one = k.clone()
    cp.cp_cache_move(*t, view(one))
    assert torch.equal(one, want[0])
    cp.cp_cache_move(*t, view(k), view(v), sc, w, pos)
    for x, y in zip((k, v, sc, w, pos), want):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ pages back

def released(p, ctx, keep, free, at):
    """(table, free list, info, pool rows that are cleared) by the rule."""
    table, free, out, clear = p.table.copy(), free.copy(), [], []
    B = len(ctx)
    for b in range(B):
        for r in range(p.C):
            n, m = shard_rows(ctx[b], p.C, r), min(shard_rows(ctx[b], p.C, r), shard_rows(keep[b], p.C, r))
            if keep[b] >= ctx[b]:
                continue
            for i in range(m // p.page, -(-n // p.page)):
                ident = table[r * B + b, i]
                clear += [ident * p.page + x for x in range(p.page) if i * p.page + x >= m]
                if i >= -(-m // p.page):
                    out.append(ident)
                    table[r * B + b, i] = -1
    free[at - len(out):at] = out
    return table, free, [0, at - len(out), len(out), 0], clear


@pytest.mark.parametrize("C,ctx,keep,page", [
    (1, [300], [0], 64), (2, [300, 0, 129, 64, 500], [100, 5, 200, 64, 1], 64), (8, [5000, 700, 1], [512, 699, 0], 64), (3, [577, 576], [576, 193], 192),
    (64, [5000] * 70, [4000] * 70, 64)])
def test_page_release(cp, C, ctx, keep, page):
    p = Pool(cp, C, ctx, (16,), page)
    total = int(sum((p.table >= 0).sum(1)))
    free, at = np.concatenate([np.full(total, 7777, np.int32), p.free]), total
    want = released(p, ctx, keep, free, at)
    t, w, pos = torch.from_numpy(free.copy()).to(DEV), p.w.clone(), torch.arange(p.w.numel(), **I32)
    info = cp.cp_page_release(p.pages, C, i32(ctx), i32(keep), t, i32([at]), w, pos)
    assert info.tolist() == want[2] and p.pages.host is None
    assert np.array_equal(t.cpu().numpy(), want[1]) and np.array_equal(p.pages.dev.cpu().numpy(), want[0])
    mask = torch.zeros(w.numel(), dtype=torch.bool, device=DEV)
    mask[torch.tensor(want[3], dtype=torch.long, device=DEV)] = True
    assert torch.equal(w, torch.where(mask, 0.0, p.w)) and torch.equal(pos, torch.where(mask, -1, torch.arange(w.numel(), **I32)))
    # the step after it takes the same pages again
    slots, _, again = cp.cp_page_slots(p.pages, C, i32([min(a, b) for a, b in zip(ctx, keep)]), i32([max(0, a - b) for a, b in zip(ctx, keep)]),
                                       t, info[1:2], sum(max(0, a - b) for a, b in zip(ctx, keep)))
    assert again[0].item() == 0 and again[1].item() == at and (slots >= 0).all()


@pytest.mark.parametrize("case", ["negative", "table", "room", "pos"])
def test_page_release_that_does_not_fit(cp, case):
    p = Pool(cp, 2, [300, 500], (16,))
    ctx, keep, at = [300, 500], [10, 10], 40
    if case == "negative":
        keep = [-1, 10]
    elif case == "table":
        ctx = [300, 100000]
    elif case == "room":
        at = 3
    else:
        at = 99
    t, w, before = torch.full((50,), 5, **I32), p.w.clone(), p.pages.dev.clone()
    info = cp.cp_page_release(p.pages, 2, i32(ctx), i32(keep), t, i32([at]), w)
    assert info[0].item() == {"negative": 1, "table": 2 + (4 if case == "table" and info[0].item() & 4 else 0), "room": 4, "pos": 4}[case]
    assert info.tolist()[1:] == [at, 0, 0] and (t == 5).all() and torch.equal(w, p.w) and torch.equal(before, p.pages.dev)


# ------------------------------------------------------------------ all of them, as a serving loop uses them

@pytest.mark.parametrize("C", [1, 2])
def test_rotate_attend_weigh_evict(cp, C):
    """Steps of a batch behind a shared prefix whose own caches are held at a
    budget: rotated keys enter pages, prefix and own tokens are attended to,
    weights pile up, the lightest tokens go, their pages come back.  Every step
    against a plain model of the caches in 64 bits."""
    B, Hq, Hkv, D, P, page, budget, room = 3, 8, 2, 128, 200, 64, 70, 90
    g, scale = gen(11), 1 / math.sqrt(128)
    freqs = cp.cp_rope_freqs(D, device=DEV)
    kp, vp = randn(g, (P, Hkv, D)), randn(g, (P, Hkv, D))
    kp = cp.cp_rope(kp, None, torch.arange(P, **I32), freqs)[0]
    pack = cp.cp_decode_plan(C, [P], device=DEV)
    sk, sv = cp.cp_kv_shard_pack(pack, kp)[0], cp.cp_kv_shard_pack(pack, vp)[0]
    pplan = cp.cp_prefix_plan(C, [P], [B], Hq, Hkv, device=DEV)
    num = 40
    pages = cp.PageTable.on_device(torch.full((C * B, 4), -1, **I32), page, num)
    free, at = torch.arange(num, **I32), torch.zeros(1, **I32)
    pool_k, pool_v = (torch.zeros((num * page, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    w, pos = torch.zeros(num * page, device=DEV), torch.full((num * page,), -1, **I32)
    model = [dict(k=[], v=[], w=[], pos=[]) for _ in range(B)]  # by request, in row order of all shards: token i on shard i % C
    seen, have = [P] * B, [0] * B
    for new in ([40, 3, 60], [30, 40, 30], [1, 50, 1], [1, 1, 1]):
        T = sum(new)
        kn, vn = randn(g, (T, Hkv, D)), randn(g, (T, Hkv, D))
        where = i32([seen[b] + i for b in range(B) for i in range(new[b])])
        q = randn(g, (B, Hq, D))
        q, _ = cp.cp_rope(q, None, i32([s + n - 1 for s, n in zip(seen, new)]), freqs)
        kn, _ = cp.cp_rope(kn, None, where, freqs)
        slots, _, info = cp.cp_page_slots(pages, C, i32(have), i32(new), free, at, T)
        assert info[0].item() == 0 and (slots >= 0).all()
        at = info[1:2].clone()
        cp.cp_cache_append(slots, kn, pool_k, vn, pool_v)
        pos[slots.long()] = where
        assert not w[slots.long()].any()  # new rows start at weight 0
        t = 0
        for b in range(B):
            m = model[b]
            for i in range(new[b]):
                m["k"].append(kn[t + i].double())
                m["v"].append(vn[t + i].double())
                m["w"].append(0.0)
                m["pos"].append(seen[b] + i)
            t += new[b]
            seen[b] += new[b]
            have[b] += new[b]
        plan = cp.cp_decode_plan(C, have, device=DEV)
        o_part, lse_part = cp.cp_decode_attn_paged(plan, pages.sync_host(), cp.CP_DECODE_GQA, q, pool_k, pool_v, sm_scale=scale)
        o, lse = cp.cp_prefix_attn(pplan, q, sk, sv, sm_scale=scale, o_part=o_part, lse_part=lse_part, out_dtype=torch.float32)
        cp.cp_decode_weights(plan, pages, cp.CP_DECODE_GQA, q, pool_k, lse, w, sm_scale=scale)
        cp.cp_device_error_check()
        host = pages.host.copy()
        row = lambda b, i: int(host[(i % C) * B + b, i // C // page]) * page + i // C % page  # noqa: E731
        for b in range(B):
            m = model[b]
            for h in range(Hq):
                k = torch.cat([kp[:, h // 4].double(), torch.stack(m["k"])[:, h // 4]])
                v = torch.cat([vp[:, h // 4].double(), torch.stack(m["v"])[:, h // 4]])
                x = k @ q[b, h].double() * scale
                prob = torch.softmax(x, 0)
                assert ((o[b, h].double() - prob @ v).abs() <= 2.0**-7 * (prob @ v.abs()) + 1e-5).all()
                for i in range(have[b]):
                    m["w"][i] += float(prob[P + i])
            got = torch.stack([w[row(b, i)] for i in range(have[b])]).double().cpu()
            assert ((got - torch.tensor(m["w"], dtype=torch.float64)).abs() <= 1e-4 * got + 1e-6).all()
            assert [int(pos[row(b, i)]) for i in range(have[b])] == m["pos"]
            m["w"] = got.tolist()  # the rule below chooses by the weights that are there
        keep = [min(n, budget) if n > room else n for n in have]
        start = [s - 5 for s in seen]
        src, dst, count = cp.cp_evict_select(pages, C, i32(have), i32(keep), w, 128, pos=pos, keep_from=i32(start))
        cp.cp_cache_move(src, dst, count, pool_k, pool_v, weights=w, pos=pos)
        info = cp.cp_page_release(pages, C, i32(have), i32(keep), free, at, w, pos)
        assert info[0].item() == 0 and (count >= 0).all()
        at = info[1:2].clone()
        for b in range(B):
            if keep[b] == have[b]:
                continue
            m, new_rows = model[b], {}
            for r in range(C):
                idx = list(range(r, have[b], C))
                n_keep = shard_rows(keep[b], C, r)
                best = sorted(idx, key=lambda i: (m["pos"][i] < start[b], -m["w"][i], i))[:n_keep]
                stay = sorted(best)
                front, late = [i for i in stay if i < n_keep * C + r], [i for i in stay if i >= n_keep * C + r]
                holes = [i for i in idx[:n_keep] if i not in front]
                for i in front:
                    new_rows[i] = i
                for i, j in zip(holes, late):
                    new_rows[i] = j
            for key in m:
                m[key] = [m[key][new_rows[i]] for i in range(keep[b])]
            have[b] = keep[b]
    assert max(have) <= room + 1


# ------------------------------------------------------------------ streams, graphs, waits

def replay(fn, *reset):
    """fn captured and replayed once, after `reset` is put back."""
    keep = [x.clone() for x in reset]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = fn()
        for x, y in zip(reset, keep):
            x.copy_(y)
        g.replay()
    side.synchronize()
    return out


def test_weights_and_eviction_replayed(cp):
    """Captured calls give the eager ones' results bit for bit."""
    ctx, C, Hq, Hkv, D = [700, 300], 2, 8, 2, 128
    p = Pool(cp, C, ctx, (Hkv, D))
    q, lse = randn(gen(2), (2, Hq, D)), torch.full((2, Hq), 5.0, device=DEV)
    w0 = p.w.clone()
    run = lambda: cp.cp_decode_weights(p.plan, p.pages, cp.CP_DECODE_GQA, q, p.k, lse, p.w)  # noqa: E731
    want = run().clone()
    p.w.copy_(w0)
    assert torch.equal(replay(run, p.w), want)
    new, pre = [300, 5], [40, 0]
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, new, pre, device=DEV)
    qq, kk = randn(gen(3), (305, Hq, D)), randn(gen(4), (345, Hkv, D))
    ll = cp.cp_prefill_attn(plan, qq, kk, kk)[1]
    want = cp.cp_prefill_weights(plan, qq, kk, ll)
    assert torch.equal(replay(lambda: cp.cp_prefill_weights(plan, qq, kk, ll)), want)
    old, keep = i32(ctx), i32([100, 300])
    at, free = i32([20]), torch.full((30,), -5, **I32)
    k0, t0 = p.k.clone(), p.pages.dev.clone()

    def step():
        src, dst, count = cp.cp_evict_select(p.pages, C, old, keep, p.w, 60)
        cp.cp_cache_move(src, dst, count, p.k, p.v)
        return src, dst, count, cp.cp_page_release(p.pages, C, old, keep, free, at)

    v0 = p.v.clone()
    want = [x.clone() for x in step()] + [p.k.clone(), p.v.clone(), p.pages.dev.clone(), free.clone()]
    for x, y in ((p.k, k0), (p.v, v0), (p.pages.dev, t0)):
        x.copy_(y)
    free.fill_(-5)
    got = list(replay(step, p.k, p.v, p.pages.dev, free)) + [p.k, p.v, p.pages.dev, free]
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_weights_on_two_streams(cp):
    """Two prompts' weights at once, each with a workspace of its own."""
    jobs = []
    for seed, new in ((1, [900, 70]), (2, [33, 500, 1])):
        plan = cp.cp_shard_plan(cp.CP_INTERLEAVE, 3, new, device=DEV)
        q, k = randn(gen(seed), (sum(new), 8, 64)), randn(gen(seed + 5), (sum(new), 2, 64))
        lse = cp.cp_prefill_attn(plan, q, k, k)[1]
        jobs.append((plan, q, k, lse, cp.cp_prefill_weights(plan, q, k, lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for s, (plan, q, k, lse, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(cp.cp_prefill_weights(plan, q, k, lse))
        torch.cuda.synchronize()
        for g, j in zip(got, jobs):
            assert torch.equal(g, j[4])


@pytest.mark.parametrize("kind", ["prompt", "short", "step", "latent"])
def test_weights_wait_that_runs_out(cp, monkeypatch, kind):
    """The issuer waits for a barrier that nothing arrives at: the kernel gives up,
    drains and returns, and the next call is right."""
    if kind in ("prompt", "short"):
        new = [6000 if kind == "prompt" else 90]
        plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, new, device=DEV)
        q, k = randn(gen(1), (new[0], 4, 64)), randn(gen(2), (new[0], 2, 64))
        lse = cp.cp_prefill_attn(plan, q, k, k)[1]
        run = lambda: cp.cp_prefill_weights(plan, q, k, lse)  # noqa: E731
    else:
        p = Pool(cp, 2, [700, 300], (576,) if kind == "latent" else (2, 64), dtype=torch.float8_e4m3fn if kind == "latent" else torch.bfloat16)
        q, lse = randn(gen(2), (2, 8, 576 if kind == "latent" else 64)), torch.full((2, 8), 9.0, device=DEV)
        mode = cp.CP_DECODE_MLA if kind == "latent" else cp.CP_DECODE_GQA
        run = lambda: cp.cp_decode_weights(p.plan, p.pages, mode, q, p.k, lse, torch.zeros_like(p.w), scale_pool=p.scale, sm_scale=0.05)  # noqa: E731
    cp.cp_device_error_check()
    want = run()
    monkeypatch.setenv("CPATTN_TEST_STALL", "1")
    run()
    with pytest.raises(cp.CpError) as ei:
        cp.cp_device_error_check()
    assert ei.value.status == -4
    monkeypatch.delenv("CPATTN_TEST_STALL")
    assert torch.equal(run(), want)
    cp.cp_device_error_check()


def test_weights_and_moves_past_31_bits(cp):
    """A pool whose last rows lie behind 2^31 elements."""
    page, row = 64, (8, 128)
    num = 2**31 // (1024 * page) + 2
    k = torch.zeros((num * page, *row), dtype=torch.bfloat16, device=DEV)
    table = np.array([[0, num - 1]], np.int32)
    pages = cp.PageTable(table, page, num, device=DEV)
    k[-page:] = randn(gen(1), (page, *row))
    last = k[-page:].clone()
    q, lse, w = randn(gen(2), (1, 8, 128)), torch.full((1, 8), 3.0, device=DEV), torch.zeros(num * page, device=DEV)
    plan = cp.cp_decode_plan(1, [100], device=DEV)
    cp.cp_decode_weights(plan, pages, cp.CP_DECODE_GQA, q, k, lse, w)
    cp.cp_device_error_check()
    x = torch.einsum("hd,khd->kh", q[0].double(), last.double()) / math.sqrt(128) - 3
    want = x.exp().sum(1)[:36]
    size = float(torch.einsum("hd,khd->kh", q[0].double().abs(), last.double().abs()).max()) / math.sqrt(128)
    assert ((w[-page:-page + 36].double() - want).abs() <= (2.0**-18 + 2.0**-20 * size) * want).all()
    w[:] = 0
    w[-page:-page + 36] = 1
    src, dst, count = cp.cp_evict_select(pages, 1, i32([100]), i32([36]), w, 36)
    assert count.item() == 36 and src[0, 0].item() == (num - 1) * page and dst[0, 35].item() == 35
    cp.cp_cache_move(src, dst, count, k, weights=w)
    assert torch.equal(k[:36], last[:36]) and bool((w[:36] == 1).all())
