"""Attention over shared prefixes against the definition in 64 bits.

Tolerances, before any run.  Scores: products of bf16 (or E4M3 times a scale)
summed in fp32, off by at most 2^-20 of the sum of the products' magnitudes, and
that is the log-sum-exp's error plus 2^-20 of it.  O: the softmax weights are
rounded to bf16 on the tensor cores (2^-8 of each, so 2^-8 of sum p |v|), the
result to bf16 (2^-8 of itself) or not at all (fp32), and the score's error
enters every weight twice.
"""

import math

import numpy as np
import pytest
import torch

from test_gpu_parity import DEV, cp  # noqa: F401

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


class Case:
    """Prefixes in token order, their shards or pages, queries and own parts."""

    def __init__(self, cp, C, lens, members, Hq, Hkv, D, kv="bf16", layout=0, page=0, P=0, workers=0, seed=1, std=1.0):
        g = gen(seed)
        self.cp, self.C, self.lens, self.members, self.G, self.D, self.kv = cp, C, lens, members, Hq // Hkv, D, kv
        N, T = sum(members), sum(lens)
        self.dtype = torch.float32 if kv == "fp32" else torch.bfloat16
        self.q = randn(g, (N, Hq, D), self.dtype, std)
        if kv == "fp8":
            self.k, self.v = (randn(g, (T, Hkv, D), torch.float32, 20.0).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
            self.scale = torch.rand(T, generator=g, device=DEV) * 0.05 + 0.01
        else:
            self.k, self.v, self.scale = randn(g, (T, Hkv, D), self.dtype), randn(g, (T, Hkv, D), self.dtype), None
        self.dplan = cp.cp_decode_plan_ex(C, lens, layout=layout, device=DEV)
        self.plan = cp.cp_prefix_plan(C, lens, members, Hq, Hkv, layout, workers, device=DEV)
        self.P = P
        self.own = {}
        if P:
            o, l = torch.randn((P, N, Hq, D), generator=g, device=DEV), torch.randn((P, N, Hq), generator=g, device=DEV) * 2
            l[:, ::3] = -math.inf  # rows without tokens of their own, some in one part only
            l[0, ::2] = -math.inf
            o[l == -math.inf] = math.nan  # such a part is not read
            self.own = dict(o_part=o, lse_part=l)
        if page:
            need = [-(-int(r) // page) for r in self.plan.pairs[:, 0]]
            ids = np.random.default_rng(seed).permutation(sum(need) + 3)
            table = np.full((len(need), max(1, max(need))), -1, np.int32)
            at = 0
            for i, n in enumerate(need):
                table[i, :n] = ids[at:at + n]
                at += n
            self.pages = cp.PageTable(table, page, len(ids), device=DEV)
            pool = lambda x: torch.full((self.pages.pool_rows, *x.shape[1:]), 7.0, device=DEV).to(x.dtype)  # noqa: E731
            pk = cp.cp_kv_shard_pack_paged(self.dplan, self.pages, self.k, self.scale, pool(self.k).view(torch.uint8) if kv == "fp8" else pool(self.k))
            pv = cp.cp_kv_shard_pack_paged(self.dplan, self.pages, self.v, None, pool(self.v).view(torch.uint8) if kv == "fp8" else pool(self.v))
            self.pool = (pk[0], pv[0], pk[1])
        else:
            self.pages = None
            (self.sk, self.sc), (self.sv, _) = cp.cp_kv_shard_pack(self.dplan, self.k, self.scale), cp.cp_kv_shard_pack(self.dplan, self.v)

    def run(self, **kw):
        if self.pages:
            return self.cp.cp_prefix_attn_paged(self.plan, self.pages, self.q, *self.pool, **self.own, **kw)
        return self.cp.cp_prefix_attn(self.plan, self.q, self.sk, self.sv, self.sc, **self.own, **kw)

    def check(self, o, lse):
        scale = 1 / math.sqrt(self.D)
        K, V = self.k.float().double(), self.v.float().double()
        if self.scale is not None:
            K, V = (x * self.scale.double()[:, None, None] for x in (K, V))
        q0 = t0 = 0
        for n, L in zip(self.members, self.lens):
            for h in range(self.q.shape[1]):
                q, k, v = self.q[q0:q0 + n, h].double(), K[t0:t0 + L, h // self.G], V[t0:t0 + L, h // self.G]
                x = q @ k.T * scale
                size = float((q.abs() @ k.abs().T).max() * scale) if n and L else 0.0
                ls, os = [torch.logsumexp(x, 1)], [torch.softmax(x, 1) @ v if L else torch.zeros_like(q)]
                mag = torch.softmax(x, 1) @ v.abs() if L else torch.zeros_like(q)
                for p in range(self.P):
                    ls.append(self.own["lse_part"][p, q0:q0 + n, h].double())
                    os.append(torch.nan_to_num(self.own["o_part"][p, q0:q0 + n, h].double()))
                ls = torch.stack(ls)
                total = torch.logsumexp(ls, 0)
                w = torch.nan_to_num((ls - total).exp(), nan=0.0)
                want = (w[..., None] * torch.stack(os)).sum(0)
                mag = w[0][:, None] * mag + (w[1:, :, None] * torch.stack(os)[1:].abs()).sum(0)
                ds = 2.0**-20 * (size + 1)
                got_l, got_o = lse[q0:q0 + n, h].double(), o[q0:q0 + n, h].double()
                assert torch.equal(got_l == -math.inf, total == -math.inf)
                fin = total > -math.inf
                assert ((got_l - total)[fin].abs() <= ds + 2.0**-20 * total[fin].abs()).all(), f"LSE of head {h}"
                tol = (2.0**-8 + 4 * ds) * mag + (2.0**-8 * want.abs() if o.dtype == torch.bfloat16 else 0) + 2.0**-20
                bad = (got_o - want).abs() > tol
                assert not bad.any(), f"O of head {h}: {int(bad.sum())} off, {float((got_o - want).abs().max())}"
            q0, t0 = q0 + n, t0 + L


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp32", 128), ("bf16", 96), ("fp8", 64), ("fp32", 32), ("bf16", 256)])
@pytest.mark.parametrize("C,lens,members,Hq,Hkv", [
    (1, [1], [1], 1, 1), (2, [300], [5], 8, 2), (3, [129, 0, 700], [3, 4, 0], 6, 2), (8, [5, 1000], [70, 1], 8, 2), (1, [257], [300], 4, 4)])
def test_prefix(cp, kv, D, C, lens, members, Hq, Hkv):
    c = Case(cp, C, lens, members, Hq, Hkv, D, kv, workers=5, P=C % 3)
    o, lse = c.run(out_dtype=torch.float32 if C == 2 else torch.bfloat16)
    cp.cp_device_error_check()
    c.check(o, lse)


@pytest.mark.parametrize("workers", [1, 7, 152, 400])
@pytest.mark.parametrize("P", [0, 2])
def test_prefix_cut_over_workers(cp, workers, P):
    """Blocks of one and two M tiles, whole and in parts."""
    c = Case(cp, 3, [3000, 40, 900], [40, 17, 130], 16, 4, 128, workers=workers, P=P)
    o, lse = c.run()
    cp.cp_device_error_check()
    c.check(o, lse)


@pytest.mark.parametrize("kv,D,page", [("bf16", 128, 64), ("bf16", 64, 192), ("bf16", 128, 128), ("fp8", 128, 64), ("fp32", 64, 64)])
def test_prefix_paged(cp, kv, D, page):
    c = Case(cp, 2, [1, 700, 0, 129], [3, 40, 2, 1], 8, 2, D, kv, page=page, P=1, workers=9)
    o, lse = c.run()
    cp.cp_device_error_check()
    c.check(o, lse)


def test_prefix_contiguous_chunks(cp):
    c = Case(cp, 4, [1001, 3], [20, 6], 8, 2, 128, layout=cp.CP_DCP_CONTIGUOUS, workers=11)
    c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_of_rising_and_large_scores(cp, D):
    """Running maxima that move at every tile, in both directions, and scores of
    hundreds: the sums stay those of the definition."""
    c = Case(cp, 1, [1500], [70], 4, 2, D, workers=2)
    c.q.copy_(torch.nn.functional.normalize(torch.randn(c.q.shape, generator=gen(3), device=DEV), dim=-1) * 20)
    base = c.q.float().mean(0).reshape(2, 2, D).mean(1)
    for step in (0.02, -0.02):
        ramp = torch.arange(1500, device=DEV).float() * step
        c.k.copy_(ramp[:, None, None] * base[None] + torch.randn(c.k.shape, generator=gen(4), device=DEV))
        (c.sk, _) = cp.cp_kv_shard_pack(c.dplan, c.k)
        o, lse = c.run()
        cp.cp_device_error_check()
        c.check(o, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("members", [9, 70])
def test_prefix_reads_its_group_only(cp, kv, members):
    """Rows of other groups next to a group's, and rows of the pool that no pair
    names, are not mixed in: they may even be NaN."""
    bad = 0x7F if kv == "fp8" else math.nan  # E4M3's NaN
    c = Case(cp, 2, [100, 130], [members, members], 8, 2, 128, kv, page=64)
    o, lse = c.run()
    used = {(int(c.pages.host[p, i // 64]) * 64 + i % 64) for p in range(4) for i in range(int(c.plan.pairs[p, 0]))}
    rest = torch.tensor(sorted(set(range(c.pages.pool_rows)) - used), device=DEV)
    for x in c.pool[:2]:
        x[rest] = bad
    if c.pool[2] is not None:
        c.pool[2][rest] = math.nan
    o2, lse2 = c.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # shards: the second group's rows follow the first one's inside a tile
    c = Case(cp, 2, [100, 130], [members, members], 8, 2, 128, kv)
    o, lse = c.run()
    for r in range(2):
        n = int(c.plan.pairs[r * 2, 0])
        c.sk[r][n:], c.sv[r][n:] = bad, bad
        if c.sc is not None:
            c.sc[r][n:] = math.nan
    o2, lse2 = c.run()
    assert torch.equal(o[:members], o2[:members]) and torch.equal(lse[:members], lse2[:members])


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
def test_prefix_of_many_shards(cp, kv, D):
    """More shards than the short list of tensor maps holds, most of them with few rows."""
    c = Case(cp, 40, [700, 30, 5000], [5, 1, 40], 8, 2, D, kv, workers=20, P=1)
    o, lse = c.run()
    cp.cp_device_error_check()
    c.check(o, lse)


@pytest.mark.parametrize("workers", [2, 3, 9])
@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp32"])
def test_prefix_of_a_query_that_is_nan(cp, kv, workers):
    """A NaN query row spoils its own results only, in parts or alone."""
    c = Case(cp, 1, [600], [20], 8, 2, 128, kv, workers=workers)
    o, lse = c.run()
    c.q[3, 5, 7] = math.nan
    o2, lse2 = c.run()
    cp.cp_device_error_check()
    assert o2[3, 5].isnan().all() and lse2[3, 5].isnan()
    o2[3, 5], lse2[3, 5] = o[3, 5], lse[3, 5]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_prefix_joins_the_requests_own_tokens(cp):
    """A batch behind one prefix: prefix and own caches against one attention
    over all tokens of each request."""
    B, P, own, Hq, Hkv, D, C = 6, 900, [1, 70, 300, 5, 64, 129], 8, 2, 128, 2
    g = gen(5)
    q, kp, vp = randn(g, (B, Hq, D)), randn(g, (P, Hkv, D)), randn(g, (P, Hkv, D))
    ko, vo = randn(g, (sum(own), Hkv, D)), randn(g, (sum(own), Hkv, D))
    dp, do = cp.cp_decode_plan(C, [P], device=DEV), cp.cp_decode_plan(C, own, device=DEV)
    pack = lambda plan, x: cp.cp_kv_shard_pack(plan, x)[0]  # noqa: E731
    o_part, lse_part = cp.cp_decode_attn(do, cp.CP_DECODE_GQA, q, pack(do, ko), pack(do, vo))
    plan = cp.cp_prefix_plan(C, [P], [B], Hq, Hkv, device=DEV)
    o, lse = cp.cp_prefix_attn(plan, q, pack(dp, kp), pack(dp, vp), o_part=o_part, lse_part=lse_part, out_dtype=torch.float32)
    cp.cp_device_error_check()
    t = 0
    for b, n in enumerate(own):
        for h in range(Hq):
            k = torch.cat([kp[:, h // 4], ko[t:t + n, h // 4]]).double()
            v = torch.cat([vp[:, h // 4], vo[t:t + n, h // 4]]).double()
            x = k @ q[b, h].double() / math.sqrt(D)
            p = torch.softmax(x, 0)
            size = float((k.abs() @ q[b, h].double().abs()).max()) / math.sqrt(D)
            assert abs(float(lse[b, h]) - float(torch.logsumexp(x, 0))) <= 2.0**-19 * (size + 10)
            assert ((o[b, h].double() - p @ v).abs() <= (2.0**-8 + 2.0**-17 * size) * (p @ v.abs()) + 2.0**-19).all()
        t += n


def test_prefix_two_streams_and_a_graph(cp):
    """Two calls at once with workspaces of their own, and a replayed call."""
    a, b = Case(cp, 2, [3000], [40], 16, 4, 128, seed=1, P=1), Case(cp, 1, [2000, 9], [3, 70], 8, 2, 64, seed=2)
    wa, wb = a.run(), b.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(c.run())
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, (wa, wb)):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = a.run()
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, wa[0]) and torch.equal(l, wa[1])


def test_prefix_refusals(cp):
    c = Case(cp, 2, [50], [3], 8, 2, 64)
    with pytest.raises(ValueError, match="shard"):
        cp.cp_prefix_attn(c.plan, c.q, c.sk[:1], c.sv)
    with pytest.raises(ValueError, match="shape"):
        cp.cp_prefix_attn(c.plan, c.q, [x[1:] for x in c.sk], c.sv)
    with pytest.raises(ValueError, match="o_part"):
        cp.cp_prefix_attn(c.plan, c.q, c.sk, c.sv, o_part=torch.zeros((1, 3, 8, 64), device=DEV))
    with pytest.raises(TypeError, match="out_dtype"):
        c.run(out_dtype=torch.float16)
    with pytest.raises(cp.CpError, match="workspace"):
        d = Case(cp, 2, [5000], [3], 8, 2, 64)
        d.run(ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    host_only = cp.cp_prefix_plan(2, [50], [3], 8, 2, n_workers=4)
    with pytest.raises(ValueError, match="device part"):
        cp.cp_prefix_attn(host_only, c.q, c.sk, c.sv)
    with pytest.raises(cp.CpError, match="scale"):
        cp.cp_prefix_attn(c.plan, c.q, c.sk, c.sv, sm_scale=0.0)


@pytest.mark.parametrize("kv,D,members", [("bf16", 128, 70), ("bf16", 64, 9), ("fp8", 128, 9), ("fp8", 128, 70)])
def test_prefix_wait_that_runs_out(cp, monkeypatch, kv, D, members):
    """The issuer waits for a barrier that nothing arrives at: the kernel gives up,
    drains and returns, and the next call is right."""
    c = Case(cp, 2, [700], [members], 16, 4, D, kv, workers=6)
    cp.cp_device_error_check()
    monkeypatch.setenv("CPATTN_TEST_STALL", "1")
    c.run()
    with pytest.raises(cp.CpError) as ei:
        cp.cp_device_error_check()
    assert ei.value.status == -4
    monkeypatch.delenv("CPATTN_TEST_STALL")
    o, lse = c.run()
    cp.cp_device_error_check()
    c.check(o, lse)


def test_prefix_of_a_long_cache(cp):
    """K and V past 2^31 elements: the last rows are the ones that are read last."""
    P, Hq, Hkv, D = 2**31 // (8 * 128) + 300, 8, 8, 128
    g = gen(1)
    k, v = torch.zeros((P, Hkv, D), dtype=torch.bfloat16, device=DEV), torch.zeros((P, Hkv, D), dtype=torch.bfloat16, device=DEV)
    q = torch.ones((2, Hq, D), dtype=torch.bfloat16, device=DEV)
    k[-200:] = 4.0  # these take all of the weight
    v[-200:] = randn(g, (200, Hkv, D))
    plan = cp.cp_prefix_plan(1, [P], [2], Hq, Hkv, device=DEV)
    o, lse = cp.cp_prefix_attn(plan, q, [k], [v], sm_scale=0.1, out_dtype=torch.float32)
    cp.cp_device_error_check()
    want = v[-200:].double().mean(0)
    # the other rows' weight: 2^21 e^-51.2, under 2^-52; P = 1 is exact, V's sums are fp32
    assert ((o.double() - want).abs() <= 2.0**-20 * v[-200:].double().abs().mean(0) + 2.0**-22).all()
    assert ((lse.double() - (51.2 + math.log(200))).abs() <= 2.0**-20 * 60).all()
