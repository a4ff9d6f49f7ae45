"""Latent attention around the MLA decode: the per-head products and the
expanded prefill against the fp64 oracle.

Tolerances, elementwise, from the roundings that the kernels make (a rounding
to bf16 is off by at most 2^-8 of the value):
  products  one rounding of the result, and fp32 sums of K terms, each of
            their K additions off by at most 2^-23 of the sum of |terms|;
  prefill   a weight's rounding moves O by at most 2^-8 A, A the softmax's
            mean of |v|, the result's own by 2^-8 |O|.  A score is a sum of
            192 terms as above, off by at most d = 192 x 2^-23 x scale x sum
            |q k|; with the exponential's 2^-20 that moves weights and their
            sum by e = d + 2^-20 relative, O by 2 e A and the LSE by e, whose
            own sum of L weights adds L x 2^-24 and whose rounding 2^-22 (|LSE| + 1).
"""

import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_canary import check_guards, guarded
from test_gpu_parity import DEV, cp, np64  # noqa: F401

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(192)


def randn(shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def weights(H, seed):
    return randn((H, 256, 512), seed, 1 / math.sqrt(512))


def close(got, ref, tol, what):
    d = np.abs(np64(got) - ref)
    worst = np.max(d - tol) if d.size else 0.0
    assert not np.isnan(d).any(), f"{what}: NaN"
    assert worst <= 0, f"{what}: {worst:.3e} past its tolerance (error {d.max():.3e})"


def product_tol(ref, terms, K):
    return 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * terms * 1.01


# ------------------------------------------------------------------ products

@pytest.mark.parametrize("T,H,stride", [(1, 1, 512), (127, 3, 576), (128, 2, 512), (129, 16, 640), (700, 5, 576),
                                        (5000, 8, 576), (2500, 33, 512), (257, 80, 576), (700, 150, 576),
                                        (513, 150, 512)])
def test_expand(cp, T, H, stride):
    lat, w = randn((T, stride), T)[:, :512], weights(H, H)
    out, buf, keep = guarded((T, H, 256), torch.bfloat16, 3)
    assert cp.cp_mla_expand(lat, w, out=out) is out
    cp.cp_device_error_check()
    check_guards(buf, keep, "expand")
    ref = oracle.mla_expand(np64(lat), np64(w))
    close(out, ref, product_tol(ref, oracle.mla_expand(np.abs(np64(lat)), np.abs(np64(w))), 512), "expand")


@pytest.mark.parametrize("N,H", [(1, 1), (1, 64), (2, 5), (3, 9), (4, 130), (5, 6), (16, 64), (17, 33), (37, 16), (64, 7), (65, 64), (128, 3), (129, 8),
                                 (300, 2), (1030, 5)])
def test_absorb_and_project(cp, N, H):
    w = weights(H, H)
    q, ol = randn((N, H, 192), N), randn((N, H, 512), N + 1)
    ql, b1, k1 = guarded((N, H, 576), torch.bfloat16, 4)
    o, b2, k2 = guarded((N, H, 128), torch.bfloat16, 5)
    cp.cp_mla_absorb(q, w, out=ql)
    cp.cp_mla_project(ol, w, out=o)
    cp.cp_device_error_check()
    check_guards(b1, k1, "absorb")
    check_guards(b2, k2, "project")
    assert torch.equal(ql[..., 512:], q[..., 128:])
    nq, no, nw = np64(q), np64(ol), np64(w)
    ref = oracle.mla_absorb(nq, nw)[..., :512]
    close(ql[..., :512], ref, product_tol(ref, oracle.mla_absorb(np.abs(nq), np.abs(nw))[..., :512], 128), "absorb")
    ref = oracle.mla_project(no, nw)
    close(o, ref, product_tol(ref, oracle.mla_project(np.abs(no), np.abs(nw)), 512), "project")


def test_products_take_query_rows_and_nothing(cp):
    """Leading dims as the decode has them ([B, s_q, H, ...]), and no token at all."""
    w = weights(4, 1)
    q = randn((3, 2, 4, 192), 1)
    a = cp.cp_mla_absorb(q, w)
    assert a.shape == (3, 2, 4, 576)
    assert torch.equal(a.reshape(6, 4, 576), cp.cp_mla_absorb(q.reshape(6, 4, 192), w))
    assert cp.cp_mla_absorb(q[:0], w).shape == (0, 2, 4, 576)
    assert cp.cp_mla_project(randn((0, 4, 512), 1), w).shape == (0, 4, 128)
    assert cp.cp_mla_expand(randn((0, 512), 1), w).shape == (0, 4, 256)


@pytest.mark.parametrize("N", [3, 20, 70, 200])
def test_product_rows_stay_apart(cp, N):
    """A token of NaN or infinities reaches its own row and no other, also
    where the tile is padded."""
    w = weights(2, 2)
    last = N - 1
    for fn, cols, rest in ((cp.cp_mla_absorb, 192, 512), (cp.cp_mla_project, 512, 128)):
        x = randn((N, 2, cols), 3)
        clean = fn(x, w)
        bad = x.clone()
        bad[min(13, N - 2), 0] = float("nan")
        bad[last, 1, 5] = float("inf")
        got = fn(bad, w)
        torch.cuda.synchronize()
        same = torch.ones(N, 2, dtype=torch.bool, device=DEV)
        same[min(13, N - 2), 0] = same[last, 1] = False
        assert torch.equal(got[same], clean[same])
        assert got[min(13, N - 2), 0].isnan().all() and not got[last, 1, :rest].isfinite().any()
    lat = randn((N, 512), 4)
    clean = cp.cp_mla_expand(lat, w)
    lat[last] = float("nan")
    got = cp.cp_mla_expand(lat, w)
    assert torch.equal(got[:last], clean[:last]) and got[last].isnan().all()


# ------------------------------------------------------------------ prefill

CASES = [("zigzag", 1, [1], [0], 1), ("zigzag", 1, [513], [0], 2), ("zigzag", 4, [5, 1, 300], [0, 7, 129], 3),
         ("zigzag", 2, [1300], [100], 2), ("interleave", 4, [700, 1, 33], [0, 0, 450], 2),
         ("interleave", 1, [600], [1], 1), ("zigzag", 8, [9, 0, 64], [3, 5, 0], 5), ("zigzag", 1, [1664], [64], 1),
         ("interleave", 3, [1, 1, 1, 1], [0, 900, 127, 128], 2), ("interleave", 2, [1280, 2], [0, 510], 3)]


def prefill_inputs(new, prefix, H, seed, q_std=1.0):
    T, KV = sum(new), sum(new) + sum(prefix)
    return randn((T, H, 192), seed, q_std), randn((KV, H, 256), seed + 1), randn((KV, 576), seed + 2)[:, 512:]


def make_plan(cp, strategy, C, new, prefix):
    code = cp.CP_ZIGZAG if strategy == "zigzag" else cp.CP_INTERLEAVE
    ref = (oracle.zigzag_plan if strategy == "zigzag" else oracle.interleave_plan)(new, prefix, C)
    return cp.cp_shard_plan(code, C, new, prefix, device=DEV), ref


def check_prefill(plan, ref_plan, new, prefix, q, kv, rope, o, lse, what, scale=SCALE):
    K, V = oracle.mla_expanded_qkv(np64(kv), np64(rope))
    nq = np64(q)
    ref = oracle.prefill_reference(ref_plan, new, prefix, nq, K, V, scale)
    mean = oracle.prefill_reference(ref_plan, new, prefix, nq, K, np.abs(V), scale)
    # sum |q k| of each query and head, at most |q| times the largest |k|
    terms = np.linalg.norm(nq, axis=-1) * np.linalg.norm(K, axis=-1).max(0)
    ro = plan.rank_off
    L = max(n + p for n, p in zip(new, prefix))
    for r in range(plan.C):
        _, ro_ref, rl = ref[r]
        e = 192 * 2.0 ** -23 * scale * terms[np.asarray(ref_plan["order"][r], dtype=np.int64)] + 2.0 ** -20
        A = mean[r][1]
        close(o[ro[r]:ro[r + 1]], ro_ref, (2.0 ** -8 + 2 * e[..., None]) * A * 1.01 + 2.0 ** -8 * np.abs(ro_ref), f"{what} rank {r} O")
        close(lse[ro[r]:ro[r + 1]], rl, e + L * 2.0 ** -24 + 2.0 ** -22 * (np.abs(rl) + 1), f"{what} rank {r} LSE")


@pytest.mark.parametrize("strategy,C,new,prefix,H", CASES)
def test_prefill(cp, strategy, C, new, prefix, H):
    q, kv, rope = prefill_inputs(new, prefix, H, 11)
    plan, ref = make_plan(cp, strategy, C, new, prefix)
    o, ob, ok = guarded((sum(new), H, 128), torch.bfloat16, 6)
    lse, lb, lk = guarded((sum(new), H), torch.float32, 7)
    cp.cp_mla_prefill_attn(plan, q, kv, rope, out=o, lse=lse)
    cp.cp_device_error_check()
    check_guards(ob, ok, "prefill O")
    check_guards(lb, lk, "prefill LSE")
    check_prefill(plan, ref, new, prefix, q, kv, rope, o, lse, strategy)


@pytest.mark.parametrize("strategy,C,n", [("zigzag", 3, 2400), ("interleave", 4, 2400), ("zigzag", 1, 1050), ("interleave", 2, 2048)])
def test_prefill_rank_by_rank(cp, strategy, C, n):
    new, prefix, H = [n, 3, 129], [65, 0, 1], 2
    q, kv, rope = prefill_inputs(new, prefix, H, 21)
    plan, _ = make_plan(cp, strategy, C, new, prefix)
    o, lse = cp.cp_mla_prefill_attn(plan, q, kv, rope)
    ro = plan.rank_off
    for r in range(C):
        orank, lrank = cp.cp_mla_prefill_attn(plan, q, kv, rope.contiguous(), rank=r)
        cp.cp_device_error_check()
        assert torch.equal(orank, o[ro[r]:ro[r + 1]]) and torch.equal(lrank, lse[ro[r]:ro[r + 1]])


@pytest.mark.parametrize("slope", [-1.0, 1.0])
@pytest.mark.parametrize("strategy,C", [("zigzag", 1), ("interleave", 2)])
def test_prefill_sharp_scores(cp, slope, strategy, C):
    """Scores that rise along the keys move every row's maximum at every tile
    (the exact path); falling ones keep the first tile's."""
    new, prefix, H = [700], [333], 2
    q, kv, rope = prefill_inputs(new, prefix, H, 31)
    KV = kv.shape[0]
    kv = kv * 0.05
    kv[:, :, 128:] *= 20
    q[..., 0] = 8.0
    # key dim 0 alone carries q0 k0 scale = 8 x k0 / sqrt(192): about 11 a tile
    kv[:, :, 0] = (slope * torch.arange(KV, device=DEV) * (11.0 / 128) / (8.0 * SCALE)).to(torch.bfloat16)[:, None]
    plan, ref = make_plan(cp, strategy, C, new, prefix)
    o, lse = cp.cp_mla_prefill_attn(plan, q, kv.contiguous(), rope)
    cp.cp_device_error_check()
    check_prefill(plan, ref, new, prefix, q, kv, rope, o, lse, "sharp")


def test_prefill_other_requests_rows_do_not_matter(cp):
    """NaN and infinities in one request's keys, values and rotated keys leave
    the neighbours' outputs bit for bit (tiles run past a request's end)."""
    new, prefix, H = [300, 65, 200], [10, 0, 77], 2
    q, kv, rope = prefill_inputs(new, prefix, H, 41)
    for C in (1, 2):
        plan, ref = make_plan(cp, "zigzag", C, new, prefix)
        o, lse = cp.cp_mla_prefill_attn(plan, q, kv, rope)
        kv2, rope2 = kv.clone(), rope.clone()
        kv2[310:375] = float("nan")
        rope2[310:375:2] = float("inf")
        o2, lse2 = cp.cp_mla_prefill_attn(plan, q, kv2, rope2)
        cp.cp_device_error_check()
        req = np.concatenate([np.asarray(x) for x in ref["req"]])
        keep = torch.as_tensor(req != 1, device=DEV)
        assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38, 1000.0])
@pytest.mark.parametrize("C,H", [(1, 2), (2, 3)])
def test_prefill_other_requests_queries_do_not_matter(cp, value, C, H):
    """Nor do its queries: a tile's rows past a request's last query hold the
    next one's."""
    new, prefix = [300, 65, 1100, 70], [200, 0, 77, 400]
    q, kv, rope = prefill_inputs(new, prefix, H, 61)
    q[300:365] = value
    q[1465:] = value
    other = q.clone()
    other[300:365] = 0
    other[1465:] = 0
    plan, ref = make_plan(cp, "zigzag", C, new, prefix)
    got = cp.cp_mla_prefill_attn(plan, q, kv, rope)
    want = cp.cp_mla_prefill_attn(plan, other, kv, rope)
    cp.cp_device_error_check()
    req = np.concatenate([np.asarray(x) for x in ref["req"]])
    keep = torch.as_tensor(req % 2 == 0, device=DEV)
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    for r in range(C):
        one = cp.cp_mla_prefill_attn(plan, q, kv, rope, rank=r)
        at = slice(int(plan.rank_off[r]), int(plan.rank_off[r + 1]))
        for a, b in zip(one, want):
            assert torch.equal(a[keep[at]], b[at][keep[at]])


def test_prefill_large_sampled(cp):
    """Several waves of CTAs, long rows: every segment's first and last query
    and random ones."""
    new, prefix, H, C = [5000, 1111], [3000, 0], 16, 8
    prefix[0] += 17
    q, kv, rope = prefill_inputs(new, prefix, H, 51)
    plan, ref = make_plan(cp, "zigzag", C, new, prefix)
    o, lse = cp.cp_mla_prefill_attn(plan, q, kv, rope)
    cp.cp_device_error_check()
    K, V = oracle.mla_expanded_qkv(np64(kv), np64(rope))
    rng = np.random.default_rng(1)
    rows = []
    for r in range(C):
        n = len(ref["order"][r])
        ends = [int(s[4]) - int(plan.rank_off[r]) for s in plan.segments if s[0] == r and s[5] > 0]
        rows.append(sorted({0, n - 1, *ends, *(max(0, x - 1) for x in ends), *rng.integers(0, n, 6).tolist()}))
    want = oracle.prefill_reference(ref, new, prefix, np64(q), K, V, SCALE, rows=rows)
    mean = oracle.prefill_reference(ref, new, prefix, np64(q), K, np.abs(V), SCALE, rows=rows)
    terms = np.linalg.norm(np64(q), axis=-1).max() * np.linalg.norm(K, axis=-1).max()
    e = 192 * 2.0 ** -23 * SCALE * terms + 2.0 ** -20
    for r in range(C):
        local, ro, rl = want[r]
        at = int(plan.rank_off[r]) + local
        close(o[at], ro, (2.0 ** -8 + 2 * e) * mean[r][1] * 1.01 + 2.0 ** -8 * np.abs(ro), f"rank {r} O")
        close(lse[at], rl, e + 8100 * 2.0 ** -24 + 2.0 ** -22 * (np.abs(rl) + 1), f"rank {r} LSE")


@pytest.mark.parametrize("n", [300, 1100])
def test_prefill_reports_a_wait_that_runs_out(cp, monkeypatch, n):
    """A wait of the issuer that nothing ends (single CTAs, pairs): every wait
    gives up in turn, the status says so and the next call is right."""
    new, prefix, H = [n], [40], 3
    q, kv, rope = prefill_inputs(new, prefix, H, 61)
    plan, ref = make_plan(cp, "zigzag", 1, new, prefix)
    cp.cp_device_error_check()
    monkeypatch.setenv("CPATTN_TEST_STALL", "1")
    cp.cp_mla_prefill_attn(plan, q, kv, rope)
    with pytest.raises(cp.CpError) as e:
        cp.cp_device_error_check()
    assert e.value.status == -4 and "kernel 7" in str(e.value)
    monkeypatch.delenv("CPATTN_TEST_STALL")
    cp.cp_device_error_check()
    o, lse = cp.cp_mla_prefill_attn(plan, q, kv, rope)
    cp.cp_device_error_check()
    check_prefill(plan, ref, new, prefix, q, kv, rope, o, lse, "after the timeout")


@pytest.mark.parametrize("op,n,H", [("expand", 300, 3), ("expand", 2560, 32), ("expand", 2400, 33), ("absorb", 5, 2), ("absorb", 700, 64),
                                    ("project", 37, 3), ("project", 1000, 64)])
def test_products_report_a_wait_that_runs_out(cp, monkeypatch, op, n, H):
    """The same for the products: single CTAs with one item and with several,
    and pairs (76 of them, whole and ragged runs of heads).  What a call that
    gave up leaves is not looked at; the next one's result is the earlier one's."""
    w = weights(H, 1)
    x = randn((n, 576) if op == "expand" else (n, H, 192 if op == "absorb" else 512), 2)

    def call():
        return cp.cp_mla_expand(x[:, :512], w) if op == "expand" else getattr(cp, f"cp_mla_{op}")(x, w)

    before = call()
    cp.cp_device_error_check()
    for _ in range(2):
        monkeypatch.setenv("CPATTN_TEST_STALL", "1")
        call()
        with pytest.raises(cp.CpError) as e:
            cp.cp_device_error_check()
        assert e.value.status == -4 and "kernel 8" in str(e.value)
        monkeypatch.delenv("CPATTN_TEST_STALL")
        cp.cp_device_error_check()
        after = call()
        cp.cp_device_error_check()
        assert torch.equal(before, after)


def test_calls_on_two_streams_at_once(cp):
    """Prefill, expansion and products of two batches side by side give what
    they give alone."""
    H = 8
    w = weights(H, 3)
    jobs = []
    for k, (new, prefix) in enumerate((([1500, 20], [100, 0]), ([900], [333]))):
        q, _, _ = prefill_inputs(new, prefix, H, 70 + k)
        jobs.append((make_plan(cp, "zigzag", 2, new, prefix)[0], q, randn((sum(new) + sum(prefix), 576), 80 + k),
                     randn((150, H, 512), 90 + k)))

    def work(plan, q, lat, ol):
        out = []
        for _ in range(6):
            kv = cp.cp_mla_expand(lat[:, :512], w)
            out = [kv, *cp.cp_mla_prefill_attn(plan, q, kv, lat[:, 512:]), cp.cp_mla_absorb(q, w), cp.cp_mla_project(ol, w)]
        return out

    alone = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    both = []
    for s, j in zip(streams, jobs):
        with torch.cuda.stream(s):
            both.append(work(*j))
    torch.cuda.synchronize()
    cp.cp_device_error_check()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_32_bits(cp):
    """Tensors of more than 2^31 elements: the last request's rows are, bit for
    bit, those of a call with that request alone."""
    H, n, R = 128, 1000, 90
    w = weights(H, 1)
    lat = randn((n * R, 576), 2)
    kv = cp.cp_mla_expand(lat[:, :512], w)
    tail = lat[-n:]
    assert kv.numel() > 2**31 and torch.equal(kv[-n:], cp.cp_mla_expand(tail[:, :512], w))
    q = torch.empty((n * R, H, 192), dtype=torch.bfloat16, device=DEV)
    for r in range(R):
        q[r * n:(r + 1) * n] = randn((n, H, 192), 100 + r)
    assert q.numel() > 2**31
    plan, _ = make_plan(cp, "zigzag", 1, [n] * R, [0] * R)
    o, lse = cp.cp_mla_prefill_attn(plan, q, kv, lat[:, 512:])
    alone, _ = make_plan(cp, "zigzag", 1, [n], [0])
    oa, la = cp.cp_mla_prefill_attn(alone, q[-n:], kv[-n:], tail[:, 512:])
    cp.cp_device_error_check()
    assert torch.equal(o[-n:], oa) and torch.equal(lse[-n:], la)
    ql = cp.cp_mla_absorb(q[-30000:], w)
    assert ql.numel() > 2**31 and torch.equal(ql[-n:], cp.cp_mla_absorb(q[-n:], w))
    ol = ql[..., :512].contiguous()
    assert torch.equal(cp.cp_mla_project(ol, w)[-n:], cp.cp_mla_project(ol[-n:], w))
    cp.cp_device_error_check()


def test_on_a_side_stream_and_in_a_graph(cp):
    """The calls run on the current stream, and a captured step follows its
    inputs when it is replayed."""
    new, prefix, H = [200, 60], [0, 30], 4
    w = weights(H, 5)
    lat = randn((290, 576), 6)
    q = randn((260, H, 192), 7)
    plan, _ = make_plan(cp, "zigzag", 2, new, prefix)

    def step():
        kv = cp.cp_mla_expand(lat[:, :512], w)
        o, lse = cp.cp_mla_prefill_attn(plan, q, kv, lat[:, 512:])
        return kv, o, lse, cp.cp_mla_absorb(q, w)

    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    lat.copy_(randn((290, 576), 8))
    q.copy_(randn((260, H, 192), 9))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, want))
    cp.cp_device_error_check()
