"""Prompts that are weighed and cut to a budget before the first token is decoded:
slots, append, attention, weights, choice, moves, pages back, and the decode over what is
left, against the rule and the definition in 64 bits."""

import math

import numpy as np
import pytest
import torch

from test_gpu_evict import I32, i32, rows_of_plan, shard_rows
from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import gen, randn

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE = 8, 2, 128, 64


def weigh(cp, chunks, b, q, k, window):
    """64-bit weights of request b's tokens: q, k by chunk and request."""
    n = sum(c[b] for c in chunks)
    w, seen = torch.zeros(n, dtype=torch.float64, device=DEV), 0
    K = torch.cat([x[b] for x in k]).double()
    for i, c in enumerate(chunks):
        seen += c[b]
        for x in range(max(0, c[b] - window) if window else 0, c[b]):
            at = seen - c[b] + x + 1  # keys that this query reads
            for h in range(HQ):
                w[:at] += torch.softmax(K[:at, h // (HQ // HKV)] @ q[i][b][x, h].double() / math.sqrt(D), 0)
    return w


@pytest.mark.parametrize("C", [1, 2])
@pytest.mark.parametrize("window", [0, 32])
def test_prompts_cut_to_a_budget(cp, C, window):
    chunks, keep, last = [[200, 77, 300], [50, 60, 1]], [64, 100, 70], 8
    B, g, num = 3, gen(C), 40
    pages = cp.PageTable.on_device(torch.full((C * B, 8), -1, **I32), PAGE, num)
    free, at = torch.arange(num, **I32).flip(0).contiguous(), torch.zeros(1, **I32)
    pool_k, pool_v = (torch.zeros((num * PAGE, HKV, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    w, pos_all = torch.zeros(num * PAGE, device=DEV), torch.full((num * PAGE + 1,), -1, **I32)
    pos, have = pos_all[:-1], [0] * B
    q, k, v = ([[randn(g, (n, h, D)) for n in c] for c in chunks] for h in (HQ, HKV, HKV))
    slots = [torch.zeros(0, dtype=torch.long, device=DEV) for _ in range(B)]
    for i, new in enumerate(chunks):
        s, cu, info = cp.cp_page_slots(pages, C, i32(have), i32(new), free, at, sum(new))
        at = info[1:2].clone()
        assert info[0].item() == 0
        cp.cp_cache_append(s, torch.cat(k[i]), pool_k, torch.cat(v[i]), pool_v)
        pos_all[s.long()] = i32([have[b] + x for b in range(B) for x in range(new[b])])
        plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, new, have, device=DEV)
        kk, vv = (torch.cat([torch.cat([y[b] for y in x[:i + 1]]) for b in range(B)]) for x in (k, v))
        lse = cp.cp_prefill_attn(plan, torch.cat(q[i]), kk, vv)[1]
        out = cp.cp_prefill_weights(plan, torch.cat(q[i]), kk, lse, window=window)
        cut = s.long().split(new)
        slots = [torch.cat([a, b]) for a, b in zip(slots, cut)]
        w[torch.cat(slots)] += out  # new rows start at 0
        have = [a + b for a, b in zip(have, new)]
    cp.cp_device_error_check()
    for b in range(B):
        want = weigh(cp, chunks, b, q, k, window)
        # score and LSE are each off by at most 2^-20 of the sum of the products' magnitudes (under
        # 2^5 here: 128 normal products over sqrt(128)), the sums by 2^-18: together under 2^-13
        assert ((w[slots[b]].double() - want).abs() <= 2.0**-13 * want).all()
        assert pos[slots[b]].tolist() == list(range(have[b]))
    start = [n - last for n in have]
    src, dst, count = cp.cp_evict_select(pages, C, i32(have), i32(keep), w, 128, pos=pos, keep_below=4, keep_from=i32(start))
    before = w.clone()
    cp.cp_cache_move(src, dst, count, pool_k, pool_v, weights=w, pos=pos, C=C)
    info = cp.cp_page_release(pages, C, i32(have), i32(keep), free, at, w, pos, count=count)
    assert (count >= 0).all() and info[0].item() == 0 and info[3].item() == 0
    need = sum(-(-shard_rows(n, C, r) // PAGE) for n in have for r in range(C))
    left = sum(-(-shard_rows(n, C, r) // PAGE) for n in keep for r in range(C))
    assert info[2].item() == need - left and info[1].item() == left
    # every shard keeps its protected tokens and its heaviest
    stay = []
    for b in range(B):
        mine = []
        for r in range(C):
            tok = list(range(r, have[b], C))
            rank = sorted(tok, key=lambda t: (not (t < 4 or t >= start[b]), 0 if t < 4 or t >= start[b] else -float(before[slots[b][t]]), t))
            mine += rank[:shard_rows(keep[b], C, r)]
        stay.append(sorted(mine))
    # decode over what is left
    qd = randn(g, (B, HQ, D))
    plan = cp.cp_decode_plan(C, keep, device=DEV)
    o, l = cp.cp_decode_attn_paged(plan, pages.sync_host(), cp.CP_DECODE_GQA, qd, pool_k, pool_v)
    o, l = cp.cp_lse_merge(o, l, out_dtype=torch.float32)
    cp.cp_device_error_check()
    for b in range(B):
        at = [int(pages.host[r * B + b, i // PAGE]) * PAGE + i % PAGE for r in range(C) for i in range(shard_rows(keep[b], C, r))]
        assert sorted(pos[torch.tensor(at, device=DEV)].tolist()) == stay[b]
        idx = torch.tensor(stay[b], device=DEV)
        K, V = (torch.cat([x[b] for x in y]).double()[idx] for y in (k, v))
        for h in range(HQ):
            p = torch.softmax(K[:, h // (HQ // HKV)] @ qd[b, h].double() / math.sqrt(D), 0)
            V_h = V[:, h // (HQ // HKV)]
            assert ((o[b, h].double() - p @ V_h).abs() <= 2.0**-7 * (p @ V_h.abs()) + 1e-5).all()
