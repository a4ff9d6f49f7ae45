"""Latent attention around its cache: what is measured, and the plain forms.

Operators (names of the package's entry points):

* ``cp_mla_prefill_attn``  causal attention of a prompt in the expanded form:
  every head has its own 128-dim key part and value, all heads share one
  rotated 64-dim key part per token; outputs in the rank-major order of a
  zigzag or interleave shard plan, with the log-sum-exp.
* ``cp_mla_expand``, ``cp_mla_absorb``, ``cp_mla_project``  the per-head products
  with the up-projection W [H, 256, 512] (rows: 128 of the key part, 128 of the
  value): latent rows to keys and values; a query's key part into the latent
  space, where the cached rows are the keys; a latent output to values.
* ``cp_page_slots``  page tables and slot maps from request lengths on the GPU.
* ``cp_cache_append``  new tokens' rows into the pages of the slot map, as they
  are or as E4M3 codes with one scale a token.

A case gives its sizes; lengths of a ragged batch are drawn from the seed
``lens`` that the case names, so that a case's shapes are the same for every
input seed.
"""

import math
import random

import numpy as np
import torch

own = False

NOPE, ROPE, VDIM, LATENT = 128, 64, 128, 512
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a chunk of a long prompt behind a cached prefix (the prefix of the zigzag workload), half of
        # 64 heads, eight zigzag ranks: the tensor cores' case
        dict(name="prefill_chunk", op="prefill", strategy="zigzag", C=8, H=32, R=1, new=16384, prefix=4096, lens=1),
        # a batch of short prompts of very different lengths, some a single token, some with a prefix
        dict(name="prefill_ragged", op="prefill", strategy="interleave", C=4, H=16, R=9, new=2500, prefix=700, lens=2),
        # keys and values of that chunk and its prefix, read out of the 576-wide latent cache
        dict(name="expand_chunk", op="expand", T=20480, H=32, stride=576),
        # a short prompt's, on a quarter of the heads
        dict(name="expand_short", op="expand", T=333, H=16, stride=512),
        # one request's next token: the smallest call of a decode step
        dict(name="absorb_one", op="absorb", N=1, H=64),
        # a full decode batch with two query rows a request
        dict(name="absorb_batch", op="absorb", N=512, H=64),
        # an odd decode batch
        dict(name="project_odd", op="project", N=37, H=64),
        # a large decode batch
        dict(name="project_batch", op="project", N=1000, H=64),
        # a decode step of the mixed-length batch: one token a request, a page needed here and there
        dict(name="slots_step", op="slots", B=128, C=8, page=64, ctx=400000, new=1, pages=1024, lens=3),
        # prompts entering the cache
        dict(name="slots_prompts", op="slots", B=16, C=8, page=64, ctx=9000, new=60000, pages=192, lens=4),
        # a decode step's latent rows into the FP8 cache
        dict(name="append_step", op="append", n=128, heads=0, dim=576, kv="fp8", page=64),
        # a prompt chunk's keys and values (8 heads of 128) into an FP8 cache
        dict(name="append_chunk", op="append", n=32768, heads=8, dim=128, kv="fp8", page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "expand", "absorb", "project", "slots", "append"])
    if op == "prefill":
        R = rng.choice([1, 1, 2, 5, 12])
        return dict(op=op, strategy=rng.choice(["zigzag", "interleave"]), C=rng.choice([1, 2, 3, 4, 8]), H=rng.choice([1, 4, 8, 16, 32]),
                    R=R, new=_log_int(rng, 1, 12000 // R), prefix=rng.choice([0, _log_int(rng, 1, 6000 // R)]), lens=rng.randrange(1 << 20))
    if op == "expand":
        return dict(op=op, T=_log_int(rng, 1, 20000), H=rng.choice([1, 2, 7, 8, 16, 32]), stride=rng.choice([512, 576, 640]))
    if op in ("absorb", "project"):
        return dict(op=op, N=_log_int(rng, 1, 1000), H=rng.choice([1, 5, 8, 16, 32, 64]))
    if op == "slots":
        B, C, page = _log_int(rng, 1, 1024), rng.choice([1, 2, 3, 8, 16, 64]), rng.choice([64, 128, 192])
        new = rng.choice([1, 3, _log_int(rng, 1, max(1, 450000 // B))])
        ctx = rng.choice([0, _log_int(rng, 1, 100000)])
        pages = -(-(-(-(ctx + new + 1) // C) + 1) // page) + rng.randrange(3)
        return dict(op=op, B=B, C=C, page=page, ctx=ctx, new=new, pages=pages, lens=rng.randrange(1 << 20))
    heads, dim = rng.choice([(0, 576), (0, 576), (1, 64), (2, 64), (8, 64), (4, 128), (8, 128), (16, 128)])
    return dict(op=op, n=_log_int(rng, 1, 30000 if heads * dim <= 1024 else 15000), heads=heads, dim=dim,
                kv=rng.choice(["fp8", "fp8", "bf16"]), page=rng.choice([64, 128]))


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """(new, prefix) lengths of a prefill case: one request has the case's own,
    a batch is spread below them, with a request of one token in it."""
    r = random.Random(case["lens"])
    if case["R"] == 1:
        return [case["new"]], [case["prefix"]]
    new = [max(1, _log_int(r, 1, case["new"])) for _ in range(case["R"])]
    new[r.randrange(case["R"])] = 1
    new[r.randrange(case["R"])] = case["new"]
    pre = [r.choice([0, r.randrange(case["prefix"] + 1)]) for _ in range(case["R"])]
    return new, pre


def _slot_lengths(case):
    """(cached, new) lengths of a slots case: cached ones up to `ctx`, new ones
    up to `new` (all of them `new` where that is a handful)."""
    r = random.Random(case["lens"])
    ctx = [r.randrange(case["ctx"] + 1) if case["ctx"] else 0 for _ in range(case["B"])]
    new = [case["new"] if case["new"] <= 3 else r.randrange(case["new"] + 1) for _ in range(case["B"])]
    return ctx, new


def _order(case, new):
    """The flattened new-token index of every output row: each rank's queries
    in its local order, ranks back to back."""
    C, T = case["C"], sum(new)
    if case["strategy"] == "interleave":
        return np.concatenate([np.arange(r, T, C) for r in range(C)])
    rows, base = [], np.concatenate([[0], np.cumsum(new)])
    for r in range(C):
        for j, n in enumerate(new):
            size, extra = divmod(n, 2 * C)
            for b in (r, 2 * C - 1 - r):
                start = b * size + min(b, extra)
                rows.append(base[j] + np.arange(start, start + size + (b < extra)))
    return np.concatenate(rows)


def _randn(gen, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _need(L, C, page):
    """Pages of each shard's rows, [C, B]."""
    L = np.asarray(L, np.int64)
    rows = np.maximum(0, -(-(L[None, :] - np.arange(C)[:, None]) // C))
    return -(-rows // page)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "prefill":
        new, pre = _lengths(case)
        T, KV, H = sum(new), sum(new) + sum(pre), case["H"]
        s["q"] = _randn(gen, (T, H, NOPE + ROPE))
        s["kv"] = _randn(gen, (KV, H, NOPE + VDIM))
        s["k_rope"] = _randn(gen, (KV, LATENT + ROPE))[:, LATENT:]  # the latent cache's last columns
        s["new"], s["prefix"] = new, pre
        s["order"] = torch.from_numpy(_order(case, new)).to(DEV)
        s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
        if own:  # a batch's plan serves every layer
            import context_long_attention_gb300 as cp
            s["plan"] = cp.cp_shard_plan(cp.CP_ZIGZAG if case["strategy"] == "zigzag" else cp.CP_INTERLEAVE, case["C"], new, pre,
                                         device=torch.device(DEV, torch.cuda.current_device()))
    elif op == "expand":
        s["latent"] = _randn(gen, (case["T"], case["stride"]))[:, :LATENT]
        s["w"] = _randn(gen, (case["H"], NOPE + VDIM, LATENT), 1 / math.sqrt(LATENT))
    elif op in ("absorb", "project"):
        s["x"] = _randn(gen, (case["N"], case["H"], NOPE + ROPE if op == "absorb" else LATENT))
        s["w"] = _randn(gen, (case["H"], NOPE + VDIM, LATENT), 1 / math.sqrt(LATENT))
    elif op == "slots":
        B, C, page, maxp = case["B"], case["C"], case["page"], case["pages"]
        ctx, new = _slot_lengths(case)
        have, want = _need(ctx, C, page), _need(np.add(ctx, new), C, page)
        held, taken = int(have.sum()), int((want - have).sum())
        ids = torch.randperm(held + taken + 16, generator=gen, device=DEV).to(torch.int32)
        grid = torch.arange(maxp, device=DEV)[None, :] < torch.from_numpy(have.reshape(-1, 1)).to(DEV)
        table = torch.full((C * B, maxp), -1, dtype=torch.int32, device=DEV)
        table[grid] = ids[:held]
        i32 = dict(dtype=torch.int32, device=DEV)
        s.update(ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), free=torch.cat([ids[:5], ids[held:]]), pos=torch.tensor([5], **i32),
                 table=table, num_pages=held + taken + 16, tokens=sum(new) + 7)
        if own:
            import context_long_attention_gb300 as cp
            s["pages"] = cp.PageTable.on_device(table, page, s["num_pages"])
    else:
        n, dim, page = case["n"], case["dim"], case["page"]
        shape = (n, dim) if case["heads"] == 0 else (n, case["heads"], dim)
        k = torch.randn(shape, generator=gen, device=DEV)
        k *= torch.randn((n,) + (1,) * (len(shape) - 1), generator=gen, device=DEV).exp()  # tokens of different size
        k[n // 2] *= float(n % 3 != 0)  # an all-zero row now and then
        s["k"] = k.to(torch.bfloat16)
        s["v"] = torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16) if case["heads"] else None
        rows = (n + n // 4 + page) // page * page
        slots = torch.randperm(rows, generator=gen, device=DEV)[:n].to(torch.int32)
        if n > 8:
            slots[n // 3] = -1  # padding of the batch
        s["slots"] = slots
        dt = torch.float8_e4m3fn if case["kv"] == "fp8" else torch.bfloat16
        s["k_pool"] = torch.zeros((rows,) + shape[1:], device=DEV).to(dt)
        s["v_pool"] = torch.zeros((rows,) + shape[1:], device=DEV).to(dt) if case["heads"] else None
        s["scale_pool"] = torch.zeros(rows, device=DEV) if case["kv"] == "fp8" else None
    return s


# ------------------------------------------------------------------ plain forms

def _plain_prefill(s, block=512):
    q, kv, rope = s["q"].float(), s["kv"].float(), s["k_rope"].float()
    T, H, _ = q.shape
    o = torch.empty((T, H, VDIM), device=q.device)
    lse = torch.empty((T, H), device=q.device)
    q0 = k0 = 0
    for n, pre in zip(s["new"], s["prefix"]):
        keys = torch.cat([kv[k0:k0 + pre + n, :, :NOPE], rope[k0:k0 + pre + n, None, :].expand(-1, H, -1)], -1).permute(1, 2, 0)
        vals = kv[k0:k0 + pre + n, :, NOPE:].transpose(0, 1)
        for a in range(0, n, block):
            e = min(n, a + block)
            end = pre + e
            x = torch.matmul(q[q0 + a:q0 + e].transpose(0, 1), keys[:, :, :end]) * s["scale"]
            pos = torch.arange(pre + a, end, device=q.device)
            x.masked_fill_(torch.arange(end, device=q.device)[None, :] > pos[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            o[q0 + a:q0 + e] = (torch.matmul(p, vals[:, :end]) / z).transpose(0, 1)
            lse[q0 + a:q0 + e] = (top + torch.log(z))[..., 0].transpose(0, 1)
        q0, k0 = q0 + n, k0 + pre + n
    return o[s["order"]].to(torch.bfloat16), lse[s["order"]]


def _plain_expand(s):
    H = s["w"].shape[0]
    kv = torch.matmul(s["latent"].float(), s["w"].float().reshape(-1, LATENT).T)
    return kv.reshape(-1, H, NOPE + VDIM).to(torch.bfloat16)


def _plain_absorb(s):
    q = s["x"].float()
    lat = torch.matmul(q[..., :NOPE].transpose(0, 1), s["w"][:, :NOPE].float()).transpose(0, 1)
    return torch.cat([lat, q[..., NOPE:]], -1).to(torch.bfloat16)


def _plain_project(s):
    w = s["w"][:, NOPE:].float()
    return torch.matmul(s["x"].float().transpose(0, 1), w.transpose(1, 2)).transpose(0, 1).contiguous().to(torch.bfloat16)


def _plain_slots(s):
    B, C, page, maxp = (s["case"][k] for k in ("B", "C", "page", "pages"))
    ctx, new, free, pos, table = s["ctx"].long(), s["new"].long(), s["free"].long(), s["pos"].long(), s["table"]
    r = torch.arange(C, device=DEV)[:, None]
    pages = lambda L: ((L[None, :] - r + C - 1).div(C, rounding_mode="floor").clamp_(min=0) + page - 1) // page  # noqa: E731
    have, want = pages(ctx), pages(ctx + new)  # [C, B]
    take = want - have
    flat = take.T.reshape(-1)  # request by request, its shards in order
    first = (torch.cumsum(flat, 0) - flat).reshape(B, C).T + pos
    i = torch.arange(maxp, device=DEV)
    at = first[..., None] + i - have[..., None]
    fresh = (i >= have[..., None]) & (i < want[..., None])
    ids = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table.reshape(C, B, maxp).long())
    table.copy_(ids.reshape(C * B, maxp))
    cu = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    torch.cumsum(new, 0, out=cu[1:])
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_(max=B - 1)
    p = ctx[b] + t - cu[b]
    shard, row = p % C, p // C
    slots = ids.reshape(-1)[((shard * B + b) * maxp + row // page).clamp_(max=C * B * maxp - 1)] * page + row % page
    slots = torch.where(t < cu[-1], slots, -1).to(torch.int32)
    info = torch.stack([torch.zeros_like(cu[-1]), pos[0] + flat.sum(), flat.sum(), cu[-1]]).to(torch.int32)
    return slots, cu.to(torch.int32), info, table


def _plain_append(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    k, v = s["k"][keep], None if s["v"] is None else s["v"][keep]
    if s["scale_pool"] is not None:
        amax = k.float().flatten(1).abs().amax(1)
        if v is not None:
            amax = torch.maximum(amax, v.float().flatten(1).abs().amax(1))
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        wide = scale.reshape((-1,) + (1,) * (k.dim() - 1))
        k = (k.float() / wide).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        v = None if v is None else (v.float() / wide).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s["scale_pool"][at] = scale
    bits = torch.uint8 if s["scale_pool"] is not None else torch.bfloat16
    s["k_pool"].view(bits)[at] = k.view(bits)
    if v is not None:
        s["v_pool"].view(bits)[at] = v.view(bits)
    return [x for x in (s["k_pool"], s["v_pool"], s["scale_pool"]) if x is not None]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"prefill": _plain_prefill, "expand": _plain_expand, "absorb": _plain_absorb, "project": _plain_project,
                "slots": _plain_slots, "append": _plain_append}[op](s)
    import context_long_attention_gb300 as cp
    if op == "prefill":
        return cp.cp_mla_prefill_attn(s["plan"], s["q"], s["kv"], s["k_rope"], s["scale"])
    if op == "expand":
        return cp.cp_mla_expand(s["latent"], s["w"])
    if op == "absorb":
        return cp.cp_mla_absorb(s["x"], s["w"])
    if op == "project":
        return cp.cp_mla_project(s["x"], s["w"])
    if op == "slots":
        slots, cu, info = cp.cp_page_slots(s["pages"], s["case"]["C"], s["ctx"], s["new"], s["free"], s["pos"], s["tokens"])
        return slots, cu, info, s["table"]
    cp.cp_cache_append(s["slots"], s["k"], s["k_pool"], s["v"], s["v_pool"], s["scale_pool"])
    return [x for x in (s["k_pool"], s["v_pool"], s["scale_pool"]) if x is not None]


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "prefill":
        new, pre = _lengths(case)
        T, KV, H = sum(new), sum(new) + sum(pre), case["H"]
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, pre))
        return {"bytes": 2 * (T * H * (NOPE + ROPE) + KV * H * (NOPE + VDIM) + KV * ROPE + T * H * VDIM) + 4 * T * H,
                "flops": 2 * (NOPE + ROPE + VDIM) * H * pairs}
    if op == "expand":
        T, H = case["T"], case["H"]
        return {"bytes": 2 * (T * LATENT + H * (NOPE + VDIM) * LATENT + T * H * (NOPE + VDIM)), "flops": 2 * T * H * (NOPE + VDIM) * LATENT}
    if op in ("absorb", "project"):
        N, H = case["N"], case["H"]
        wide = NOPE + ROPE + LATENT + ROPE if op == "absorb" else LATENT + VDIM
        return {"bytes": 2 * (N * H * wide + H * NOPE * LATENT), "flops": 2 * N * H * NOPE * LATENT}
    if op == "slots":
        ctx, new = _slot_lengths(case)
        taken = int((_need(np.add(ctx, new), case["C"], case["page"]) - _need(ctx, case["C"], case["page"])).sum())
        return {"bytes": 12 * case["B"] + 4 * sum(new) + 8 * taken, "flops": 0}
    elems = case["dim"] if case["heads"] == 0 else 2 * case["heads"] * case["dim"]
    out = elems + 4 if case["kv"] == "fp8" else 2 * elems
    return {"bytes": case["n"] * (2 * elems + out + 4), "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _exact_prefill(s):
    """Each request's rows attend one after another in blocks of heads."""
    q, kv, rope = s["q"].double(), s["kv"].double(), s["k_rope"].double()
    T, H, _ = q.shape
    o, lse = torch.zeros((T, H, VDIM), dtype=torch.float64, device=DEV), torch.zeros((T, H), dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for n, pre in zip(s["new"], s["prefix"]):
        L = n + pre
        for h in range(H):
            K = torch.hstack([kv[k0:k0 + L, h, :NOPE], rope[k0:k0 + L]])
            for a in range(0, n, 4096):
                rows = torch.arange(a, min(n, a + 4096), device=DEV)
                x = (q[q0 + rows, h] @ K.T) * s["scale"]
                x = x.where(torch.arange(L, device=DEV) <= (pre + rows)[:, None], torch.full((), -math.inf, dtype=torch.float64, device=DEV))
                total = torch.logsumexp(x, 1)
                o[q0 + rows, h] = torch.exp(x - total[:, None]) @ kv[k0:k0 + L, h, NOPE:]
                lse[q0 + rows, h] = total
        q0, k0 = q0 + n, k0 + L
    return o[s["order"]], lse[s["order"]]


def _exact_slots(s):
    """Token by token in plain integers, pages taken in the order of requests and shards."""
    case = s["case"]
    B, C, page = case["B"], case["C"], case["page"]
    ctx, new = _slot_lengths(case)
    have, want = _need(ctx, C, page), _need(np.add(ctx, new), C, page)
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    pos = int(s["pos"])
    slots = []
    for b in range(B):
        for r in range(C):
            m = int(want[r, b] - have[r, b])
            table[r * B + b, have[r, b]:want[r, b]] = free[pos:pos + m]
            pos += m
        p = np.arange(ctx[b], ctx[b] + new[b], dtype=np.int64)
        slots.append(table[(p % C) * B + b, p // C // page].astype(np.int64) * page + p // C % page)
    slots.append(np.full(s["tokens"] - sum(new), -1))
    cu = np.concatenate([[0], np.cumsum(new)])
    info = np.array([0, pos, pos - int(s["pos"]), sum(new)])
    return tuple(x.astype(np.int32) for x in (np.concatenate(slots), cu, info, table))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":
        return _exact_prefill(s) if work(case)["flops"] < 6e12 else None
    if op == "expand":
        return torch.einsum("tc,hdc->thd", s["latent"].double(), s["w"].double())
    if op == "absorb":
        q, w = s["x"].double(), s["w"].double()
        return torch.cat([torch.einsum("nhd,hdc->nhc", q[..., :NOPE], w[:, :NOPE]), q[..., NOPE:]], -1)
    if op == "project":
        return torch.einsum("nhc,hdc->nhd", s["x"].double(), s["w"][:, NOPE:].double())
    if op == "slots":
        return _exact_slots(s)
    # codes stand for value / scale; a copy's value is the row itself
    keep = s["slots"] >= 0
    at, k, v = s["slots"][keep].long(), s["k"].double()[keep], None if s["v"] is None else s["v"].double()[keep]
    out = []
    if case["kv"] == "fp8":
        both = k.flatten(1) if v is None else torch.cat([k.flatten(1), v.flatten(1)], 1)
        top = both.abs().amax(1)
        scale = torch.where(top > 0, top / 448, 1.0)
        wide = scale.reshape((-1,) + (1,) * (k.dim() - 1))
        k, v = k / wide, None if v is None else v / wide
        out = [s["scale_pool"].double().index_copy(0, at, scale)]
    pools = [s["k_pool"].float().double().index_copy(0, at, k)]
    if v is not None:
        pools.append(s["v_pool"].float().double().index_copy(0, at, v))
    return pools + out
