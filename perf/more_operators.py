"""Around a decode cache that is shared, weighed and thinned out: what is
measured, and the plain forms.

Operators (names of the package's entry points):

* ``cp_rope``  rotary positions of a step's queries and keys: half or
  interleaved pairs, the whole head or the first or last part of it, frequencies
  as they are or scaled for long contexts (``cp_rope_freqs``).
* ``cp_prefix_attn``  attention of groups of queries over the cached prefix that
  each group shares, read once for the group, over the token shards of the
  cache or a paged pool; partial results of the queries' own tokens join in.
* ``cp_prefill_weights``, ``cp_decode_weights``  the attention weight that every
  cached token received, exp(score - LSE) summed over queries and heads: of a
  prompt (all of its queries, or its last ones) and of a decode step.
* ``cp_evict_select``, ``cp_cache_move``  eviction by those weights: each pair of
  a token-sharded paged cache keeps its heaviest rows and some by position, and
  the kept rows past the new length move into the places of evicted ones.

A case gives its sizes; lengths of a ragged batch are drawn from the seed
``lens`` that the case names, so that a case's shapes are the same for every
input seed.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
LATENT, ROPE = 512, 64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's queries and keys, one token a request: the smallest call
        dict(name="rope_step", op="rope", T=64, Hq=32, Hk=8, Dq=128, Dk=128, rot=128, layout="half", tail=False, scaling="none", far=131072),
        # a prompt chunk of latent attention: the last 64 of 192 query dims and the one shared key part
        dict(name="rope_latent", op="rope", T=16384, Hq=64, Hk=1, Dq=192, Dk=64, rot=64, layout="interleaved", tail=True, scaling="yarn", far=1000000),
        # a few requests behind a short system prompt
        dict(name="prefix_few", op="prefix", N=4, groups=1, P=4096, C=1, Hq=32, Hkv=8, D=128, kv="bf16", paged=False, parts=1, lens=11),
        # a decode batch behind a long shared document, over eight token shards
        dict(name="prefix_batch", op="prefix", N=64, groups=1, P=32768, C=8, Hq=32, Hkv=8, D=128, kv="bf16", paged=False, parts=1, lens=12),
        # several shared documents of different length, one group without any, pages
        dict(name="prefix_groups", op="prefix", N=300, groups=5, P=20000, C=2, Hq=64, Hkv=8, D=128, kv="bf16", paged=True, parts=2, lens=13),
        # some requests over one very long document in an FP8 cache
        dict(name="prefix_long", op="prefix", N=16, groups=1, P=131072, C=8, Hq=32, Hkv=8, D=128, kv="fp8", paged=False, parts=0, lens=14),
        # every query of a long prompt chunk weighs the chunk and the prefix before it
        dict(name="weights_prompt", op="weights", strategy="zigzag", C=8, Hq=32, Hkv=8, D=128, R=1, new=16384, prefix=4096, window=0, lens=21),
        # the last queries of ragged prompts weigh their whole prompts
        dict(name="weights_window", op="weights", strategy="interleave", C=4, Hq=32, Hkv=8, D=128, R=9, new=30000, prefix=3000, window=64, lens=22),
        # a decode step's weights over a paged cache
        dict(name="weights_step", op="step", B=16, C=8, ctx=32768, Hq=32, Hkv=8, D=128, kv="bf16", page=64, lens=23),
        # the same over latent entries in 8 bits
        dict(name="weights_latent", op="step", B=64, C=8, ctx=20000, Hq=64, Hkv=1, D=576, kv="fp8", page=64, lens=24),
        # caches held at a budget: the tokens since the last eviction push others out
        dict(name="evict_step", op="evict", B=64, C=8, ctx=2112, keep=2048, heads=8, dim=128, kv="bf16", page=64, same=True, lens=31),
        # long prompts cut to a budget before the first token is decoded
        dict(name="evict_prompt", op="evict", B=8, C=8, ctx=32768, keep=4096, heads=8, dim=128, kv="bf16", page=64, same=False, lens=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefix", "prefix", "weights", "step", "step", "evict"])
    lens = rng.randrange(1 << 20)
    if op == "rope":
        Dq, Dk, rot, tail = rng.choice([(128, 128, 128, False), (64, 64, 64, False), (192, 64, 64, True), (128, 128, 64, False), (256, 256, 64, False), (96, 96, 96, True)])
        Hq, Hk = rng.choice([(32, 8), (64, 8), (8, 2), (16, 1), (5, 5)])
        return dict(op=op, T=_log_int(rng, 1, 16384 * 64 * 192 // (Hq * Dq + Hk * Dk)), Hq=Hq, Hk=Hk, Dq=Dq, Dk=Dk, rot=rot, layout=rng.choice(["half", "interleaved"]), tail=tail,
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), far=_log_int(rng, 100, 2000000))
    heads = [(32, 8), (64, 8), (8, 2), (16, 16), (6, 2), (12, 1)]
    if op == "prefix":
        Hq, Hkv = rng.choice(heads)
        kv, D = rng.choice([("bf16", 128), ("bf16", 128), ("bf16", 64), ("fp8", 128)])
        groups = rng.choice([1, 1, 2, 7])
        N = max(groups, _log_int(rng, 1, 300))
        return dict(op=op, N=N, groups=groups, P=_log_int(rng, 1, max(1, min(60000 // groups, 500000000 // (N * Hq)))), C=rng.choice([1, 2, 3, 8]), Hq=Hq, Hkv=Hkv, D=D, kv=kv,
                    paged=kv == "bf16" and rng.random() < 0.4, parts=rng.choice([0, 1, 3]), lens=lens)
    if op == "weights":
        Hq, Hkv = rng.choice(heads)
        R = rng.choice([1, 2, 6])
        return dict(op=op, strategy=rng.choice(["zigzag", "interleave"]), C=rng.choice([1, 2, 3, 8]), Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128]), R=R,
                    new=_log_int(rng, 1, 10000 // R), prefix=rng.choice([0, _log_int(rng, 1, 6000 // R)]), window=rng.choice([0, 0, 1, 32, 100]), lens=lens)
    B, C, page = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 8]), rng.choice([64, 128, 192])
    if op == "step":
        Hq, Hkv, D = rng.choice([(32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 16, 128), (64, 1, 576), (16, 1, 576), (5, 1, 576)])
        kv = "bf16" if D == 64 else rng.choice(["bf16", "fp8"])
        return dict(op=op, B=B, C=C, ctx=_log_int(rng, 1, min(60000, 400000000 // (B * Hkv * D))), Hq=Hq, Hkv=Hkv, D=D, kv=kv, page=page, lens=lens)
    kv, heads, dim = rng.choice([("bf16", 8, 128), ("bf16", 2, 64), ("bf16", 0, 576), ("fp8", 0, 576), ("fp8", 8, 128)])
    ctx = _log_int(rng, 2, min(60000, 2000000 // B))
    return dict(op=op, B=B, C=C, ctx=ctx, keep=rng.choice([_log_int(rng, 1, ctx), max(1, ctx - rng.randrange(1, 65))]), heads=heads, dim=dim, kv=kv, page=page,
                same=rng.random() < 0.5, lens=lens)


# ------------------------------------------------------------------ inputs

def _randn(gen, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _rows(L, C):
    """Rows of every shard, [C, len(L)]: token p of a request lies on shard p mod C."""
    L = np.asarray(L, np.int64)
    return np.maximum(0, -(-(L[None, :] - np.arange(C)[:, None]) // C))


def _spread(case, most, count, least=1):
    """`count` lengths of a ragged batch, up to `most`, which one of them has."""
    r = random.Random(case["lens"])
    got = [_log_int(r, max(least, most // 8, 1), max(most, 1)) for _ in range(count)]
    got[r.randrange(count)] = most
    return got, r


def _groups(case):
    """(prefix length, queries) of every group; the last of several has no prefix."""
    got, r = _spread(case, case["P"], case["groups"])
    if case["groups"] > 1:
        got[-1] = 0
        got[0] = case["P"]
    cuts = sorted(r.sample(range(1, case["N"]), case["groups"] - 1)) if case["groups"] > 1 else []
    return got, [b - a for a, b in zip([0] + cuts, cuts + [case["N"]])]


def _prompts(case):
    """(new, prefix) lengths: one request has the case's own, a batch is spread
    below them, with a request of one token in it."""
    if case["R"] == 1:
        return [case["new"]], [case["prefix"]]
    new, r = _spread(case, case["new"], case["R"])
    new[(new.index(case["new"]) + 1) % case["R"]] = 1
    return new, [r.choice([0, r.randrange(case["prefix"] + 1)]) for _ in range(case["R"])]


def _order(case, new):
    """The flattened new-token index of every row in the order of the ranks."""
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


def _pages(gen, L, C, page):
    """A page table [C * B, most] of shuffled pages, the pool's pages, and the
    pool row of every (pair, row), -1 past a pair's rows."""
    have = -(-_rows(L, C) // page).reshape(-1)
    total, most = int(have.sum()) + 5, max(1, int(have.max()))
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((have.size, most), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(most, device=DEV)[None, :] < torch.from_numpy(have).to(DEV)[:, None]] = ids[:int(have.sum())]
    return table, total


def _pool_rows(table, L, C, page):
    """The pool row of every (pair, row) of an on-GPU table, and which exist."""
    rows = torch.from_numpy(_rows(L, C).reshape(-1)).to(DEV)
    i = torch.arange(max(1, int(rows.max())), device=DEV)
    there = i[None, :] < rows[:, None]
    at = table.long().gather(1, (i // page)[None, :].expand(table.shape[0], -1).clamp(max=table.shape[1] - 1)) * page + i % page
    return torch.where(there, at, 0), there


def _codes(gen, shape):
    """E4M3 codes of normal values and one scale a row."""
    return _randn(gen, shape, 30.0, torch.float32).clamp_(-448, 448).to(torch.float8_e4m3fn), \
        torch.rand(shape[0], generator=gen, device=DEV) * 0.04 + 0.01


FREQ = {"none": None, "linear": dict(kind="linear", factor=8.0), "ntk": dict(kind="ntk", factor=4.0),
        "bands": dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0),
        "yarn": dict(kind="yarn", factor=40.0, original=4096, beta_fast=32.0, beta_slow=1.0, mscale=1.0)}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    cp = None
    if own:
        import context_long_attention_gb300 as cp
    return {"rope": _prepare_rope, "prefix": _prepare_prefix, "weights": _prepare_weights, "step": _prepare_step, "evict": _prepare_evict}[case["op"]](case, s, gen, cp)


def _prepare_rope(case, s, gen, cp):
    T = case["T"]
    s["q"], s["k"] = _randn(gen, (T, case["Hq"], case["Dq"])), _randn(gen, (T, case["Hk"], case["Dk"]))
    if case["tail"] and case["Hk"] == 1:  # the latent cache's last columns
        s["k"] = _randn(gen, (T, LATENT + case["Dk"]))[:, LATENT:].unsqueeze(1)
    start = torch.randint(0, max(1, case["far"] - T), (1,), generator=gen, device=DEV)
    s["pos"] = ((start + torch.arange(T, device=DEV)) if T > 512 else
                torch.randint(0, case["far"], (T,), generator=gen, device=DEV)).to(torch.int32)
    if own:  # a model's frequencies
        s["freqs"] = cp.cp_rope_freqs(case["rot"], 10000.0, FREQ[case["scaling"]], device=DEV)
    return s


def _prepare_prefix(case, s, gen, cp):
    C, Hkv, D = case["C"], case["Hkv"], case["D"]
    lens, members = _groups(case)
    s.update(prefix=lens, members=members, q=_randn(gen, (case["N"], case["Hq"], D)), scale=1 / math.sqrt(D))
    rows = _rows(lens, C)
    s["k_scale"] = None
    if case["paged"]:
        s["page"] = 64
        s["table"], s["num_pages"] = _pages(gen, lens, C, 64)
        s["k"], s["v"] = ([_randn(gen, (s["num_pages"] * 64, Hkv, D))] for _ in range(2))
    elif case["kv"] == "fp8":
        both = [(_codes(gen, (int(n), Hkv, D)), _codes(gen, (int(n), Hkv, D))[0]) for n in rows.sum(1)]
        s["k"], s["v"], s["k_scale"] = [x[0][0] for x in both], [x[1] for x in both], [x[0][1] for x in both]
    else:
        s["k"], s["v"] = ([_randn(gen, (int(n), Hkv, D)) for n in rows.sum(1)] for _ in range(2))
    if case["parts"]:  # what the queries' own tokens gave
        shape = (case["parts"], case["N"], case["Hq"])
        s["o_part"] = torch.randn(shape + (D,), generator=gen, device=DEV) * 0.1
        s["lse_part"] = torch.randn(shape, generator=gen, device=DEV) + math.log(max(2, case["P"] // 2))
        s["lse_part"][0, ::7] = -math.inf  # a shard without tokens of the request
        s["o_part"][0, ::7] = 0.0
    if own:  # a batch's plan serves every layer
        s["plan"] = cp.cp_prefix_plan(C, lens, members, case["Hq"], Hkv, device=torch.device(DEV, torch.cuda.current_device()))
        if case["paged"]:
            s["pages"] = cp.PageTable.on_device(s["table"], 64, s["num_pages"]).sync_host()
    return s


def _prepare_weights(case, s, gen, cp):
    new, pre = _prompts(case)
    T, KV, Hq, Hkv, D = sum(new), sum(new) + sum(pre), case["Hq"], case["Hkv"], case["D"]
    s.update(new=new, prefix=pre, scale=1 / math.sqrt(D), q=_randn(gen, (T, Hq, D)), k=_randn(gen, (KV, Hkv, D)))
    s["order"] = torch.from_numpy(_order(case, new)).to(DEV)
    lse = torch.empty((T, Hq), device=DEV)
    q0 = 0
    for rows, pos, keys in _blocks(s, 1024):  # the attention's own, in blocks of queries
        x = torch.einsum("qgid,kgd->giqk", s["q"][rows].float().unflatten(1, (Hkv, -1)), s["k"][keys].float()) * s["scale"]
        x.masked_fill_(torch.arange(x.shape[-1], device=DEV) > pos[:, None], -math.inf)
        lse[rows] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(-1, Hq)
    s["lse"] = lse[s["order"]]
    if own:
        s["plan"] = cp.cp_shard_plan(cp.CP_ZIGZAG if case["strategy"] == "zigzag" else cp.CP_INTERLEAVE, case["C"], new, pre,
                                     device=torch.device(DEV, torch.cuda.current_device()))
    return s


def _prepare_step(case, s, gen, cp):
    B, C, page, Hq, Hkv, D = (case[k] for k in ("B", "C", "page", "Hq", "Hkv", "D"))
    L, _ = _spread(case, case["ctx"], B)
    s["table"], s["num_pages"] = _pages(gen, L, C, page)
    rows = s["num_pages"] * page
    shape = (rows, D) if D == 576 else (rows, Hkv, D)
    s.update(L=L, scale=1 / math.sqrt(192 if D == 576 else D), q=_randn(gen, (B, Hq, D), 0.5 if D == 576 else 1.0), k_scale=None)
    if case["kv"] == "fp8":
        s["k"], s["k_scale"] = _codes(gen, shape)
    else:
        s["k"] = _randn(gen, shape)
    s["w"] = torch.rand(rows, generator=gen, device=DEV)
    s["lse"] = torch.zeros((B, Hq), device=DEV)
    x, _, there = _step_scores(s, torch.float32)
    x.masked_fill_(~there[:, None], -math.inf)
    s["lse"] = torch.logsumexp(x, -1)
    if own:
        s["plan"] = cp.cp_decode_plan(C, L, device=torch.device(DEV, torch.cuda.current_device()))
        s["pages"] = cp.PageTable.on_device(s["table"], page, s["num_pages"]).sync_host()
    return s


def _prepare_evict(case, s, gen, cp):
    B, C, page = case["B"], case["C"], case["page"]
    L = [case["ctx"]] * B if case["same"] else _spread(case, case["ctx"], B)[0]
    keep = [min(case["keep"], n) for n in L]
    s["table"], s["num_pages"] = _pages(gen, L, C, page)
    rows = s["num_pages"] * page
    shape = (rows, case["dim"]) if case["heads"] == 0 else (rows, case["heads"], case["dim"])
    i32 = dict(dtype=torch.int32, device=DEV)
    s.update(L=L, keep=keep, ctx_len=torch.tensor(L, **i32), keep_len=torch.tensor(keep, **i32))
    s["keep_from"] = torch.tensor([n + n // 3 - min(32, n // 4) for n in L], **i32)  # the newest tokens stay
    make = (lambda: _codes(gen, shape)[0]) if case["kv"] == "fp8" else (lambda: _randn(gen, shape))
    s["k"], s["v"] = make(), make() if case["heads"] else None
    s["k_scale"] = torch.rand(rows, generator=gen, device=DEV) if case["kv"] == "fp8" else None
    # heavy and light tokens, many that nothing looked at, equal ones among them
    w = torch.randn(rows, generator=gen, device=DEV).mul_(3).exp_()
    s["w"] = torch.where(w < 0.2, 0.0, torch.where(w > 5, w.round(), w))
    at, there = _pool_rows(s["table"], L, C, page)
    pos = torch.full((rows,), -1, **i32)  # positions after earlier evictions: in no order, a quarter of the tokens gone
    order = torch.rand(at.shape, generator=gen, device=DEV).masked_fill(~there, 9).argsort(1).argsort(1)
    pair = torch.arange(C * B, device=DEV)[:, None]
    pos[at[there]] = ((order * C + pair // B) * 4 // 3)[there].to(torch.int32)
    s["pos"] = pos
    s["most"] = int((_rows(L, C) - _rows(keep, C)).clip(0).max())
    s["most"] = max(1, min(s["most"], int(_rows(keep, C).max())))
    if own:
        s["pages"] = cp.PageTable.on_device(s["table"], page, s["num_pages"])
    return s


# ------------------------------------------------------------------ plain forms

def _inv_freq(rot, scaling, base=10000.0):
    """(radians a position of every pair, in 64 bits; factor on cos and sin)."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot
    f, c = base ** -i, FREQ[scaling]
    if c is None:
        return f, 1.0
    if c["kind"] == "linear":
        return f / c["factor"], 1.0
    if c["kind"] == "ntk":
        return (base * c["factor"] ** (rot / (rot - 2))) ** -i, 1.0
    turns = c["original"] * f / (2 * math.pi)  # of a pair over the original context
    if c["kind"] == "bands":
        share = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        return f * share + f / c["factor"] * (1 - share), 1.0
    at = [rot * math.log(c["original"] / (2 * math.pi * b)) / (2 * math.log(base)) for b in (c["beta_fast"], c["beta_slow"])]
    lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
    share = ((torch.arange(rot // 2, dtype=torch.float64, device=DEV) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f * (1 - share) + f / c["factor"] * share, 0.1 * c["mscale"] * math.log(c["factor"]) + 1


def _plain_rope(s):
    case = s["case"]
    f, m = _inv_freq(case["rot"], case["scaling"])
    angle = s["pos"].double()[:, None, None] * f
    cos, sin = (angle.cos() * m).float(), (angle.sin() * m).float()

    def rotate(x):
        y = x.float().clone()
        part = y[..., -case["rot"]:] if case["tail"] else y[..., :case["rot"]]
        if case["layout"] == "half":
            a, b = part[..., :case["rot"] // 2], part[..., case["rot"] // 2:]
        else:
            a, b = part[..., ::2], part[..., 1::2]
        u, v = a * cos - b * sin, b * cos + a * sin
        a.copy_(u)
        b.copy_(v)
        return y.to(x.dtype)

    return rotate(s["q"]), rotate(s["k"])


def _group_rows(s):
    """For every group: its query rows, and its keys and values [P, Hkv, D] with
    the scales applied, shard after shard."""
    case = s["case"]
    rows = _rows(s["prefix"], case["C"])
    if case["paged"]:
        at, there = _pool_rows(s["table"], s["prefix"], case["C"], s["page"])
    q0 = 0
    for g, n in enumerate(s["members"]):
        if case["paged"]:
            pairs = np.arange(case["C"]) * len(s["members"]) + g
            pick = at[pairs][there[pairs]]
            k, v = s["k"][0][pick], s["v"][0][pick]
        else:
            part = [slice(int(rows[r, :g].sum()), int(rows[r, :g + 1].sum())) for r in range(case["C"])]
            k, v = (torch.cat([x[p].to(torch.float32 if x.dtype != torch.bfloat16 else x.dtype) for x, p in zip(s[i], part)]) for i in "kv")
            if s["k_scale"] is not None:
                wide = torch.cat([x[p] for x, p in zip(s["k_scale"], part)])[:, None, None]
                k, v = k * wide, v * wide
        yield slice(q0, q0 + n), k, v
        q0 += n


def _plain_prefix(s):
    case = s["case"]
    N, Hq, Hkv, D = case["N"], case["Hq"], case["Hkv"], case["D"]
    o = torch.zeros((N, Hq, D), device=DEV)
    lse = torch.full((N, Hq), -math.inf, device=DEV)
    for rows, k, v in _group_rows(s):
        if k.shape[0] == 0:
            continue
        q = s["q"][rows].float().unflatten(1, (Hkv, -1))
        x = torch.matmul(q.permute(1, 2, 0, 3).flatten(1, 2), k.float().permute(1, 2, 0)) * s["scale"]
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        z = p.sum(-1, keepdim=True)
        back = lambda y: y.unflatten(1, (Hq // Hkv, -1)).permute(2, 0, 1, 3).reshape(q.shape[0], Hq, -1)  # noqa: E731
        o[rows] = back(torch.matmul(p, v.float().transpose(0, 1)) / z)
        lse[rows] = back(top + z.log())[..., 0]
    if case["parts"]:
        o, lse = torch.cat([o[None], s["o_part"]]), torch.cat([lse[None], s["lse_part"]])
        top = lse.amax(0)
        w = (lse - top.masked_fill(top == -math.inf, 0)).exp()
        z = w.sum(0)
        o, lse = (w[..., None] * o).sum(0) / z.clamp(min=1e-30)[..., None], top + z.log()
    return o.to(torch.bfloat16), lse


def _blocks(s, size, last=0):
    """Queries in blocks of one request: their rows, positions, and its keys as
    far as the last of them reads; `last`: only that many queries a request."""
    q0 = k0 = 0
    for n, pre in zip(s["new"], s["prefix"]):
        for a in range(max(0, n - last) if last else 0, n, size):
            e = min(n, a + size)
            yield slice(q0 + a, q0 + e), torch.arange(pre + a, pre + e, device=DEV), slice(k0, k0 + pre + e)
        q0, k0 = q0 + n, k0 + n + pre


def _plain_weights(s):
    case = s["case"]
    Hkv = case["Hkv"]
    lse = torch.empty_like(s["lse"])
    lse[s["order"]] = s["lse"]
    w = torch.zeros(s["k"].shape[0], device=DEV)
    for rows, pos, keys in _blocks(s, 512, case["window"]):
        q = s["q"][rows].float().unflatten(1, (Hkv, -1))
        x = torch.matmul(q.permute(1, 2, 0, 3).flatten(1, 2), s["k"][keys].float().permute(1, 2, 0)).unflatten(1, (q.shape[2], -1))
        x.mul_(s["scale"]).sub_(lse[rows].unflatten(1, (Hkv, -1)).permute(1, 2, 0)[..., None]).exp_()
        x.masked_fill_(torch.arange(x.shape[-1], device=DEV) > pos[:, None], 0.0)
        w[keys] += x.sum((0, 1, 2))
    return w


def _step_scores(s, dtype):
    """Scores [B, Hq, C * most] of a decode step, the pool row of each column
    and which columns exist."""
    case = s["case"]
    B, C, Hkv = case["B"], case["C"], case["Hkv"]
    at, there = _pool_rows(s["table"], s["L"], C, case["page"])
    at, there = (x.unflatten(0, (C, B)).transpose(0, 1).flatten(1) for x in (at, there))
    k = s["k"].reshape(-1, Hkv, case["D"])[at].to(dtype)  # [B, keys, Hkv, D]
    if s["k_scale"] is not None:
        k *= s["k_scale"].to(dtype)[at][..., None, None]
    q = s["q"].to(dtype).unflatten(1, (Hkv, -1))  # [B, Hkv, G, D]
    return torch.matmul(q, k.permute(0, 2, 3, 1)).flatten(1, 2) * s["scale"], at, there


def _plain_step(s):
    x, at, there = _step_scores(s, torch.float32)
    w = x.sub_(s["lse"][..., None]).exp_().sum(1)
    return s["w"].index_add(0, at[there], w[there])


def _plain_evict(s):
    case = s["case"]
    C, B = case["C"], case["B"]
    at, there = _pool_rows(s["table"], s["L"], C, case["page"])
    r = torch.arange(C, device=DEV)[:, None]
    rows = lambda L: ((L.long()[None, :] - r + C - 1).div(C, rounding_mode="floor")).clamp(min=0).reshape(-1, 1)  # noqa: E731
    m = torch.minimum(rows(s["keep_len"]), rows(s["ctx_len"]))
    pos = s["pos"][at]
    kept = (pos < 4) | (pos >= s["keep_from"].repeat(C)[:, None])
    key = torch.where(kept, math.inf, s["w"][at]).masked_fill(~there, -math.inf)
    best = key.argsort(dim=1, descending=True, stable=True)
    stay = torch.zeros_like(there).scatter(1, best, torch.arange(at.shape[1], device=DEV)[None, :] < m)
    i = torch.arange(at.shape[1], device=DEV)[None, :]
    hole, moved = ~stay & (i < m), stay & (i >= m)
    src, dst = (torch.full((C * B, s["most"] + 1), -1, dtype=torch.int64, device=DEV) for _ in range(2))
    for to, flag in ((src, moved), (dst, hole)):  # the i-th kept row past the new length takes the i-th hole
        to.scatter_(1, torch.where(flag, flag.cumsum(1) - 1, s["most"]), torch.where(flag, at, -1))
    src, dst, count = src[:, :-1], dst[:, :-1], moved.sum(1)
    a, b = src[src >= 0], dst[dst >= 0]
    for x in (s["k"], s["v"], s["k_scale"]):
        if x is not None:
            bits = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            bits[b] = bits[a]
    return [src.to(torch.int32), dst.to(torch.int32), count.to(torch.int32)] + [x for x in (s["k"], s["v"], s["k_scale"]) if x is not None]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "prefix": _plain_prefix, "weights": _plain_weights, "step": _plain_step, "evict": _plain_evict}[op](s)
    import context_long_attention_gb300 as cp
    if op == "rope":
        return cp.cp_rope(s["q"], s["k"], s["pos"], s["freqs"], layout=cp.CP_ROPE_HALF if case["layout"] == "half" else cp.CP_ROPE_INTERLEAVED, tail=case["tail"])
    if op == "prefix":
        parts = dict(o_part=s["o_part"], lse_part=s["lse_part"]) if case["parts"] else {}
        if case["paged"]:
            return cp.cp_prefix_attn_paged(s["plan"], s["pages"], s["q"], s["k"][0], s["v"][0], sm_scale=s["scale"], **parts)
        return cp.cp_prefix_attn(s["plan"], s["q"], s["k"], s["v"], s["k_scale"], sm_scale=s["scale"], **parts)
    if op == "weights":
        return cp.cp_prefill_weights(s["plan"], s["q"], s["k"], s["lse"], sm_scale=s["scale"], window=case["window"])
    if op == "step":
        w = s["w"].clone()
        cp.cp_decode_weights(s["plan"], s["pages"], cp.CP_DECODE_MLA if case["D"] == 576 else cp.CP_DECODE_GQA, s["q"], s["k"], s["lse"], w, scale_pool=s["k_scale"], sm_scale=s["scale"])
        return w
    src, dst, count = cp.cp_evict_select(s["pages"], case["C"], s["ctx_len"], s["keep_len"], s["w"], s["most"], pos=s["pos"], keep_below=4, keep_from=s["keep_from"])
    cp.cp_cache_move(src, dst, count, s["k"], s["v"], s["k_scale"])
    return [src, dst, count] + [x for x in (s["k"], s["v"], s["k_scale"]) if x is not None]


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "rope":
        elems = case["T"] * (case["Hq"] * case["Dq"] + case["Hk"] * case["Dk"])
        return {"bytes": 4 * elems + 4 * case["T"], "flops": 3 * case["T"] * (case["Hq"] + case["Hk"]) * case["rot"]}
    if op == "prefix":
        lens, members = _groups(case)
        P, row = sum(lens), case["Hkv"] * case["D"]
        out = case["N"] * case["Hq"]
        return {"bytes": P * (4 * row if case["kv"] == "bf16" else 2 * row + 4) + out * (4 * case["D"] + 4) + 4 * case["parts"] * out * (case["D"] + 1),
                "flops": 4 * case["Hq"] * case["D"] * sum(p * n for p, n in zip(lens, members))}
    if op == "weights":
        new, pre = _prompts(case)
        last = [min(n, case["window"] or n) for n in new]
        pairs = sum((p + n - w) * w + w * (w + 1) // 2 for n, p, w in zip(new, pre, last))
        KV = sum(new) + sum(pre)
        return {"bytes": 2 * KV * case["Hkv"] * case["D"] + sum(last) * case["Hq"] * (2 * case["D"] + 4) + 4 * KV, "flops": 2 * case["Hq"] * case["D"] * pairs}
    if op == "step":
        L = sum(_spread(case, case["ctx"], case["B"])[0])
        row = case["Hkv"] * case["D"]
        return {"bytes": L * ((2 * row if case["kv"] == "bf16" else row + 4) + 8) + case["B"] * case["Hq"] * (2 * case["D"] + 4), "flops": 2 * L * case["Hq"] * case["D"]}
    L = [case["ctx"]] * case["B"] if case["same"] else _spread(case, case["ctx"], case["B"])[0]
    rows = (case["dim"] if case["heads"] == 0 else 2 * case["heads"] * case["dim"]) * (2 if case["kv"] == "bf16" else 1)
    moved = 0  # as many rows as light ones are expected in front, of the rows that stay
    for n in L:
        k = min(case["keep"], n)
        moved += k * (n - k) // n
    return {"bytes": 8 * sum(L) + 2 * moved * rows, "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _exact_prefix(s):
    """Query by query heads in 64 bits, over the concatenated prefix and parts."""
    case = s["case"]
    G = case["Hq"] // case["Hkv"]
    o = torch.zeros((case["N"], case["Hq"], case["D"]), dtype=torch.float64, device=DEV)
    lse = torch.full((case["N"], case["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for rows, k, v in _group_rows({**s, "k": [x.double() for x in s["k"]], "v": [x.double() for x in s["v"]],
                                   "k_scale": None if s["k_scale"] is None else [x.double() for x in s["k_scale"]]}):
        for h in range(case["Hq"]):
            x = (s["q"][rows, h].double() @ k[:, h // G].double().T) * s["scale"]
            lse[rows, h] = torch.logsumexp(x, 1)
            if k.shape[0]:
                o[rows, h] = torch.softmax(x, 1) @ v[:, h // G].double()
    if case["parts"]:
        both = torch.cat([lse[None], s["lse_part"].double()])
        total = torch.logsumexp(both, 0)
        share = torch.nan_to_num((both - total).exp(), nan=0.0)
        o, lse = torch.einsum("pnh,pnhd->nhd", share, torch.cat([o[None], s["o_part"].double()])), total
    return o, lse


def _exact_weights(s):
    """Head by head in 64 bits, queries one request after another."""
    case = s["case"]
    G = case["Hq"] // case["Hkv"]
    w = torch.zeros(s["k"].shape[0], dtype=torch.float64, device=DEV)
    back = torch.argsort(s["order"])
    q0 = k0 = 0
    for n, pre in zip(s["new"], s["prefix"]):
        first = max(0, n - case["window"]) if case["window"] else 0
        for h in range(case["Hq"]):
            K = s["k"][k0:k0 + n + pre, h // G].double()
            for a in range(first, n, 4096):
                rows = torch.arange(a, min(n, a + 4096), device=DEV)
                x = s["q"][q0 + rows, h].double() @ K.T * s["scale"] - s["lse"][back[q0 + rows], h].double()[:, None]
                seen = torch.arange(n + pre, device=DEV) <= (pre + rows)[:, None]
                w[k0:k0 + n + pre] += torch.where(seen, x.exp(), 0.0).sum(0)
        q0, k0 = q0 + n, k0 + n + pre
    return w


def _exact_step(s):
    """Request by request, rows found token by token through the page table."""
    case = s["case"]
    table, C, page = s["table"].cpu().numpy().astype(np.int64), case["C"], case["page"]
    w = s["w"].double().clone()
    for b, n in enumerate(s["L"]):
        p = np.arange(n)
        at = torch.from_numpy(table[(p % C) * case["B"] + b, p // C // page] * page + p // C % page).to(DEV)
        k = s["k"][at].double().reshape(n, case["Hkv"], case["D"])
        if s["k_scale"] is not None:
            k = k * s["k_scale"][at].double()[:, None, None]
        x = torch.einsum("gid,kgd->gik", s["q"][b].double().unflatten(0, (case["Hkv"], -1)), k) * s["scale"]
        w[at] += (x.flatten(0, 1) - s["lse"][b].double()[:, None]).exp().sum(0)
    return w


def _exact_evict(s):
    """Pair by pair in numpy: a stable sort by weight, then the moves."""
    case = s["case"]
    C, B, page = case["C"], case["B"], case["page"]
    table, w, pos = s["table"].cpu().numpy().astype(np.int64), s["w"].cpu().numpy(), s["pos"].cpu().numpy()
    n_rows, m_rows, start = _rows(s["L"], C), _rows(s["keep"], C), s["keep_from"].cpu().numpy()
    src, dst = (np.full((C * B, s["most"]), -1, np.int32) for _ in range(2))
    count = np.zeros(C * B, np.int32)
    for pair in range(C * B):
        r, b = divmod(pair, B)
        n, m = int(n_rows[r, b]), int(m_rows[r, b])
        at = table[pair, np.arange(n) // page] * page + np.arange(n) % page
        heavy = np.where((pos[at] < 4) | (pos[at] >= start[b]), np.inf, w[at])
        stay = np.sort(np.argsort(-heavy, kind="stable")[:m])
        late = stay[stay >= m]
        holes = np.setdiff1d(np.arange(m), stay)
        count[pair] = late.size
        src[pair, :late.size], dst[pair, :late.size] = at[late], at[holes]
    out = [src, dst, count]
    a, b = torch.from_numpy(src[src >= 0]).long().to(DEV), torch.from_numpy(dst[dst >= 0]).long().to(DEV)
    for x in (s["k"], s["v"], s["k_scale"]):
        if x is not None:
            y = x.float()
            y[b] = y[a]
            out.append(y)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        f, m = _inv_freq(case["rot"], case["scaling"])
        turn = torch.exp(1j * s["pos"].double()[:, None, None] * f) * m
        out = []
        for x in (s["q"], s["k"]):
            y = x.double()
            part = y[..., -case["rot"]:] if case["tail"] else y[..., :case["rot"]]
            z = part.unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (-1, 2))
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            part.copy_((z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2))
            out.append(y)
        return out
    return {"prefix": _exact_prefix, "weights": _exact_weights, "step": _exact_step, "evict": _exact_evict}[op](s)
