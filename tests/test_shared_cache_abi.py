"""Rotary frequencies, plans over shared prefixes and the refusals of the calls
around a shared and thinned-out cache: answered on the host, with a message, before
any launch (no GPU needed)."""

import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def cp():
    import __graft_entry__
    __graft_entry__.ensure_built()
    import context_long_attention_gb300 as cp
    return cp


P = ctypes.c_void_p(256)  # never dereferenced: every case is answered before a launch
ODD = ctypes.c_void_p(264)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5
SCALINGS = [None, dict(kind="linear", factor=8.0), dict(kind="ntk", factor=4.0),
            dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0), dict(kind="yarn", factor=40.0, original=4096)]


def refuse(lib, status, words, got):
    assert got == status and words in lib.cp_last_error(), (got, lib.cp_last_error())


def test_frequencies(cp):
    """What the scalings do at their ends."""
    f = cp.cp_rope_freqs(64)
    assert f.inv_freq[0] == 1 and math.isclose(f.inv_freq[-1], 10000.0 ** (-62 / 64))
    assert np.allclose(cp.cp_rope_freqs(64, scaling=SCALINGS[1]).inv_freq, f.inv_freq / 8)
    n = cp.cp_rope_freqs(64, scaling=SCALINGS[2]).inv_freq
    assert n[0] == 1 and math.isclose(n[-1], f.inv_freq[-1] / 4)
    b = cp.cp_rope_freqs(64, scaling=SCALINGS[3]).inv_freq
    assert b[0] == 1 and math.isclose(b[-1], f.inv_freq[-1] / 8)
    y = cp.cp_rope_freqs(64, scaling=SCALINGS[4])
    assert y.inv_freq[0] == 1 and math.isclose(y.inv_freq[-1], f.inv_freq[-1] / 40) and math.isclose(y.scale, 0.1 * math.log(40) + 1)
    assert f.turns[0].item() == round(2.0**64 / (2 * math.pi)) and f.rot == 64
    for bad in (dict(kind="linear", factor=0.5), dict(kind="other", factor=2), dict(kind="bands", factor=2, low=1, high=4)):
        with pytest.raises(ValueError):
            cp.cp_rope_freqs(64, scaling=bad)
    with pytest.raises(ValueError):
        cp.cp_rope_freqs(63)


def test_rope(cp):
    lib = cp.lib

    def call(T=4, pos=P, turns=P, rot=64, layout=0, scale=1.0, dtype=0, q=P, qs=256, Hq=2, Dq=128, qo=P, qos=256, k=P, ks=128, Hk=1, Dk=128,
             ko=P, kos=128):
        return lib.cp_rope(T, pos, turns, rot, layout, 0, 0, scale, dtype, q, qs, Hq, Dq, qo, qos, k, ks, Hk, Dk, ko, kos, None)

    refuse(lib, INVALID, b"T=-1", call(T=-1))
    refuse(lib, INVALID, b"layout", call(layout=2))
    refuse(lib, UNSUPPORTED, b"dtype", call(dtype=2))
    for rot in (0, 8, 24, 1040, -16):
        refuse(lib, UNSUPPORTED, b"rot=", call(rot=rot))
    for scale in (0.0, -1.0, float("nan")):
        refuse(lib, INVALID, b"scale", call(scale=scale))
    refuse(lib, INVALID, b"q_heads", call(Hq=0))
    refuse(lib, INVALID, b"q_heads", call(Hk=-1))
    refuse(lib, UNSUPPORTED, b"head dim", call(Dq=48))
    refuse(lib, UNSUPPORTED, b"head dim", call(Dk=132))
    for st in (248, 260, 0, -256, 1 << 40):
        refuse(lib, INVALID, b"stride", call(qs=st))
        refuse(lib, INVALID, b"stride", call(kos=st if st != 248 else 120))
    refuse(lib, UNSUPPORTED, b"262,144", call(Hq=4096, qs=1 << 20, qos=1 << 20))
    refuse(lib, UNSUPPORTED, b"262,144", call(Hq=1 << 30, qs=1 << 20, qos=1 << 20))
    refuse(lib, INVALID, b"NULL", call(pos=None))
    refuse(lib, INVALID, b"NULL", call(ko=None))
    refuse(lib, INVALID, b"8-byte", call(turns=ctypes.c_void_p(260)))
    refuse(lib, INVALID, b"aligned", call(q=ODD))
    refuse(lib, INVALID, b"two strides", call(qos=512))
    assert call(T=0, pos=None, q=None) == 0


PLANS = [(8, [32768], [64], 32, 8, 152), (1, [4096], [4], 32, 8, 152), (3, [1000, 0, 5], [3, 4, 5], 8, 2, 7), (2, [200, 77], [0, 100], 64, 8, 400),
         (5, [0, 0], [1, 2], 4, 4, 3), (64, [100000, 3], [1000, 1], 6, 2, 152)]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("C,lens,members,Hq,Hkv,workers", PLANS)
def test_prefix_plan(cp, C, lens, members, Hq, Hkv, workers, layout):
    """Every tile of every block belongs to one item, in order; parts are the
    items' own and a block's are consecutive; costs are even."""
    p = cp.cp_prefix_plan(C, lens, members, Hq, Hkv, layout, workers)
    d = cp.cp_decode_plan_ex(C, lens, layout=layout, n_workers=1)
    assert np.array_equal(p.pairs[:, [0, 1, 2, 5, 6]], d.pairs[:, [0, 1, 2, 5, 6]]) and p.shard_rows() == d.shard_rows()
    G = Hq // Hkv
    for g in range(len(lens)):
        rows = [int(p.pairs[r * len(lens) + g, 0]) for r in range(C)]
        assert p.tile_off[g].tolist() == np.concatenate([[0], np.cumsum([-(-n // 128) for n in rows])]).tolist()
    first = np.concatenate([[0], np.cumsum(members)])
    blocks = {(int(b[0]), int(b[1]), int(b[3])): b for b in p.blocks}
    assert len(blocks) == sum(Hkv * -(-m * G // 256) for m in members)
    seen = {k: [] for k in blocks}
    assert p.worker_off[0] == 0 and p.worker_off[-1] == len(p.items) and (np.diff(p.worker_off) >= 0).all()
    for it in p.items:
        key = (int(it[0]), int(it[1]), int(it[3]))
        b = blocks[key]
        assert it[2] == b[2] == first[it[0]] and it[4] == b[4] == min(256, members[it[0]] * G - it[3]) and it[8] == (b[6] == 1)
        assert it[6] > it[5] and it[7] == b[5] + len(seen[key])
        seen[key].append((int(it[5]), int(it[6])))
    for key, b in blocks.items():
        total = int(p.tile_off[key[0]][-1])
        assert len(seen[key]) == b[6] and [x for x, _ in seen[key]] + [total] == [0] * (total > 0) + [y for _, y in seen[key]] + [0] * (total == 0)
    assert sorted(int(i[7]) for i in p.items) == list(range(p.n_parts))
    assert [b[6] != 1 for b in p.blocks] == [True] * p.n_merge + [False] * (len(p.blocks) - p.n_merge)
    cost = [sum((int(i[6]) - int(i[5])) * (16 if i[4] > 128 else 14) for i in p.items[p.worker_off[w]:p.worker_off[w + 1]]) for w in range(workers)]
    whole = sum(cost) + 64 * sum(1 for b in p.blocks if b[6])
    assert max(cost, default=0) <= whole / workers + 16 + 16
    need = [cp.cp_prefix_workspace_size(p, 128, n) for n in (0, 1)]
    assert need[1] == p.n_parts * 256 * 129 * 4 and need[0] == sum(int(b[6]) for b in p.blocks[:p.n_merge]) * 256 * 129 * 4


def test_prefix_plan_refusals(cp):
    for args, words in [((0, [1], [1], 4, 2), "C=0"), ((65, [1], [1], 4, 2), "C=65"), ((1, [-1], [1], 4, 2), "ctx_len"), ((1, [1], [-1], 4, 2), "members"),
                        ((1, [1], [0], 4, 2), "no query rows"), ((1, [1], [1], 4, 3), "multiple"), ((1, [1], [1], 0, 2), "multiple"),
                        ((1, [2**30, 2**30], [1, 1], 4, 2), "total tokens"), ((1, [1], [2**30], 4, 2), "past 2")]:
        with pytest.raises(cp.CpError, match=words):
            cp.cp_prefix_plan(*args, n_workers=4)
    with pytest.raises(cp.CpError, match="layout"):
        cp.cp_prefix_plan(1, [1], [1], 4, 2, layout=2, n_workers=4)
    with pytest.raises(cp.CpError, match="n_workers"):
        cp.cp_prefix_plan(1, [1], [1], 4, 2, n_workers=-1)
    with pytest.raises(cp.CpError, match="n_workers"):
        cp.cp_prefix_plan(1, [1], [1], 4, 2, n_workers=2**31 - 1)
    with pytest.raises(ValueError, match="one length"):
        cp.cp_prefix_plan(1, [1, 2], [1], 4, 2, n_workers=4)


def test_prefix_attn(cp):
    lib = cp.lib
    plan = cp.cp_prefix_plan(2, [300], [3], 8, 2, n_workers=4)
    h = plan.host.ctypes.data_as(ctypes.c_void_p)
    two = (ctypes.c_void_p * 2)(256, 256)

    def call(host=h, dev=P, dtype=0, q=P, k=two, v=two, sc=None, Hq=8, Hkv=2, D=128, scale=0.1, parts=0, oo=None, ol=None, o=P, od=0, lse=P, ws=P,
             wsb=1 << 30):
        return lib.cp_prefix_attn(host, dev, dtype, q, k, v, sc, Hq, Hkv, D, scale, parts, oo, ol, o, od, lse, ws, wsb, None)

    refuse(lib, INVALID, b"host_plan is NULL", call(host=None))
    decode = cp.cp_decode_plan(2, [300], n_workers=2)
    refuse(lib, INVALID, b"expected a shared-prefix plan", call(host=decode.host.ctypes.data_as(ctypes.c_void_p)))
    with pytest.raises(cp.CpError, match="expected a decode plan"):
        cp.cp_decode_workspace_size(plan, 8, 128)
    refuse(lib, INVALID, b"expected a prefill plan", lib.cp_prefill_attn(h, P, -1, 0, P, P, P, 8, 2, 128, 0.1, P, P, None))
    for kw in (dict(dev=None), dict(q=None), dict(k=None), dict(o=None), dict(lse=None)):
        refuse(lib, INVALID, b"NULL", call(**kw))
    for kw in (dict(dev=ODD), dict(q=ODD), dict(o=ODD), dict(lse=ODD)):
        refuse(lib, INVALID, b"aligned", call(**kw))
    refuse(lib, INVALID, b"needs shard_v", call(v=None))
    refuse(lib, INVALID, b"shard_scale", call(sc=two))
    refuse(lib, INVALID, b"shard_scale", call(dtype=2))
    refuse(lib, INVALID, b"o_dtype", call(od=2))
    for D in (0, 33, 288, 576):
        refuse(lib, UNSUPPORTED, b"multiple of 32", call(D=D))
    refuse(lib, INVALID, b"the plan was made for 8 and 2", call(Hq=16))
    refuse(lib, INVALID, b"the plan was made for 8 and 2", call(Hkv=4))
    for parts in (-1, 65):
        refuse(lib, INVALID, b"P=", call(parts=parts))
    refuse(lib, INVALID, b"own_o", call(parts=1, ol=P))
    refuse(lib, INVALID, b"own_o", call(parts=1, oo=ODD, ol=P))
    refuse(lib, WORKSPACE, b"workspace", call(parts=1, oo=P, ol=P, wsb=16))
    refuse(lib, WORKSPACE, b"workspace", call(parts=1, oo=P, ol=P, ws=None))
    refuse(lib, INVALID, b"ws is not", call(parts=1, oo=P, ol=P, ws=ODD))
    for scale in (0.0, float("nan")):
        refuse(lib, INVALID, b"sm_scale", call(scale=scale))
    refuse(lib, INVALID, b"shard_k[1]", call(k=(ctypes.c_void_p * 2)(256, None)))
    refuse(lib, INVALID, b"shard_k[0]", call(v=(ctypes.c_void_p * 2)(264, 256)))

    table = np.zeros((2, 3), np.int32)
    table[0], table[1] = [0, 1, 2], [3, 4, 5]

    def paged(t=table, page=64, num=6, most=3, kp=P):
        return lib.cp_prefix_attn_paged(h, P, 0, P, kp, P, None, t.ctypes.data_as(ctypes.c_void_p), P, most, page, num, 8, 2, 128, 0.1, 0, None, None,
                                        P, 0, P, P, 1 << 30, None)

    refuse(lib, UNSUPPORTED, b"page_size", paged(page=96))
    refuse(lib, INVALID, b"outside", paged(num=5))
    refuse(lib, INVALID, b"max_pages", paged(most=2))
    refuse(lib, INVALID, b"aligned", paged(kp=ODD))
    bad = table.copy()
    bad[1, 2] = -1
    refuse(lib, INVALID, b"outside", paged(t=bad))


def test_weights(cp):
    lib = cp.lib
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [5], [3], device=None)
    h = plan.host.ctypes.data_as(ctypes.c_void_p)

    def prompt(host=h, dev=P, dtype=0, q=P, k=P, lse=P, Hq=4, Hkv=2, D=128, scale=0.1, window=0, out=P, ws=P, wsb=1 << 30):
        return lib.cp_prefill_weights(host, dev, dtype, q, k, lse, Hq, Hkv, D, scale, window, out, ws, wsb, None)

    refuse(lib, INVALID, b"magic", prompt(host=np.zeros(64, np.int32).ctypes.data_as(ctypes.c_void_p)))
    refuse(lib, INVALID, b"multiple", prompt(Hkv=3))
    refuse(lib, UNSUPPORTED, b"dtype", prompt(dtype=2))
    refuse(lib, UNSUPPORTED, b"D in", prompt(D=96))
    refuse(lib, UNSUPPORTED, b"head dim", prompt(D=256, dtype=1))
    refuse(lib, INVALID, b"sm_scale", prompt(scale=float("nan")))
    refuse(lib, INVALID, b"window", prompt(window=-1))
    for kw in (dict(dev=None), dict(q=None), dict(k=None), dict(lse=None), dict(out=None)):
        refuse(lib, INVALID, b"NULL", prompt(**kw))
    for kw in (dict(dev=ODD), dict(q=ODD), dict(k=ODD), dict(lse=ODD), dict(out=ODD)):
        refuse(lib, INVALID, b"aligned", prompt(**kw))

    dplan = cp.cp_decode_plan(1, [100, 70], n_workers=2)
    d = dplan.host.ctypes.data_as(ctypes.c_void_p)
    table = np.array([[0, 1], [2, 3]], np.int32)

    def step(host=d, dev=P, mode=0, dtype=0, q=P, k=P, sc=None, t=table, page=64, num=4, Hq=4, Hkv=2, D=128, scale=0.1, lse=P, w=P):
        return lib.cp_decode_weights(host, dev, mode, dtype, q, k, sc, t.ctypes.data_as(ctypes.c_void_p), P, 2, page, num, Hq, Hkv, D, scale, lse, w, None)

    refuse(lib, INVALID, b"expected a decode plan", step(host=h))
    refuse(lib, INVALID, b"selection", step(host=cp.cp_sparse_plan(1, 2, 16, n_workers=2).host.ctypes.data_as(ctypes.c_void_p)))
    for kw in (dict(dev=None), dict(q=None), dict(k=None), dict(lse=None), dict(w=None)):
        refuse(lib, INVALID, b"NULL", step(**kw))
    for kw in (dict(q=ODD), dict(k=ODD), dict(lse=ODD), dict(w=ODD)):
        refuse(lib, INVALID, b"aligned", step(**kw))
    refuse(lib, UNSUPPORTED, b"MLA needs", step(mode=1))
    refuse(lib, UNSUPPORTED, b"outside [1, 64]", step(mode=1, Hq=65, Hkv=1, D=576))
    refuse(lib, INVALID, b"shard_scale", step(dtype=2))
    refuse(lib, INVALID, b"shard_scale", step(sc=P))
    refuse(lib, INVALID, b"used twice", step(t=np.array([[0, 1], [1, 3]], np.int32)))
    refuse(lib, INVALID, b"outside", step(num=2))
    refuse(lib, UNSUPPORTED, b"page_size", step(page=32))


def test_eviction(cp):
    lib = cp.lib

    def select(C=2, B=2, ctx=P, keep=P, t=P, most=3, page=64, num=8, w=P, moves=9, src=P, dst=P, count=P):
        return lib.cp_evict_select(C, B, ctx, keep, t, most, page, num, w, None, 0, None, moves, src, dst, count, None)

    refuse(lib, INVALID, b"C=0", select(C=0))
    refuse(lib, INVALID, b"C=65", select(C=65))
    refuse(lib, INVALID, b"B=8193", select(B=8193))
    refuse(lib, UNSUPPORTED, b"page_size", select(page=100))
    refuse(lib, UNSUPPORTED, b"too large", select(num=1 << 26))
    refuse(lib, INVALID, b"max_pages", select(most=0))
    refuse(lib, UNSUPPORTED, b"rows a pair", select(most=1 << 25))
    for moves in (0, -1, 1 << 30):
        refuse(lib, INVALID, b"max_moves", select(moves=moves))
    for kw in (dict(ctx=None), dict(keep=None), dict(t=None), dict(w=None), dict(src=None), dict(dst=None), dict(count=None)):
        refuse(lib, INVALID, b"NULL", select(**kw))

    def move(pairs=4, most=9, src=P, dst=P, count=P, k=P, v=None, rb=256, rows=512):
        return lib.cp_cache_move(pairs, most, src, dst, count, k, v, rb, None, None, None, rows, None)

    refuse(lib, INVALID, b"pairs", move(pairs=-1))
    refuse(lib, INVALID, b"max_moves", move(most=0))
    refuse(lib, INVALID, b"pool_rows", move(rows=0))
    for rb in (0, 8, 100, -16):
        refuse(lib, UNSUPPORTED, b"row_bytes", move(rb=rb))
    for kw in (dict(src=None), dict(dst=None), dict(count=None), dict(k=None)):
        refuse(lib, INVALID, b"NULL", move(**kw))
    refuse(lib, INVALID, b"aligned", move(v=ODD))
    assert move(pairs=0, src=None) == 0

    info = ctypes.c_void_p(512)

    def release(C=2, B=2, ctx=P, t=P, free=P, n=5, at=P, i=info):
        return lib.cp_page_release(C, B, ctx, P, t, 3, 64, 8, free, n, at, None, None, i, None)

    refuse(lib, INVALID, b"B=0", release(B=0))
    refuse(lib, INVALID, b"n_free", release(n=-1))
    for kw in (dict(ctx=None), dict(t=None), dict(free=None), dict(at=None), dict(i=None)):
        refuse(lib, INVALID, b"NULL", release(**kw))
    refuse(lib, INVALID, b"info is not", release(i=ODD))
    refuse(lib, INVALID, b"free_pos lies", release(at=ctypes.c_void_p(516)))
