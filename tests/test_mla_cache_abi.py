"""Refusals of the latent-attention and cache-append entry points: every bad
argument is answered before a launch (no GPU needed), with a message."""

import ctypes

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
INVALID, UNSUPPORTED = -1, -2


def refuse(lib, status, words, got):
    assert got == status and words in lib.cp_last_error(), (got, lib.cp_last_error())


def test_products(cp):
    lib = cp.lib
    refuse(lib, INVALID, b"H >= 1", lib.cp_mla_expand(P, 512, P, 4, 0, P, None))
    refuse(lib, INVALID, b"T >= 0", lib.cp_mla_expand(P, 512, P, -1, 2, P, None))
    for stride in (504, 516, 0, -512, 1 << 40):
        refuse(lib, INVALID, b"latent_stride", lib.cp_mla_expand(P, stride, P, 4, 2, P, None))
    refuse(lib, INVALID, b"NULL", lib.cp_mla_expand(None, 512, P, 4, 2, P, None))
    refuse(lib, INVALID, b"aligned", lib.cp_mla_expand(P, 512, ODD, 4, 2, P, None))
    for fn in (lib.cp_mla_absorb, lib.cp_mla_project):
        refuse(lib, INVALID, b"N >= 0", fn(P, P, -1, 2, P, None))
        refuse(lib, INVALID, b"H >= 1", fn(P, P, 1, 0, P, None))
        refuse(lib, INVALID, b"NULL", fn(P, P, 1, 2, None, None))
        refuse(lib, INVALID, b"aligned", fn(ODD, P, 1, 2, P, None))
        assert fn(None, None, 0, 2, None, None) == 0
    assert lib.cp_mla_expand(None, 0, None, 0, 2, None, None) == 0


def test_prefill(cp):
    lib = cp.lib
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [5], [3], device=None)
    h = plan.host.ctypes.data_as(ctypes.c_void_p)

    def call(host=h, dev=P, rank=-1, q=P, rope=P, stride=576, H=2, scale=0.1, lse=P):
        return lib.cp_mla_prefill_attn(host, dev, rank, q, P, rope, stride, H, scale, P, lse, None)

    refuse(lib, INVALID, b"host_plan is NULL", call(host=None))
    bogus = np.zeros(64, np.int32)
    refuse(lib, INVALID, b"magic", call(host=bogus.ctypes.data_as(ctypes.c_void_p)))
    decode = cp.cp_decode_plan(2, [5], n_workers=2)
    refuse(lib, INVALID, b"expected a prefill plan", call(host=decode.host.ctypes.data_as(ctypes.c_void_p)))
    for rank in (-2, 2):
        refuse(lib, INVALID, b"rank", call(rank=rank))
    refuse(lib, INVALID, b"H=0", call(H=0))
    for scale in (0.0, -1.0, float("nan")):
        refuse(lib, INVALID, b"sm_scale", call(scale=scale))
    refuse(lib, INVALID, b"NULL", call(dev=None))
    refuse(lib, INVALID, b"NULL", call(lse=None))
    refuse(lib, INVALID, b"aligned", call(rope=ODD))
    for stride in (56, 68, -64, 1 << 40):
        refuse(lib, INVALID, b"rope_stride", call(stride=stride))
    old = plan.host.copy()
    old[cp._binding.HEADER_FIELDS.index("off_run")] = 0
    refuse(lib, INVALID, b"no request tiles", call(host=old.ctypes.data_as(ctypes.c_void_p)))
    empty = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [0], [3], device=None)
    assert call(host=empty.host.ctypes.data_as(ctypes.c_void_p), dev=None, q=None) == 0  # no query: nothing to do


@pytest.mark.parametrize("strategy,C", [(0, 1), (0, 8), (1, 3)])
def test_request_tiles_of_a_plan(cp, strategy, C):
    """The request tiles cover every request's new tokens once, 256 and 512 at a
    time, those whose last query has most keys first; each holds its request."""
    new, prefix = [700, 0, 1, 256, 513, 90], [5, 3, 4000, 0, 77, 0]
    plan = cp.cp_shard_plan(strategy, C, new, prefix, device=None)
    at = plan.off_run
    for size in (256, 512):
        want = [(j, o) for j, n in enumerate(new) for o in range(0, n, size)]
        tiles = plan.words(at, 8 * len(want)).reshape(-1, 8).tolist()
        at += 8 * len(want)
        assert size == 512 or plan.n_parts == len(want)
        assert sorted((t[0], t[1]) for t in tiles) == want
        for j, _, n, pre, q_base, kv_base, *_ in tiles:
            assert (n, pre, q_base, kv_base) == (new[j], prefix[j], sum(new[:j]), sum(new[:j]) + sum(prefix[:j]))
        keys = [prefix[j] + min(o + size, new[j]) for j, o, *_ in tiles]
        assert keys == sorted(keys, reverse=True)


def test_page_slots(cp):
    lib = cp.lib
    pos, info = ctypes.c_void_p(512), ctypes.c_void_p(1024)

    def call(C=2, B=3, ctx=P, max_pages=4, page=64, num=10, free=P, n_free=5, pos=pos, slots=P, most=8, info=info):
        return lib.cp_page_slots(C, B, ctx, P, P, max_pages, page, num, free, n_free, pos, slots, most, P, info, None)

    for C in (0, 65, -1):
        refuse(lib, INVALID, b"C=", call(C=C))
    for B in (0, -1, 8193):
        refuse(lib, INVALID, b"B=", call(B=B))
    for page in (0, 32, 96, -64):
        refuse(lib, UNSUPPORTED, b"multiple of 64", call(page=page))
    refuse(lib, INVALID, b"max_pages", call(max_pages=0))
    refuse(lib, INVALID, b"num_pages", call(num=0))
    refuse(lib, UNSUPPORTED, b"too large", call(num=1 << 25))
    refuse(lib, INVALID, b"n_free", call(n_free=-1))
    refuse(lib, INVALID, b"max_tokens", call(most=-1))
    refuse(lib, INVALID, b"NULL", call(ctx=None))
    refuse(lib, INVALID, b"NULL", call(free=None))
    refuse(lib, INVALID, b"NULL", call(slots=None))
    refuse(lib, INVALID, b"aligned", call(slots=ODD))
    for k in range(4):
        refuse(lib, INVALID, b"earlier call", call(pos=ctypes.c_void_p(1024 + 4 * k)))


def test_cache_append(cp):
    lib = cp.lib
    BF16, FP32, FP8 = cp.CP_BF16, cp.CP_FP32, cp.CP_FP8_E4M3

    def call(slots=P, n=4, src=BF16, k=P, ks=576, v=None, vs=0, ns=None, row=576, pool=BF16, kp=P, vp=None, sp=None, rows=64):
        return lib.cp_cache_append(slots, n, src, k, ks, v, vs, ns, row, pool, kp, vp, sp, rows, None)

    refuse(lib, INVALID, b"bad dtype", call(src=7))
    for src, pool, sp in ((BF16, FP32, None), (FP32, BF16, None), (FP8, BF16, None)):
        refuse(lib, UNSUPPORTED, b"own dtype", call(src=src, pool=pool, sp=sp))
    for row in (0, 8, 24, -16):
        refuse(lib, UNSUPPORTED, b"row_elems", call(row=row))
    refuse(lib, INVALID, b"n=-1", call(n=-1))
    for rows in (0, 1 << 31):
        refuse(lib, INVALID, b"pool_rows", call(rows=rows))
    refuse(lib, INVALID, b"v_new and v_pool", call(v=P))
    refuse(lib, INVALID, b"v_new and v_pool", call(vp=P))
    refuse(lib, INVALID, b"scale_pool", call(pool=FP8))
    refuse(lib, INVALID, b"scale_pool", call(sp=P))
    refuse(lib, INVALID, b"new_scale", call(src=FP8, pool=FP8, sp=P))
    refuse(lib, INVALID, b"new_scale", call(ns=P))
    for ks in (568, 580, 0, -576):
        refuse(lib, INVALID, b"row stride", call(ks=ks))
    refuse(lib, INVALID, b"row stride", call(v=P, vp=P, vs=8))
    refuse(lib, INVALID, b"NULL", call(k=None))
    refuse(lib, INVALID, b"aligned", call(kp=ODD))
    refuse(lib, INVALID, b"aligned", call(v=ODD, vp=P, vs=576))
    assert call(n=0, slots=None, k=None, kp=None) == 0


def test_binding_checks(cp):
    """The binding answers host tensors, wrong dtypes and shapes itself."""
    import torch
    w = torch.zeros(2, 256, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        cp.cp_mla_expand(torch.zeros(3, 512, dtype=torch.bfloat16), w)
    with pytest.raises(TypeError, match="latent"):
        cp.cp_mla_expand(torch.zeros(3, 512), w)
    with pytest.raises(ValueError, match="CUDA"):
        cp.cp_mla_absorb(torch.zeros(3, 2, 192, dtype=torch.bfloat16), w)
    with pytest.raises(TypeError, match="w_kv"):
        cp.cp_mla_project(torch.zeros(3, 2, 512, dtype=torch.bfloat16), w.float())
    pages = cp.PageTable(np.zeros((4, 2)), 64, 8)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device copy"):
        cp.cp_page_slots(pages, 2, i32, i32, i32, i32[:1], 4)
    with pytest.raises(ValueError, match="int32 CUDA"):
        cp.PageTable.on_device(torch.zeros(4, 2, dtype=torch.int32), 64, 8)
    with pytest.raises(ValueError, match="CUDA"):
        cp.cp_cache_append(i32, torch.zeros(2, 576), torch.zeros(64, 576))


def host_only(monkeypatch, cp, **calls):
    """The binding's own steps around calls that only record their arguments."""
    b = cp._binding
    monkeypatch.setattr(b, "_need", lambda name, t, *rest: t)
    monkeypatch.setattr(b, "_device_index", lambda: -1)
    monkeypatch.setattr(b, "_raw_stream", lambda index: None)
    for name, status in calls.items():
        monkeypatch.setattr(b.lib, name, lambda *a, status=status: status)


@pytest.mark.parametrize("synced", [False, True])
def test_page_slots_drops_the_host_copy(cp, monkeypatch, synced):
    """The paged pack and decode check the host copy of a table: after a
    slots call it no longer holds the table's ids, and both ask for sync_host()."""
    import torch
    host_only(monkeypatch, cp, cp_page_slots=0)
    i32 = dict(dtype=torch.int32)
    pages = cp.PageTable(np.zeros((4, 2)), 64, 8, device="cpu")
    if synced:
        pages.dev.fill_(3)
        assert (pages.sync_host().host == 3).all()
    out = dict(slots=torch.zeros(4, **i32), cu_new=torch.zeros(3, **i32), info=torch.zeros(4, **i32))
    two = torch.zeros(2, **i32)
    cp.cp_page_slots(pages, 2, two, two, two, two[:1], 4, **out)
    plan = cp.cp_decode_plan(2, [5, 5], n_workers=2)
    x = torch.zeros(10, 576, dtype=torch.bfloat16)
    monkeypatch.setattr(cp._binding, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(cp._binding, "_stream", lambda d: None)
    with pytest.raises(ValueError, match="sync_host"):
        cp.cp_kv_shard_pack_paged(plan, pages, x, pool=x)
    o = dict(o_part=torch.zeros(1), lse_part=torch.zeros(1), ws=torch.zeros(1))
    with pytest.raises(ValueError, match="sync_host"):
        cp.cp_decode_attn_paged(plan, pages, cp.CP_DECODE_MLA, torch.zeros(2, 1, 576, dtype=torch.bfloat16), x, sm_scale=1.0, **o)
    pages.dev.fill_(5)
    assert (pages.sync_host().host == 5).all()  # and have it from then on


def test_page_slots_that_fails_keeps_the_host_copy(cp, monkeypatch):
    import torch
    host_only(monkeypatch, cp, cp_page_slots=INVALID)
    pages = cp.PageTable(np.zeros((4, 2)), 64, 8, device="cpu")
    two = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(cp.CpError):
        cp.cp_page_slots(pages, 2, two, two, two, two[:1], 4, slots=two, cu_new=two, info=two)
    assert (pages.host == 0).all()


def test_prefill_takes_the_rotated_columns_only(cp, monkeypatch):
    """A k_rope of other columns or rows than the plan's [KV, 64], such as the
    whole cache entries, is refused."""
    import torch
    host_only(monkeypatch, cp, cp_mla_prefill_attn=0)
    monkeypatch.setattr(cp._binding, "_rows", lambda name, t, cols, dtype, dev: (t.data_ptr(), t.stride(0)))
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [5], [3], device=None)
    plan.dev = torch.from_numpy(plan.host)
    bf = dict(dtype=torch.bfloat16)
    q, kv, lat = torch.zeros(5, 2, 192, **bf), torch.zeros(8, 2, 256, **bf), torch.zeros(9, 576, **bf)
    out = dict(out=torch.zeros(5, 2, 128, **bf), lse=torch.zeros(5, 2))
    cp.cp_mla_prefill_attn(plan, q, kv, lat[:8, 512:], **out)
    for rope in (lat[:8], lat[:8, 448:], lat[:8, 520:], lat[:, 512:], lat[:7, 512:]):
        with pytest.raises(ValueError, match="k_rope"):
            cp.cp_mla_prefill_attn(plan, q, kv, rope, **out)


def test_outputs_come_from_torch(cp, monkeypatch):
    """The calls' own outputs are made through torch's dispatcher, on their
    inputs' device: a mode sees them."""
    import torch
    from torch.utils._python_dispatch import TorchDispatchMode

    class Made(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if func is torch.ops.aten.empty.memory_format:
                self.made.append(out)
            return out

    host_only(monkeypatch, cp, cp_page_slots=0, cp_mla_expand=0, cp_mla_absorb=0, cp_mla_project=0, cp_mla_prefill_attn=0)
    monkeypatch.setattr(cp._binding, "_rows", lambda name, t, cols, dtype, dev: (t.data_ptr(), t.stride(0)))
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG, 2, [5], [3], device=None)
    plan.dev = torch.from_numpy(plan.host)
    pages, two = cp.PageTable(np.zeros((4, 2)), 64, 8, device="cpu"), torch.zeros(2, **i32)
    w, lat = torch.zeros(2, 256, 512, **bf), torch.zeros(8, 576, **bf)
    q, kv = torch.zeros(5, 2, 192, **bf), torch.zeros(8, 2, 256, **bf)
    mode = Made()
    mode.made = []
    with mode:
        got = [cp.cp_mla_expand(lat, w), cp.cp_mla_absorb(q, w), cp.cp_mla_absorb(q[None], w), cp.cp_mla_project(torch.zeros(2, 512, **bf), w),
               *cp.cp_mla_prefill_attn(plan, q, kv, lat[:, 512:]), *cp.cp_mla_prefill_attn(plan, q, kv, lat[:, 512:], rank=1),
               *cp.cp_page_slots(pages, 2, two, two, two, two[:1], 7)]
    want = [((8, 2, 256), bf), ((5, 2, 576), bf), ((1, 5, 2, 576), bf), ((2, 128), bf), ((5, 2, 128), bf), ((5, 2), dict(dtype=torch.float32)),
            ((plan.rank_rows(1), 2, 128), bf), ((plan.rank_rows(1), 2), dict(dtype=torch.float32)), ((7,), i32), ((3,), i32), ((4,), i32)]
    assert [(tuple(t.shape), dict(dtype=t.dtype)) for t in got] == want
    assert all(t.is_contiguous() and any(t.data_ptr() == m.data_ptr() for m in mode.made) for t in got)


def test_counts_past_31_bits(cp, monkeypatch):
    """Counts that the C interface cannot hold are refused, not cut to 32 bits."""
    import torch
    host_only(monkeypatch, cp, cp_page_slots=0, cp_cache_append=0)
    pages, two = cp.PageTable(np.zeros((4, 2)), 64, 8, device="cpu"), torch.zeros(2, dtype=torch.int32)
    out = dict(slots=two, cu_new=two, info=two)
    for n in (2**31, 2**32 + 5):
        many = two[:1].expand(n)
        with pytest.raises(ValueError, match="max_tokens"):
            cp.cp_page_slots(pages, 2, two, two, two, two[:1], n, **out)
        with pytest.raises(ValueError, match="n_free"):
            cp.cp_page_slots(pages, 2, two, two, many, two[:1], 4, **out)
        assert pages.host is not None
        with pytest.raises(ValueError, match="slots"):
            cp.cp_cache_append(many, torch.zeros(1, 16).expand(n, 16), torch.zeros(64, 16))


def test_paged_calls_need_a_row_for_every_pair(cp, monkeypatch):
    """A table of a smaller batch than the plan's is refused by the paged pack and
    decode (the library reads a row of both copies for every pair)."""
    import torch
    b = cp._binding
    monkeypatch.setattr(b, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(b, "_stream", lambda d: None)
    monkeypatch.setattr(b, "_ptr", lambda t: None)
    monkeypatch.setattr(b.lib, "cp_kv_shard_pack_paged", lambda *a: 0)
    monkeypatch.setattr(b.lib, "cp_decode_attn_paged", lambda *a: 0)
    plan = cp.cp_decode_plan(2, [5, 5, 9], n_workers=2)
    x, q = torch.zeros(19, 576, dtype=torch.bfloat16), torch.zeros(3, 1, 576, dtype=torch.bfloat16)
    pool = torch.zeros(8 * 64, 576, dtype=torch.bfloat16)
    o = dict(o_part=torch.zeros(1), lse_part=torch.zeros(1), ws=torch.zeros(1))
    for rows in (6, 8):
        pages = cp.PageTable(np.zeros((rows, 2)), 64, 8, device="cpu")
        cp.cp_kv_shard_pack_paged(plan, pages, x, pool=pool)
        cp.cp_decode_attn_paged(plan, pages, cp.CP_DECODE_MLA, q, pool, sm_scale=1.0, **o)
    for rows in (1, 4, 5):
        pages = cp.PageTable(np.zeros((rows, 2)), 64, 8, device="cpu")
        with pytest.raises(ValueError, match="6 pairs"):
            cp.cp_kv_shard_pack_paged(plan, pages, x, pool=pool)
        with pytest.raises(ValueError, match="6 pairs"):
            cp.cp_decode_attn_paged(plan, pages, cp.CP_DECODE_MLA, q, pool, sm_scale=1.0, **o)


def test_paged_calls_need_the_pool_of_the_table(cp, monkeypatch):
    """A pool, or a pool of scales, with fewer rows than the table's pages is
    refused by the paged pack and decode."""
    import torch
    b = cp._binding
    monkeypatch.setattr(b, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(b, "_stream", lambda d: None)
    monkeypatch.setattr(b, "_ptr", lambda t: None)
    monkeypatch.setattr(b.lib, "cp_kv_shard_pack_paged", lambda *a: 0)
    monkeypatch.setattr(b.lib, "cp_decode_attn_paged", lambda *a: 0)
    plan, pages = cp.cp_decode_plan(2, [5], n_workers=2), cp.PageTable(np.zeros((2, 1)), 64, 3, device="cpu")
    x, q, sx = torch.zeros(5, 576, dtype=torch.uint8), torch.zeros(1, 1, 576, dtype=torch.bfloat16), torch.zeros(5)
    g, qg = torch.zeros(192, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    o = dict(o_part=torch.zeros(1), lse_part=torch.zeros(1), ws=torch.zeros(1))
    pool, scales = torch.zeros(192, 576, dtype=torch.uint8), torch.zeros(192)
    for p, s, why in ((pool, scales, None), (pool[:191], scales, "pool has 191"), (pool, scales[:64], "scale_pool has 64")):
        for fn, args, kw in ((cp.cp_kv_shard_pack_paged, (plan, pages, x, sx, p, s), {}),
                             (cp.cp_decode_attn_paged, (plan, pages, cp.CP_DECODE_MLA, q, p), dict(scale_pool=s, sm_scale=1.0, **o))):
            if why is None:
                fn(*args, **kw)
            else:
                with pytest.raises(ValueError, match=why):
                    fn(*args, **kw)
    cp.cp_decode_attn_paged(plan, pages, cp.CP_DECODE_GQA, qg, g, g, sm_scale=1.0, **o)
    with pytest.raises(ValueError, match="v_pool has 128"):
        cp.cp_decode_attn_paged(plan, pages, cp.CP_DECODE_GQA, qg, g, g[:128], sm_scale=1.0, **o)
