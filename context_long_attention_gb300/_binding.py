"""ctypes binding of libcpattn.so (argument marshalling only)."""

from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "_lib", "libcpattn.so")

CP_ZIGZAG, CP_INTERLEAVE = 0, 1
CP_BF16, CP_FP32, CP_FP8_E4M3 = 0, 1, 2
CP_DECODE_GQA, CP_DECODE_MLA = 0, 1
CP_DCP_ROUND_ROBIN, CP_DCP_CONTIGUOUS, CP_DCP_SELECTED = 0, 1, 2
_STATUS = {0: "CP_OK", -1: "CP_ERR_INVALID_ARG", -2: "CP_ERR_UNSUPPORTED", -3: "CP_ERR_CUDA",
           -4: "CP_ERR_DEVICE_TIMEOUT", -5: "CP_ERR_WORKSPACE"}
MAX_SHARDS = 64
HEADER_WORDS = 24
SEG_WORDS, PAIR_WORDS, WORK_WORDS = 12, 8, 4
HEADER_FIELDS = ["magic", "kind", "C", "R", "T", "KV", "n_seg", "n_tiles", "off_rank", "off_req",
                 "off_seg", "off_tiles", "off_rtile", "off_idx", "off_qpos", "off_qreq",
                 "host_words", "dev_words", "n_parts", "tile_rows", "n_split", "layout", "s_q",
                 "off_run"]
SEG_FIELDS = ["rank", "req", "block", "which", "local_start", "count", "first_f", "stride",
              "q_start", "first_pos", "kv_len", "kv_base"]


class CpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


if not os.path.exists(lib_path):
    raise ImportError(f"{lib_path} is missing: build it with __graft_entry__.build()")
if os.path.isdir(os.path.join(_HERE, "csrc")):
    from . import _build
    if _build.is_stale():
        raise ImportError(f"{lib_path} was built from other sources than the ones in "
                          f"{os.path.join(_HERE, 'csrc')}: rebuild it with __graft_entry__.build()")
lib = ctypes.CDLL(lib_path)

_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_i64 = ctypes.c_int64
_szp = ctypes.POINTER(ctypes.c_size_t)
_SIGS = {
    "cp_last_error": (ctypes.c_char_p, []),
    "cp_version": (_i, []),
    "cp_device_error_check": (_i, [_vp]),
    "cp_plan_size": (_i, [_i, _i, _i, _vp, _vp, _szp, _szp]),
    "cp_shard_plan": (_i, [_i, _i, _i, _vp, _vp, _vp, _sz, _vp, _sz, _vp]),
    "cp_prefill_attn": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _i, _i, _i, _f, _vp, _vp, _vp]),
    "cp_decode_plan_size": (_i, [_i, _i, _vp, _i, _szp, _szp]),
    "cp_decode_plan": (_i, [_i, _i, _vp, _i, _vp, _sz, _vp, _sz, _vp]),
    "cp_decode_plan_ex_size": (_i, [_i, _i, _vp, _i, _i, _i, _szp, _szp]),
    "cp_decode_plan_ex": (_i, [_i, _i, _vp, _i, _i, _i, _vp, _sz, _vp, _sz, _vp]),
    "cp_kv_shard_pack": (_i, [_vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp]),
    "cp_decode_workspace_size": (_i, [_vp, _i, _i, _szp]),
    "cp_decode_attn": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp,
                            _vp, _sz, _vp]),
    "cp_decode_merged_workspace_size": (_i, [_vp, _i, _i, _i, _i, _szp]),
    "cp_decode_attn_merged": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _i,
                                   _vp, _vp, _sz, _vp]),
    "cp_lse_merge": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp]),
    "cp_lse_fold": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "cp_decode_attn_noalloc": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp,
                                    _vp, _vp]),
    "cp_noalloc_scratch_bytes": (_sz, []),
    "cp_kv_shard_pack_paged": (_i, [_vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i,
                                    _vp]),
    "cp_decode_attn_paged": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                  _i, _i, _i, _f, _vp, _vp, _vp, _sz, _vp]),
    "cp_sparse_workspace_size": (_i, [_vp, _i, _szp]),
    "cp_sparse_topk": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "cp_sparse_gather": (_i, [_vp, _vp, _i, _vp, _sz, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp]),
    "cp_sparse_plan_size": (_i, [_i, _i, _i, _i, _szp, _szp]),
    "cp_sparse_plan": (_i, [_i, _i, _i, _i, _vp, _sz, _vp, _sz, _vp]),
    "cp_sparse_decode_attn": (_i, [_vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f,
                                   _vp, _vp, _vp, _sz, _vp]),
    "cp_sparse_decode_attn_merged": (_i, [_vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f,
                                          _vp, _i, _vp, _vp, _sz, _vp]),
    "cp_mla_expand": (_i, [_vp, _i64, _vp, _i, _i, _vp, _vp]),
    "cp_mla_absorb": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "cp_mla_project": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "cp_mla_prefill_attn": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _i64, _i, _f, _vp, _vp, _vp]),
    "cp_page_slots": (_i, [_i, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp]),
    "cp_cache_append": (_i, [_vp, _i, _i, _vp, _i64, _vp, _i64, _vp, _i, _i, _vp, _vp, _vp, _i64, _vp]),
    "cp_rope": (_i, [_i, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _i64, _i, _i, _vp, _i64, _vp, _i64, _i, _i, _vp, _i64, _vp]),
    "cp_prefix_plan_size": (_i, [_i, _i, _vp, _vp, _i, _i, _i, _i, _szp, _szp]),
    "cp_prefix_plan": (_i, [_i, _i, _vp, _vp, _i, _i, _i, _i, _vp, _sz, _vp, _sz, _vp]),
    "cp_prefix_workspace_size": (_i, [_vp, _i, _i, _szp]),
    "cp_prefix_attn": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "cp_prefix_attn_paged": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _i,
                                  _vp, _vp, _sz, _vp]),
    "cp_prefill_weights_workspace_size": (_i, [_vp, _i, _i, _i, _i, _szp]),
    "cp_prefill_weights": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp, _vp, _sz, _vp]),
    "cp_decode_weights": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp]),
    "cp_evict_select": (_i, [_i, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp]),
    "cp_cache_move": (_i, [_i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i64, _vp]),
    "cp_cache_move_ex": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i64, _vp]),
    "cp_page_release": (_i, [_i, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp]),
    "cp_page_release_ex": (_i, [_i, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args
NOALLOC_SCRATCH_BYTES = int(lib.cp_noalloc_scratch_bytes())


def _check(status: int):
    if status != 0:
        raise CpError(status, lib.cp_last_error().decode())


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return CP_BF16
    if t.dtype == torch.float32:
        return CP_FP32
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return CP_FP8_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


class _Plan:
    def __init__(self, host: np.ndarray, dev: torch.Tensor | None):
        self.host = host  # int32 words (host part)
        self.dev = dev    # int32 device words, or None for a host-only plan
        self.header = {k: int(v) for k, v in zip(HEADER_FIELDS, host[:len(HEADER_FIELDS)])}

    @property
    def host_ptr(self) -> int:
        """Address of the host part (looked up once for each array)."""
        known = self.__dict__.get("_host_ptr")
        if known is None or known[0] is not self.host:
            known = self.__dict__["_host_ptr"] = (self.host, self.host.ctypes.data)
        return known[1]

    def __getattr__(self, k):
        h = self.__dict__.get("header", {})
        if k in h:
            return h[k]
        raise AttributeError(k)

    def words(self, off, n):
        return self.host[off:off + n]


class PrefillPlan(_Plan):
    """A prefill shard plan (zigzag or interleave)."""

    @property
    def rank_off(self):
        return self.words(self.off_rank, self.C + 1)

    @property
    def requests(self):
        return self.words(self.off_req, 4 * self.R).reshape(self.R, 4)

    @property
    def segments(self):
        return self.words(self.off_seg, SEG_WORDS * self.n_seg).reshape(self.n_seg, SEG_WORDS)

    @property
    def tiles(self):
        return self.words(self.off_tiles, 2 * self.n_tiles).reshape(-1, 2)

    @property
    def rank_tile_off(self):
        return self.words(self.off_rtile, self.C + 1)

    @property
    def tiles_by_rank(self):
        return self.words(self.off_rtile + self.C + 1, 2 * self.n_tiles).reshape(-1, 2)

    def device_maps(self):
        """(idx, qpos, qreq) int32 device tensors of length T."""
        d = self.dev
        return (d[self.off_idx:self.off_idx + self.T], d[self.off_qpos:self.off_qpos + self.T],
                d[self.off_qreq:self.off_qreq + self.T])

    def rank_rows(self, rank: int) -> int:
        return self.T if rank < 0 else int(self.rank_off[rank + 1] - self.rank_off[rank])


class DecodePlan(_Plan):
    """A decode token-shard plan with its split-KV schedule."""

    @property
    def pairs(self):
        P = self.C * self.R
        return self.words(self.off_rank, PAIR_WORDS * P).reshape(P, PAIR_WORDS)

    @property
    def worker_off(self):
        return self.words(self.off_req, self.n_tiles + 1)

    @property
    def work(self):
        return self.words(self.off_seg, WORK_WORDS * self.n_seg).reshape(-1, WORK_WORDS)

    @property
    def requests(self):
        return self.words(self.off_tiles, 2 * self.R).reshape(self.R, 2)

    @property
    def split_pairs(self):
        return self.words(self.off_rtile, self.n_split)

    @property
    def run_out(self):
        """Per work item, for the merged-output decode: -1 the run goes on to
        the worker's next item; -2 the last item of a run holding its whole
        request; k >= 0 the last item of a partial run, written to part slot
        k; -3 an empty pair's item."""
        return self.words(self.off_run + 2, self.n_seg)

    @property
    def merge_list(self):
        """[m, 3]: (request, first part slot, parts) of the requests merged from parts."""
        n = int(self.words(self.off_run + 1, 1)[0])
        return self.words(self.off_run + 2 + self.n_seg, 3 * n).reshape(n, 3)

    @property
    def n_merge_parts(self):
        return int(self.words(self.off_run, 1)[0])

    def shard_rows(self):
        p = self.pairs
        return [int(p[r * self.R:(r + 1) * self.R, 0].sum()) for r in range(self.C)]

    @property
    def query_rows(self):
        """Query rows per request (s_q; 1 unless planned for MTP)."""
        return max(1, self.header.get("s_q", 1))


def cp_plan_size(strategy: int, C: int, new_len, prefix_len):
    nl, pl = _i32(new_len), _i32(prefix_len)
    hb, db = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.cp_plan_size(strategy, C, len(nl), _np_ptr(nl), _np_ptr(pl), ctypes.byref(hb),
                            ctypes.byref(db)))
    return hb.value, db.value


def cp_shard_plan(strategy: int, C: int, new_len, prefix_len=None, device=None) -> PrefillPlan:
    """Builds a prefill shard plan.  With ``device=None`` only the host part
    is computed (no CUDA call); otherwise the plan is copied to ``device`` and
    the per-query maps are filled there by a kernel on the current stream."""
    nl = _i32(new_len)
    pl = _i32(prefix_len if prefix_len is not None else np.zeros_like(nl))
    hb, db = cp_plan_size(strategy, C, nl, pl)
    host = np.zeros(hb // 4, dtype=np.int32)
    dev = None
    if device is not None:
        dev = torch.empty(db // 4, dtype=torch.int32, device=device)
    _check(lib.cp_shard_plan(strategy, C, len(nl), _np_ptr(nl), _np_ptr(pl), _np_ptr(host), hb,
                             _ptr(dev), db, _stream(dev.device) if dev is not None else None))
    return PrefillPlan(host, dev)


def cp_prefill_attn(plan: PrefillPlan, q, k, v, sm_scale=None, rank: int = -1, out=None,
                    lse=None):
    """Causal GQA prefill for the queries of ``rank`` (-1: all ranks,
    rank-major).  q [T, Hq, D]; k, v [KV, Hkv, D]; returns (o, lse)."""
    _need_cuda(q, k, v, out, lse)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    rows = plan.rank_rows(rank)
    if out is None:
        out = torch.empty((rows, Hq, D), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    _check(lib.cp_prefill_attn(_np_ptr(plan.host), _ptr(plan.dev), rank, _dtype_code(q), _ptr(q),
                               _ptr(k), _ptr(v), Hq, Hkv, D, float(sm_scale), _ptr(out), _ptr(lse),
                               _stream(q.device)))
    return out, lse


def cp_decode_plan(C: int, ctx_len, n_workers: int = 0, device=None) -> DecodePlan:
    cl = _i32(ctx_len)
    hb, db = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.cp_decode_plan_size(C, len(cl), _np_ptr(cl), n_workers, ctypes.byref(hb),
                                   ctypes.byref(db)))
    host = np.zeros(hb.value // 4, dtype=np.int32)
    dev = None
    if device is not None:
        dev = torch.empty(db.value // 4, dtype=torch.int32, device=device)
    _check(lib.cp_decode_plan(C, len(cl), _np_ptr(cl), n_workers, _np_ptr(host), hb.value,
                              _ptr(dev), db.value, _stream(dev.device) if dev is not None else None))
    return DecodePlan(host, dev)


def cp_decode_plan_ex(C: int, ctx_len, layout: int = 0, s_q: int = 1, n_workers: int = 0,
                      device=None) -> DecodePlan:
    """cp_decode_plan with a shard layout (CP_DCP_ROUND_ROBIN or
    CP_DCP_CONTIGUOUS) and s_q query rows per request."""
    cl = _i32(ctx_len)
    hb, db = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.cp_decode_plan_ex_size(C, len(cl), _np_ptr(cl), layout, s_q, n_workers,
                                      ctypes.byref(hb), ctypes.byref(db)))
    host = np.zeros(hb.value // 4, dtype=np.int32)
    dev = None
    if device is not None:
        dev = torch.empty(db.value // 4, dtype=torch.int32, device=device)
    _check(lib.cp_decode_plan_ex(C, len(cl), _np_ptr(cl), layout, s_q, n_workers, _np_ptr(host),
                                 hb.value, _ptr(dev), db.value,
                                 _stream(dev.device) if dev is not None else None))
    return DecodePlan(host, dev)


def _decode_shapes(plan, q):
    """(lead, H, Dqk) of a decode query: lead = (B,) or (B, s_q) for MTP plans."""
    s_q = plan.query_rows
    if s_q > 1:
        B, sq, H, Dqk = q.shape
        if sq != s_q:
            raise ValueError(f"q has {sq} query rows, the plan {s_q}")
        return (B, s_q), H, Dqk
    B, H, Dqk = q.shape
    return (B,), H, Dqk


def _ptr_array(ts):
    arr = (ctypes.c_void_p * max(1, len(ts)))()
    for i, t in enumerate(ts):
        arr[i] = None if t is None else t.data_ptr()
    return arr


def cp_kv_shard_pack(plan: DecodePlan, kv, kv_scale=None, shards=None, shard_scales=None):
    """Gathers a token-ordered cache kv [T, ...] into C token shards.
    Returns (shards, shard_scales) — lists of C tensors."""
    _need_cuda(kv, kv_scale)
    if kv.dtype == torch.float8_e4m3fn:
        kv = kv.view(torch.uint8)
    row_elems = int(np.prod(kv.shape[1:]))
    rows = plan.shard_rows()
    if shards is None:
        shards = [torch.empty((n, *kv.shape[1:]), dtype=kv.dtype, device=kv.device) for n in rows]
    if kv_scale is not None and shard_scales is None:
        shard_scales = [torch.empty((n,), dtype=torch.float32, device=kv.device) for n in rows]
    _need_cuda(*shards)
    sarr = _ptr_array(shards)
    scarr = _ptr_array(shard_scales) if kv_scale is not None else None
    _check(lib.cp_kv_shard_pack(_np_ptr(plan.host), _ptr(plan.dev), _dtype_code(kv), _ptr(kv),
                                _ptr(kv_scale), row_elems, sarr, scarr, _stream(kv.device)))
    return shards, (shard_scales if kv_scale is not None else None)


class PageTable:
    """A paged decode cache's page table: int32 [C * R][max_pages] page ids
    (row i of pair (shard r, request b) is row i % page_size of page
    table[r * R + b][i // page_size]), kept as a host array and a device copy.

    The paged pack and decode check the host copy and read the device one, so
    both must hold the same ids.  cp_page_slots changes the device copy and
    drops the host one (``host`` is None); sync_host() reads it back.  So does
    a caller who changes ``dev`` in another way, as by replaying a captured
    cp_page_slots: sync_host() after it."""

    def __init__(self, table, page_size: int, num_pages: int, device=None):
        self.host = np.ascontiguousarray(np.asarray(table, dtype=np.int32))
        assert self.host.ndim == 2
        self.max_pages = int(self.host.shape[1])
        self.page_size = int(page_size)
        self.num_pages = int(num_pages)
        self.dev = torch.from_numpy(self.host).to(device) if device is not None else None

    @classmethod
    def on_device(cls, table, page_size: int, num_pages: int):
        """A table [C * R, max_pages] int32 that lives on the GPU
        (cp_page_slots fills it in place); it has no host copy until
        sync_host()."""
        if table.dtype != torch.int32 or table.dim() != 2 or not table.is_cuda or not table.is_contiguous():
            raise ValueError("the table must be a contiguous int32 CUDA tensor [C * R, max_pages]")
        self = cls.__new__(cls)
        self.host, self.dev = None, table
        self.max_pages, self.page_size, self.num_pages = int(table.shape[1]), int(page_size), int(num_pages)
        return self

    def sync_host(self):
        """Copies the device table to the host copy that the paged pack and
        decode check (waits for the current stream)."""
        self.host = self.dev.cpu().numpy()
        return self

    @property
    def pool_rows(self) -> int:
        return self.num_pages * self.page_size


def _host_table(pages: PageTable, plan, **pools):
    """The host copy's address: what the library checks; it cannot check that
    the table has a row for every pair and the pools one for every page's."""
    if pages.host is None:
        raise ValueError("the page table has no host copy of its present ids: call sync_host() first")
    if pages.host.shape[0] < plan.C * plan.R:
        raise ValueError(f"the page table has {pages.host.shape[0]} rows, the plan C * R = {plan.C * plan.R} pairs")
    for name, t in pools.items():
        if t is not None and t.shape[0] < pages.pool_rows:
            raise ValueError(f"{name} has {t.shape[0]} rows, the page table's pool {pages.pool_rows}")
    return _np_ptr(pages.host)


def cp_kv_shard_pack_paged(plan: DecodePlan, pages: PageTable, kv, kv_scale=None, pool=None,
                           scale_pool=None):
    """Gathers a token-ordered cache kv [T, ...] into a paged pool
    [pool_rows, ...].  Returns (pool, scale_pool)."""
    _need_cuda(kv, kv_scale)
    if kv.dtype == torch.float8_e4m3fn:
        kv = kv.view(torch.uint8)
    row_elems = int(np.prod(kv.shape[1:]))
    if pool is None:
        pool = torch.empty((pages.pool_rows, *kv.shape[1:]), dtype=kv.dtype, device=kv.device)
    if kv_scale is not None and scale_pool is None:
        scale_pool = torch.empty((pages.pool_rows,), dtype=torch.float32, device=kv.device)
    table = _host_table(pages, plan, pool=pool, scale_pool=scale_pool if kv_scale is not None else None)
    _check(lib.cp_kv_shard_pack_paged(_np_ptr(plan.host), _ptr(plan.dev), _dtype_code(kv), _ptr(kv),
                                      _ptr(kv_scale), row_elems, _ptr(pool),
                                      _ptr(scale_pool) if kv_scale is not None else None,
                                      table, _ptr(pages.dev), pages.max_pages,
                                      pages.page_size, pages.num_pages, _stream(kv.device)))
    return pool, (scale_pool if kv_scale is not None else None)


def cp_decode_attn_paged(plan: DecodePlan, pages: PageTable, mode: int, q, k_pool, v_pool=None,
                         scale_pool=None, sm_scale=None, o_part=None, lse_part=None, ws=None):
    """cp_decode_attn over a paged pool (k_pool [pool_rows, 576] for MLA, or
    k_pool / v_pool [pool_rows, Hkv, D] for GQA)."""
    lead, H, Dqk = _decode_shapes(plan, q)
    _need_cuda(q, k_pool)
    table = _host_table(pages, plan, k_pool=k_pool, v_pool=v_pool, scale_pool=scale_pool)
    kp = k_pool.view(torch.uint8) if k_pool.dtype == torch.float8_e4m3fn else k_pool
    kv_dtype = _dtype_code(kp)
    if mode == CP_DECODE_MLA:
        Hkv, Dv = 1, 512
    else:
        Hkv, Dv = kp.shape[1], Dqk
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dqk)
    C = plan.C
    if o_part is None:
        o_part = torch.empty((C, *lead, H, Dv), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((C, *lead, H), dtype=torch.float32, device=q.device)
    need = cp_decode_workspace_size(plan, H, Dv)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.cp_decode_attn_paged(_np_ptr(plan.host), _ptr(plan.dev), mode, kv_dtype, _ptr(q),
                                    _ptr(kp), _ptr(v_pool), _ptr(scale_pool), table,
                                    _ptr(pages.dev), pages.max_pages, pages.page_size,
                                    pages.num_pages, H, Hkv, Dqk, Dv, float(sm_scale), _ptr(o_part),
                                    _ptr(lse_part), _ptr(ws), ws_bytes, _stream(q.device)))
    return o_part, lse_part


def cp_decode_workspace_size(plan: DecodePlan, H: int, Dv: int) -> int:
    b = ctypes.c_size_t()
    _check(lib.cp_decode_workspace_size(_np_ptr(plan.host), H, Dv, ctypes.byref(b)))
    return b.value


def cp_decode_attn(plan: DecodePlan, mode: int, q, shard_k, shard_v=None, shard_scale=None,
                   sm_scale=None, o_part=None, lse_part=None, ws=None):
    """Per-shard partial decode attention.  MLA: q [B, H, 576] bf16,
    shard_k[r] [rows_r, 576] bf16 or fp8 codes (+ shard_scale[r]).
    GQA: q [B, Hq, D], shard_k[r]/shard_v[r] [rows_r, Hkv, D] bf16 or fp32 (q
    of the same type), or E4M3 codes with shard_scale[r] [rows_r] fp32, one
    scale per token for its K and V rows (q bf16).
    Returns (o_part [C, B, H, Dv] fp32, lse_part [C, B, H] fp32).  With an
    MTP plan (s_q > 1) q is [B, s_q, H, Dqk] and the outputs [C, B, s_q, ...]."""
    lead, H, Dqk = _decode_shapes(plan, q)
    _need_cuda(q, *[t for t in shard_k if t is not None])
    sk = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in shard_k]
    kv_dtype = _dtype_code(sk[0]) if sk else CP_BF16
    if mode == CP_DECODE_MLA:
        Hkv, Dv = 1, 512
    else:
        Hkv, Dv = sk[0].shape[1], Dqk
        want_q = torch.float32 if kv_dtype == CP_FP32 else torch.bfloat16
        if q.dtype != want_q:
            raise TypeError(f"GQA decode over this cache takes a {want_q} query, got {q.dtype}")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dqk)
    C = plan.C
    if o_part is None:
        o_part = torch.empty((C, *lead, H, Dv), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((C, *lead, H), dtype=torch.float32, device=q.device)
    need = cp_decode_workspace_size(plan, H, Dv)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.cp_decode_attn(_np_ptr(plan.host), _ptr(plan.dev), mode, kv_dtype, _ptr(q),
                              _ptr_array(sk), _ptr_array(shard_v) if shard_v is not None else None,
                              _ptr_array(shard_scale) if shard_scale is not None else None,
                              H, Hkv, Dqk, Dv, float(sm_scale), _ptr(o_part), _ptr(lse_part),
                              _ptr(ws), ws_bytes, _stream(q.device)))
    return o_part, lse_part


def cp_decode_merged_workspace_size(plan: DecodePlan, mode: int, kv_dtype: int, H: int, Dv: int) -> int:
    b = ctypes.c_size_t()
    _check(lib.cp_decode_merged_workspace_size(_np_ptr(plan.host), mode, kv_dtype, H, Dv, ctypes.byref(b)))
    return b.value


def cp_decode_attn_merged(plan: DecodePlan, mode: int, q, shard_k, shard_v=None, shard_scale=None,
                          sm_scale=None, out_dtype=torch.bfloat16, o=None, lse=None, ws=None):
    """cp_decode_attn and the LSE merge of its partials in one call: returns
    (o [B, H, Dv] out_dtype, lse [B, H] fp32); with an MTP plan (s_q > 1)
    q is [B, s_q, H, Dqk] and the outputs [B, s_q, ...].  MLA over an FP8
    cache accumulates each worker's items of one request together and writes
    partials only for requests cut by a worker boundary."""
    lead, H, Dqk = _decode_shapes(plan, q)
    _need_cuda(q, *[t for t in shard_k if t is not None], o, lse)
    sk = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in shard_k]
    kv_dtype = _dtype_code(sk[0]) if sk else CP_BF16
    if mode == CP_DECODE_MLA:
        Hkv, Dv = 1, 512
    else:
        Hkv, Dv = sk[0].shape[1], Dqk
        want_q = torch.float32 if kv_dtype == CP_FP32 else torch.bfloat16
        if q.dtype != want_q:
            raise TypeError(f"GQA decode over this cache takes a {want_q} query, got {q.dtype}")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dqk)
    if o is None:
        o = torch.empty((*lead, H, Dv), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((*lead, H), dtype=torch.float32, device=q.device)
    need = cp_decode_merged_workspace_size(plan, mode, kv_dtype, H, Dv)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.cp_decode_attn_merged(_np_ptr(plan.host), _ptr(plan.dev), mode, kv_dtype, _ptr(q),
                                     _ptr_array(sk), _ptr_array(shard_v) if shard_v is not None else None,
                                     _ptr_array(shard_scale) if shard_scale is not None else None,
                                     H, Hkv, Dqk, Dv, float(sm_scale), _ptr(o), _dtype_code(o), _ptr(lse),
                                     _ptr(ws), ws_bytes, _stream(q.device)))
    return o, lse


def cp_decode_attn_noalloc(plan: DecodePlan, mode: int, q, shard_k, shard_v=None,
                           shard_scale=None, sm_scale=None, o_part=None, lse_part=None):
    """cp_decode_attn without a workspace argument: the split-KV scratch is a
    fixed library-owned device array (NOALLOC_SCRATCH_BYTES).  Calls must not
    overlap on the GPU."""
    lead, H, Dqk = _decode_shapes(plan, q)
    _need_cuda(q, *[t for t in shard_k if t is not None])
    sk = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in shard_k]
    kv_dtype = _dtype_code(sk[0]) if sk else CP_BF16
    if mode == CP_DECODE_MLA:
        Hkv, Dv = 1, 512
    else:
        Hkv, Dv = sk[0].shape[1], Dqk
        want_q = torch.float32 if kv_dtype == CP_FP32 else torch.bfloat16
        if q.dtype != want_q:
            raise TypeError(f"GQA decode over this cache takes a {want_q} query, got {q.dtype}")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dqk)
    C = plan.C
    if o_part is None:
        o_part = torch.empty((C, *lead, H, Dv), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((C, *lead, H), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):  # the library uses the current device's array
        _check(lib.cp_decode_attn_noalloc(
            _np_ptr(plan.host), _ptr(plan.dev), mode, kv_dtype, _ptr(q), _ptr_array(sk),
            _ptr_array(shard_v) if shard_v is not None else None,
            _ptr_array(shard_scale) if shard_scale is not None else None, H, Hkv, Dqk, Dv,
            float(sm_scale), _ptr(o_part), _ptr(lse_part), _stream(q.device)))
    return o_part, lse_part


def cp_lse_merge(o_part, lse_part, out_dtype=torch.bfloat16, out=None, lse=None):
    """Exact LSE merge over the leading dim: o_part [P, N, H, Dv],
    lse_part [P, N, H] -> (o [N, H, Dv], lse [N, H])."""
    _need_cuda(o_part, lse_part, out, lse)
    P, N, H, Dv = o_part.shape
    if out is None:
        out = torch.empty((N, H, Dv), dtype=out_dtype, device=o_part.device)
    if lse is None:
        lse = torch.empty((N, H), dtype=torch.float32, device=o_part.device)
    _check(lib.cp_lse_merge(P, N, H, Dv, _ptr(o_part), _ptr(lse_part), _ptr(out),
                            _dtype_code(out), _ptr(lse), _stream(o_part.device)))
    return out, lse


def cp_lse_fold(o, lse, o_add, lse_add):
    """(o, lse) <- exact combine of (o, lse) and (o_add, lse_add), in place;
    o, o_add [N, H, Dv] fp32 contiguous, lse, lse_add [N, H] fp32."""
    _need_cuda(o, lse, o_add, lse_add)
    for t in (o, lse, o_add, lse_add):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError("cp_lse_fold takes contiguous fp32 tensors")
    N, H, Dv = o.shape
    _check(lib.cp_lse_fold(N, H, Dv, _ptr(o), _ptr(lse), _ptr(o_add), _ptr(lse_add),
                           _stream(o.device)))
    return o, lse


def cp_device_error_check(device=None):
    _check(lib.cp_device_error_check(_stream(device)))


# ---------------------------------------------------------------- sparse decode

def cp_sparse_workspace_size(plan: DecodePlan, k: int) -> int:
    b = ctypes.c_size_t()
    _check(lib.cp_sparse_workspace_size(_np_ptr(plan.host), k, ctypes.byref(b)))
    return b.value


def cp_sparse_topk(plan: DecodePlan, shard_scores, k: int, sel_ids=None, sel_count=None, ws=None):
    """Exact sharded top-k: shard_scores[r] fp32 [rows_r] (the plan's rows).
    Returns (sel_ids [B, k] int32 ascending, -1 padded; sel_count [B]; ws),
    ws holding the candidates for cp_sparse_gather."""
    dev = next(t.device for t in shard_scores if t is not None)
    _need_cuda(*[t for t in shard_scores if t is not None])
    B = plan.R
    if sel_ids is None:
        sel_ids = torch.empty((B, k), dtype=torch.int32, device=dev)
    if sel_count is None:
        sel_count = torch.empty((B,), dtype=torch.int32, device=dev)
    need = cp_sparse_workspace_size(plan, k)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib.cp_sparse_topk(_np_ptr(plan.host), _ptr(plan.dev), _ptr_array(shard_scores), k,
                              _ptr(sel_ids), _ptr(sel_count), _ptr(ws), ws.numel(), _stream(dev)))
    return sel_ids, sel_count, ws


def sparse_slot_rows(k: int) -> int:
    """Rows per (shard, request) slot of a selection buffer: k rounded up to 128."""
    return (k + 127) // 128 * 128


def cp_sparse_gather(plan: DecodePlan, k: int, ws, shard_kv, shard_scale=None, sel_kv=None,
                     sel_scale=None, pair_count=None):
    """Packs each owner's selected rows (after cp_sparse_topk with the same
    plan, k, ws) into selection buffers [B kp, ...] (kp = sparse_slot_rows(k));
    returns
    (sel_kv list, sel_scale list or None, pair_count [C * B])."""
    sk = [t.view(torch.uint8) if t is not None and t.dtype == torch.float8_e4m3fn else t
          for t in shard_kv]
    ref = next(t for t in sk if t is not None)
    _need_cuda(*[t for t in sk if t is not None])
    C, B = plan.C, plan.R
    kp = sparse_slot_rows(k)
    if sel_kv is None:
        sel_kv = [torch.empty((B * kp, *ref.shape[1:]), dtype=ref.dtype, device=ref.device)
                  for _ in range(C)]
    if shard_scale is not None and sel_scale is None:
        sel_scale = [torch.empty((B * kp,), dtype=torch.float32, device=ref.device) for _ in range(C)]
    if pair_count is None:
        pair_count = torch.empty((C * B,), dtype=torch.int32, device=ref.device)
    row_elems = int(np.prod(ref.shape[1:]))
    _check(lib.cp_sparse_gather(_np_ptr(plan.host), _ptr(plan.dev), k, _ptr(ws), ws.numel(),
                                _dtype_code(ref), _ptr_array(sk),
                                _ptr_array(shard_scale) if shard_scale is not None else None,
                                row_elems, _ptr_array(sel_kv),
                                _ptr_array(sel_scale) if sel_scale is not None else None,
                                _ptr(pair_count), _stream(ref.device)))
    return sel_kv, sel_scale, pair_count


def cp_sparse_plan(C: int, B: int, k: int, n_workers: int = 0, device=None) -> DecodePlan:
    """The decode plan over selection buffers with room for k rows per pair."""
    hb, db = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.cp_sparse_plan_size(C, B, k, n_workers, ctypes.byref(hb), ctypes.byref(db)))
    host = np.zeros(hb.value // 4, dtype=np.int32)
    dev = None
    if device is not None:
        dev = torch.empty(db.value // 4, dtype=torch.int32, device=device)
    _check(lib.cp_sparse_plan(C, B, k, n_workers, _np_ptr(host), hb.value, _ptr(dev), db.value,
                              _stream(dev.device) if dev is not None else None))
    return DecodePlan(host, dev)


def cp_sparse_decode_attn(plan: DecodePlan, pair_count, mode: int, q, sel_k, sel_v=None,
                          sel_scale=None, sm_scale=None, o_part=None, lse_part=None, ws=None):
    """cp_decode_attn over the selection buffers (plan from cp_sparse_plan)."""
    B, H, Dqk = q.shape
    sk = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in sel_k]
    _need_cuda(q, pair_count, *sk)
    kv_dtype = _dtype_code(sk[0])
    if mode == CP_DECODE_MLA:
        Hkv, Dv = 1, 512
    else:
        Hkv, Dv = sk[0].shape[1], Dqk
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dqk)
    C = plan.C
    if o_part is None:
        o_part = torch.empty((C, B, H, Dv), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((C, B, H), dtype=torch.float32, device=q.device)
    need = cp_decode_workspace_size(plan, H, Dv)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.cp_sparse_decode_attn(_np_ptr(plan.host), _ptr(plan.dev), _ptr(pair_count), mode,
                                     kv_dtype, _ptr(q), _ptr_array(sk),
                                     _ptr_array(sel_v) if sel_v is not None else None,
                                     _ptr_array(sel_scale) if sel_scale is not None else None,
                                     H, Hkv, Dqk, Dv, float(sm_scale), _ptr(o_part), _ptr(lse_part),
                                     _ptr(ws), ws_bytes, _stream(q.device)))
    return o_part, lse_part


def cp_sparse_decode_attn_merged(plan: DecodePlan, pair_count, mode: int, q, sel_k, sel_v=None,
                                 sel_scale=None, sm_scale=None, out_dtype=torch.bfloat16, o=None, lse=None,
                                 ws=None):
    """cp_sparse_decode_attn and the LSE merge of its partials in one call:
    returns (o [B, H, Dv] out_dtype, lse [B, H] fp32)."""
    B, H, Dqk = q.shape
    sk = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in sel_k]
    _need_cuda(q, pair_count, *sk, o, lse)
    kv_dtype = _dtype_code(sk[0])
    if mode == CP_DECODE_MLA:
        Hkv, Dv = 1, 512
    else:
        Hkv, Dv = sk[0].shape[1], Dqk
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dqk)
    if o is None:
        o = torch.empty((B, H, Dv), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    need = cp_decode_merged_workspace_size(plan, mode, kv_dtype, H, Dv)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.cp_sparse_decode_attn_merged(_np_ptr(plan.host), _ptr(plan.dev), _ptr(pair_count), mode,
                                            kv_dtype, _ptr(q), _ptr_array(sk),
                                            _ptr_array(sel_v) if sel_v is not None else None,
                                            _ptr_array(sel_scale) if sel_scale is not None else None,
                                            H, Hkv, Dqk, Dv, float(sm_scale), _ptr(o), _dtype_code(o), _ptr(lse),
                                            _ptr(ws), ws_bytes, _stream(q.device)))
    return o, lse


# ---------------------------------------------------------------- latent attention
#
# These calls are as short as a decode step's kernels (a few us), so their
# checks are one comparison chain a tensor, a message is only put together once
# one of them fails, and stream and device come from torch's own short paths
# where it has them.

LATENT_DIM, MLA_NOPE_DIM, MLA_ROPE_DIM, MLA_V_DIM = 512, 128, 64, 128
_bf16, _i32t = torch.bfloat16, torch.int32


def _complain(name, t, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: need {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, other arguments on {f'cuda:{device}' if device >= 0 else 'no GPU'}")
    if t.shape != shape:
        raise ValueError(f"{name}: need shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _need(name, t, dtype, shape, device):
    """A contiguous CUDA tensor of this dtype and shape on `device`, the index
    of a CUDA device (a tensor of another kind has index -1)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device >= 0 and t.is_contiguous():
        return t
    return _complain(name, t, dtype, shape, device)


def _rows(name, t, cols, dtype, device):
    """(pointer, row stride) of a CUDA tensor [n, >= cols] whose rows are
    dense and may lie apart (a view of a wider tensor)."""
    if t.dtype is not dtype or not t.is_cuda or t.get_device() != device:
        _complain(name, t, dtype, t.shape, device)
    if t.dim() != 2 or t.shape[1] < cols or t.stride(1) != 1:
        raise ValueError(f"{name}: need [n, {cols}] with dense rows, got {tuple(t.shape)}, strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else cols


_MAX_COUNT = 2**31 - 1  # of the C interface; ctypes would pass a larger one's low 32 bits

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device, fn, *args):
    """fn with the arguments' device current (outputs are made and kernels
    launched on the current device)."""
    with torch.cuda.device(device):
        return fn(*args)


def cp_mla_expand(latent, w_kv, out=None):
    """Keys and values of latent rows: latent [T, >= 512] bf16 (its first 512
    columns; rows may be a view of the 576-wide cache), w_kv [H, 256, 512]
    -> kv [T, H, 256] (128 key dims, then 128 value dims of each head)."""
    dev = latent.get_device()
    ptr, stride = _rows("latent", latent, LATENT_DIM, _bf16, dev)
    T, H = latent.shape[0], w_kv.shape[0]
    _need("w_kv", w_kv, _bf16, (H, MLA_NOPE_DIM + MLA_V_DIM, LATENT_DIM), dev)
    if dev != _device_index():
        return _on(dev, cp_mla_expand, latent, w_kv, out)
    cols = MLA_NOPE_DIM + MLA_V_DIM
    out = torch.empty((T, H, cols), dtype=_bf16, device=latent.device) if out is None else _need("out", out, _bf16, (T, H, cols), dev)
    st = lib.cp_mla_expand(ptr, stride, w_kv.data_ptr(), T, H, out.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    return out


def _per_head(name, x, w_kv, cols, out_cols, out, fn):
    dev = x.get_device()
    H = w_kv.shape[0]
    lead = x.shape[:-2]
    _need("w_kv", w_kv, _bf16, (H, MLA_NOPE_DIM + MLA_V_DIM, LATENT_DIM), dev)
    _need(name, x, _bf16, (*lead, H, cols), dev)
    if dev != _device_index():
        return _on(dev, _per_head, name, x, w_kv, cols, out_cols, out, fn)
    shape = (*lead, H, out_cols)
    out = torch.empty(shape, dtype=_bf16, device=x.device) if out is None else _need("out", out, _bf16, shape, dev)
    st = fn(x.data_ptr(), w_kv.data_ptr(), lead.numel(), H, out.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    return out


def cp_mla_absorb(q, w_kv, out=None):
    """Queries into the latent space: q [..., H, 192] bf16 (128 dims, 64
    rotated), w_kv [H, 256, 512] -> [..., H, 576], the query of
    cp_decode_attn(mode CP_DECODE_MLA)."""
    return _per_head("q", q, w_kv, MLA_NOPE_DIM + MLA_ROPE_DIM, LATENT_DIM + MLA_ROPE_DIM, out, lib.cp_mla_absorb)


def cp_mla_project(o_lat, w_kv, out=None):
    """Latent outputs of the MLA decode to value dims: o_lat [..., H, 512]
    bf16, w_kv [H, 256, 512] -> [..., H, 128]."""
    return _per_head("o_lat", o_lat, w_kv, LATENT_DIM, MLA_V_DIM, out, lib.cp_mla_project)


def cp_mla_prefill_attn(plan: PrefillPlan, q, kv, k_rope, sm_scale=None, rank: int = -1, out=None, lse=None):
    """Causal latent attention in its expanded form for the queries of
    ``rank`` (-1: all ranks, rank-major).  q [T, H, 192]; kv [KV, H, 256]
    (cp_mla_expand); k_rope [KV, 64], a view of the latent cache's last
    columns or a tensor of its own; returns (o [rows, H, 128], lse [rows, H])."""
    dev = q.get_device()
    T, KV, H = plan.header["T"], plan.header["KV"], q.shape[1]
    _need("q", q, _bf16, (T, H, MLA_NOPE_DIM + MLA_ROPE_DIM), dev)
    _need("kv", kv, _bf16, (KV, H, MLA_NOPE_DIM + MLA_V_DIM), dev)
    rope, stride = _rows("k_rope", k_rope, MLA_ROPE_DIM, _bf16, dev)
    if k_rope.shape != (KV, MLA_ROPE_DIM):  # a whole cache entry's first columns are its latent part
        raise ValueError(f"k_rope: need {(KV, MLA_ROPE_DIM)}, got {tuple(k_rope.shape)}")
    if plan.dev is None or plan.dev.get_device() != dev:
        raise ValueError(f"the plan has no device part on {q.device}")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(MLA_NOPE_DIM + MLA_ROPE_DIM)
    if dev != _device_index():
        return _on(dev, cp_mla_prefill_attn, plan, q, kv, k_rope, sm_scale, rank, out, lse)
    rows = T if rank < 0 else plan.rank_rows(rank)
    out = torch.empty((rows, H, MLA_V_DIM), dtype=_bf16, device=q.device) if out is None else \
        _need("out", out, _bf16, (rows, H, MLA_V_DIM), dev)
    lse = torch.empty((rows, H), dtype=torch.float32, device=q.device) if lse is None else \
        _need("lse", lse, torch.float32, (rows, H), dev)
    st = lib.cp_mla_prefill_attn(plan.host_ptr, plan.dev.data_ptr(), rank, q.data_ptr(), kv.data_ptr(), rope, stride,
                                 H, sm_scale, out.data_ptr(), lse.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    return out, lse


# ---------------------------------------------------------------- pages, slots, new tokens

CP_SLOTS_BAD_LENGTH, CP_SLOTS_TABLE_FULL, CP_SLOTS_NO_PAGES, CP_SLOTS_TOO_MANY = 1, 2, 4, 8


def cp_page_slots(pages: PageTable, C: int, ctx_len, new_len, free_ids, free_pos, max_tokens: int, slots=None,
                  cu_new=None, info=None):
    """Pages and slots of a step's new tokens, from lengths on the GPU.

    ctx_len, new_len [B] int32: cached and new tokens of every request; the
    pages that the new ones need are taken from free_ids at free_pos ([1]
    int32, or an earlier call's info[1:2]) on and written into
    ``pages.dev``.  The table's host copy is dropped, since the paged pack and
    decode check it: they need ``pages.sync_host()`` after this call, and
    after every replay of a graph that holds it.  Returns (slots
    [max_tokens], cu_new [B + 1], info [4] = status, next free_pos, pages
    taken, new tokens), all int32 on the GPU; see cpattn.h for the status."""
    i32, table = _i32t, pages.dev
    if table is None:
        raise ValueError("the page table has no device copy")
    dev = table.get_device()
    B, n_free = ctx_len.shape[0], free_ids.shape[0]
    if max_tokens > _MAX_COUNT or n_free > _MAX_COUNT:
        raise ValueError(f"max_tokens={max_tokens}, n_free={n_free}: at most 2^31 - 1")
    _need("page table", table, i32, (C * B, pages.max_pages), dev)
    _need("ctx_len", ctx_len, i32, (B,), dev)
    _need("new_len", new_len, i32, (B,), dev)
    _need("free_ids", free_ids, i32, (n_free,), dev)
    _need("free_pos", free_pos, i32, (1,), dev)
    if dev != _device_index():
        return _on(dev, cp_page_slots, pages, C, ctx_len, new_len, free_ids, free_pos, max_tokens, slots, cu_new, info)
    where = table.device
    slots = torch.empty(max_tokens, dtype=i32, device=where) if slots is None else _need("slots", slots, i32, (max_tokens,), dev)
    cu_new = torch.empty(B + 1, dtype=i32, device=where) if cu_new is None else _need("cu_new", cu_new, i32, (B + 1,), dev)
    info = torch.empty(4, dtype=i32, device=where) if info is None else _need("info", info, i32, (4,), dev)
    st = lib.cp_page_slots(C, B, ctx_len.data_ptr(), new_len.data_ptr(), table.data_ptr(), pages.max_pages,
                           pages.page_size, pages.num_pages, free_ids.data_ptr(), n_free, free_pos.data_ptr(),
                           slots.data_ptr(), max_tokens, cu_new.data_ptr(), info.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    pages.host = None
    return slots, cu_new, info


def _new_rows(name, t, n, row, dev):
    """(pointer, row stride, row elements) of new tokens' rows [n, *row]; only
    the first dimension may be strided."""
    shape = t.shape
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, not {t.device}")
    if shape[0] != n or shape[1:] != row:
        raise ValueError(f"{name}: need {(n, *row)}, got {tuple(shape)}")
    elems = row.numel()
    if t.is_contiguous():
        return t.data_ptr(), elems, elems
    inner = 1
    for size, st in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if st != inner and size != 1:
            raise ValueError(f"{name}: a row must be dense, got strides {t.stride()}")
        inner *= size
    return t.data_ptr(), t.stride(0), elems


def cp_cache_append(slots, k_new, k_pool, v_new=None, v_pool=None, scale_pool=None, new_scale=None):
    """New tokens' rows into a paged pool at slots [n] int32 (a slot outside
    the pool, such as -1, is skipped; slots must differ).

    k_new [n, ...] and, for a GQA cache, v_new [n, ...] into k_pool / v_pool
    [pool_rows, ...] of the same row shape.  Pools of the rows' own dtype take
    them as they are (E4M3 codes with new_scale [n]); bf16 or fp32 rows into
    an E4M3 pool (uint8 or float8_e4m3fn) are quantised with one scale a
    token, amax / 448 over its K and V (at least 2^-149), written to scale_pool [pool_rows]."""
    dev = k_pool.get_device()
    n, rows = slots.shape[0], k_pool.shape[0]
    if n > _MAX_COUNT:
        raise ValueError(f"{n} slots: at most 2^31 - 1")
    if not k_pool.is_cuda or not k_pool.is_contiguous():
        raise ValueError("k_pool must be a contiguous CUDA tensor")
    _need("slots", slots, _i32t, (n,), dev)
    kp, ks, elems = _new_rows("k_new", k_new, n, k_pool.shape[1:], dev)
    src, pool = _dtype_code(k_new), _dtype_code(k_pool)
    vp = vpool = None
    vs = 0
    if (v_new is None) != (v_pool is None):
        raise ValueError("v_new and v_pool must both be given or both None")
    if v_new is not None:
        if _dtype_code(v_new) != src or _dtype_code(v_pool) != pool:
            raise TypeError("V must have K's dtypes")
        if v_pool.shape != k_pool.shape or v_pool.get_device() != dev or not v_pool.is_contiguous():
            raise ValueError("v_pool must be a contiguous tensor like k_pool")
        vp, vs, _ = _new_rows("v_new", v_new, n, v_pool.shape[1:], dev)
        vpool = v_pool.data_ptr()
    scale = pool_scale = None
    if new_scale is not None:
        scale = _need("new_scale", new_scale, torch.float32, (n,), dev).data_ptr()
    if scale_pool is not None:
        pool_scale = _need("scale_pool", scale_pool, torch.float32, (rows,), dev).data_ptr()
    if dev != _device_index():
        return _on(dev, cp_cache_append, slots, k_new, k_pool, v_new, v_pool, scale_pool, new_scale)
    st = lib.cp_cache_append(slots.data_ptr(), n, src, kp, ks, vp, vs, scale, elems, pool, k_pool.data_ptr(), vpool,
                             pool_scale, rows, _raw_stream(dev))
    if st:
        _check(st)


# ---------------------------------------------------------------- rotary positions

CP_ROPE_HALF, CP_ROPE_INTERLEAVED = 0, 1
_f32 = torch.float32


class RopeFreqs:
    """Frequencies of cp_rope: ``turns`` [rot / 2] int64 on the device, the
    angle that a pair turns by at each position in units of 2^-64 turn (modulo
    one turn; from the frequency in 64-bit floating point, so within 2^-52 of it), and
    ``scale``, the factor on cos and sin.  ``inv_freq`` keeps the radians a position in
    64 bits."""

    def __init__(self, inv_freq, scale: float = 1.0, device=None):
        self.inv_freq = np.asarray(inv_freq, dtype=np.float64)
        if self.inv_freq.ndim != 1 or not np.all(np.isfinite(self.inv_freq)):
            raise ValueError("inv_freq: need a list of finite frequencies")
        self.scale, self.rot = float(scale), 2 * self.inv_freq.size
        turns = [int(round(math.fmod(float(f) / (2 * math.pi), 1.0) * 2.0**64)) % 2**64 for f in self.inv_freq]
        self.turns = torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)).to(device)


def cp_rope_freqs(rot: int, base: float = 10000.0, scaling=None, device=None) -> RopeFreqs:
    """Frequencies base^(-2 i / rot) of rot / 2 pairs, as they are or scaled for
    contexts longer than the trained one.  scaling: None, or a dict with "kind"
      "linear"  factor: every frequency divided by it (position interpolation)
      "ntk"     factor: base x factor^(rot / (rot - 2)), so that the slowest pair
                is interpolated by about the factor and the fastest stays
      "bands"   factor, original, low, high: by a pair's turns over the original
                context, original f / (2 pi): divided up to `low` turns, as they are
                from `high` on, a linear blend between
      "yarn"    factor, original, beta_fast = 32, beta_slow = 1, mscale = 1: the blend is
                linear in the pair's index between those of beta_fast and beta_slow turns,
                and cos and sin carry 0.1 mscale ln(factor) + 1 (Peng et al., "YaRN", 2023);
                for a model that has the factor in its softmax scale instead (an mscale_all_dim
                equal to its mscale) mscale=0, which leaves cos and sin as they are, and
                sm_scale times (0.1 mscale_all_dim ln(factor) + 1)^2
    """
    if rot < 2 or rot % 2 or not base > 1:
        raise ValueError(f"rot={rot}, base={base}: need an even rot >= 2 and a base above 1")
    i = np.arange(rot // 2, dtype=np.float64) * 2 / rot
    f, scale = base ** -i, 1.0
    if scaling is not None:
        c = dict(scaling)
        kind, factor = c.pop("kind"), float(c.pop("factor"))
        if not factor >= 1:
            raise ValueError(f"factor={factor}: need at least 1")
        want = {"linear": (), "ntk": (), "bands": ("original", "low", "high"),
                "yarn": ("original", "beta_fast", "beta_slow", "mscale")}
        if kind not in want:
            raise ValueError(f"unknown scaling {kind!r}")
        if kind == "yarn":
            c = {"beta_fast": 32.0, "beta_slow": 1.0, "mscale": 1.0, **c}
        if set(c) != set(want[kind]):
            raise ValueError(f"scaling {kind!r}: need {want[kind]}, got {tuple(c)}")
        if kind == "linear":
            f = f / factor
        elif kind == "ntk":
            if rot < 4:
                raise ValueError("scaling 'ntk' needs rot >= 4")
            f = (base * factor ** (rot / (rot - 2))) ** -i
        elif kind == "bands":
            if not c["high"] > c["low"]:
                raise ValueError("scaling 'bands': need high > low")
            keep = np.clip((c["original"] * f / (2 * math.pi) - c["low"]) / (c["high"] - c["low"]), 0, 1)
            f = f * keep + f / factor * (1 - keep)
        else:
            at = [rot * math.log(c["original"] / (2 * math.pi * b)) / (2 * math.log(base)) for b in (c["beta_fast"], c["beta_slow"])]
            lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
            part = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
            f = f * (1 - part) + f / factor * part
            scale = 0.1 * c["mscale"] * math.log(factor) + 1
    return RopeFreqs(f, scale, device)


def _tokens(name, t, T, dtype, dev):
    """(pointer, token stride, heads, dim) of [T, heads, dim] with dense heads."""
    if t.dtype is not dtype or t.get_device() != dev or dev < 0:
        _complain(name, t, dtype, t.shape, dev)
    shape = t.shape
    if len(shape) != 3 or shape[0] != T:
        raise ValueError(f"{name}: need [{T}, heads, dim], got {tuple(shape)}")
    _, heads, dim = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * dim, heads, dim
    st, sh, sd = t.stride()
    if (sd != 1 and dim != 1) or (sh != dim and heads != 1):
        raise ValueError(f"{name}: a token's heads must be dense, got strides {t.stride()}")
    return t.data_ptr(), st if T > 1 else heads * dim, heads, dim


def cp_rope(q, k, pos, freqs: RopeFreqs, layout: int = CP_ROPE_HALF, tail: bool = False, inverse: bool = False, q_out=None,
            k_out=None):
    """Rotary positions: q [T, Hq, Dq] and k [T, Hk, Dk] (or None), bf16 or fp32,
    views whose tokens may lie apart; pos [T] int32 (cp_shard_plan's qpos for the
    rows of a rank).  The first freqs.rot dims of every head turn, or with
    ``tail`` the last ones.  Returns (q_out, k_out): new tensors, or the given ones;
    q_out=q turns in place.  ``inverse`` turns back, the gradient's direction."""
    dev, dtype, turns = q.get_device(), q.dtype, freqs.turns
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError(f"q: need bf16 or fp32, got {dtype}")
    T = q.shape[0]
    if T > _MAX_COUNT:
        raise ValueError(f"{T} tokens: at most 2^31 - 1")
    qp, qs, Hq, Dq = _tokens("q", q, T, dtype, dev)
    if pos.dtype is not _i32t or pos.get_device() != dev or pos.shape != (T,) or not pos.is_contiguous():
        _need("pos", pos, _i32t, (T,), dev)
    if turns.get_device() != dev:
        raise ValueError(f"the frequencies are on {turns.device}, q on {q.device}")
    if dev != _device_index():
        return _on(dev, cp_rope, q, k, pos, freqs, layout, tail, inverse, q_out, k_out)
    if q_out is None:
        q_out = torch.empty((T, Hq, Dq), dtype=dtype, device=q.device)
        op, os = q_out.data_ptr(), Hq * Dq
    else:
        op, os, Ho, Do = _tokens("q_out", q_out, T, dtype, dev)
        if (Ho, Do) != (Hq, Dq):
            raise ValueError(f"q_out: need {(T, Hq, Dq)}, got {tuple(q_out.shape)}")
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        st = lib.cp_rope(T, pos.data_ptr(), turns.data_ptr(), freqs.rot, layout, tail, inverse, freqs.scale,
                         CP_BF16 if dtype is _bf16 else CP_FP32, qp, qs, Hq, Dq, op, os, None, 0, 0, 0, None, 0, _raw_stream(dev))
    else:
        kp, ks, Hk, Dk = _tokens("k", k, T, dtype, dev)
        if k_out is None:
            k_out = torch.empty((T, Hk, Dk), dtype=dtype, device=q.device)
            kop, kos = k_out.data_ptr(), Hk * Dk
        else:
            kop, kos, Ho, Do = _tokens("k_out", k_out, T, dtype, dev)
            if (Ho, Do) != (Hk, Dk):
                raise ValueError(f"k_out: need {(T, Hk, Dk)}, got {tuple(k_out.shape)}")
        st = lib.cp_rope(T, pos.data_ptr(), turns.data_ptr(), freqs.rot, layout, tail, inverse, freqs.scale,
                         CP_BF16 if dtype is _bf16 else CP_FP32, qp, qs, Hq, Dq, op, os, kp, ks, Hk, Dk, kop, kos, _raw_stream(dev))
    if st:
        _check(st)
    return q_out, k_out


# ---------------------------------------------------------------- shared prefixes

PREFIX_ITEM_FIELDS = ["group", "kv_head", "row0", "m0", "m_rows", "tile_begin", "tile_end", "part", "alone",
                      "first_shard", "first_y", "first_row", "first_rows"]
PREFIX_BLOCK_FIELDS = ["group", "kv_head", "row0", "m0", "m_rows", "first_part", "n_parts"]


class PrefixPlan(_Plan):
    """Work of cp_prefix_attn over R shared prefixes (cp_prefix_plan)."""

    def __init__(self, host: np.ndarray, dev: torch.Tensor | None):
        super().__init__(host, dev)
        p, R, at = self.pairs, self.R, self.off_idx
        self.heads = int(host[at]), int(host[at + 1])  # (Hq, Hkv) that the plan was made for
        self.n_merge, self.merge_parts = int(host[at + 2]), int(host[at + 3])
        self._shard_rows = [int(p[r * R:(r + 1) * R, 0].sum()) for r in range(self.C)]

    @property
    def pairs(self):
        P = self.C * self.R
        return self.words(self.off_rank, PAIR_WORDS * P).reshape(P, PAIR_WORDS)

    @property
    def worker_off(self):
        return self.words(self.off_req, self.n_tiles + 1)

    @property
    def items(self):
        """[n, 16]: PREFIX_ITEM_FIELDS and padding."""
        return self.words(self.off_seg, 16 * self.n_seg).reshape(-1, 16)

    @property
    def blocks(self):
        """[n, 8]: PREFIX_BLOCK_FIELDS and padding, those that need a merge first."""
        return self.words(self.off_run, 8 * self.n_split).reshape(-1, 8)

    @property
    def tile_off(self):
        return self.words(self.off_tiles, self.R * (self.C + 1)).reshape(self.R, self.C + 1)

    def shard_rows(self):
        return list(self._shard_rows)

    def workspace_bytes(self, D: int, P: int) -> int:
        """cp_prefix_workspace_size without the call."""
        return (self.header["n_parts"] if P else self.merge_parts) * 256 * (D + 1) * 4


def cp_prefix_plan(C: int, prefix_len, members, Hq: int, Hkv: int, layout: int = CP_DCP_ROUND_ROBIN, n_workers: int = 0,
                   device=None) -> PrefixPlan:
    """The plan of cp_prefix_attn: members[g] consecutive query rows read the
    prefix of prefix_len[g] tokens, stored as request g of
    cp_decode_plan_ex(C, prefix_len, layout)."""
    pl, mb = _i32(prefix_len), _i32(members)
    if pl.shape != mb.shape or pl.ndim != 1:
        raise ValueError(f"prefix_len and members must be lists of one length, got {pl.shape} and {mb.shape}")
    hb, db = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.cp_prefix_plan_size(C, len(pl), _np_ptr(pl), _np_ptr(mb), layout, Hq, Hkv, n_workers, ctypes.byref(hb),
                                   ctypes.byref(db)))
    host = np.zeros(hb.value // 4, dtype=np.int32)
    dev = torch.empty(db.value // 4, dtype=torch.int32, device=device) if device is not None else None
    _check(lib.cp_prefix_plan(C, len(pl), _np_ptr(pl), _np_ptr(mb), layout, Hq, Hkv, n_workers, _np_ptr(host), hb.value,
                              _ptr(dev), db.value, _stream(dev.device) if dev is not None else None))
    return PrefixPlan(host, dev)


def cp_prefix_workspace_size(plan: PrefixPlan, D: int, P: int = 0) -> int:
    b = ctypes.c_size_t()
    _check(lib.cp_prefix_workspace_size(plan.host_ptr, D, P, ctypes.byref(b)))
    return b.value


def _prefix_call(plan, q, D, o_part, lse_part, out_dtype, o, lse, ws, dev):
    """Checks what shards and pages share and makes the outputs."""
    N, Hq = plan.header["T"], plan.heads[0]
    if plan.dev is None or plan.dev.get_device() != dev:
        raise ValueError(f"the plan has no device part on {q.device}")
    P = 0
    if (o_part is None) != (lse_part is None):
        raise ValueError("o_part and lse_part must both be given or both None")
    if o_part is not None:
        P = o_part.shape[0]
        if o_part.numel() != P * N * Hq * D or lse_part.shape[0] != P or lse_part.numel() != P * N * Hq:
            raise ValueError(f"need o_part [P, {N}, {Hq}, {D}] and lse_part [P, {N}, {Hq}], got {tuple(o_part.shape)} and "
                             f"{tuple(lse_part.shape)}")
        _need("o_part", o_part, _f32, o_part.shape, dev)
        _need("lse_part", lse_part, _f32, lse_part.shape, dev)
    if out_dtype is not _bf16 and out_dtype is not _f32:
        raise TypeError(f"out_dtype: need bf16 or fp32, got {out_dtype}")
    where = q.device
    o = torch.empty((N, Hq, D), dtype=out_dtype, device=where) if o is None else _need("o", o, out_dtype, (N, Hq, D), dev)
    lse = torch.empty((N, Hq), dtype=_f32, device=where) if lse is None else _need("lse", lse, _f32, (N, Hq), dev)
    if ws is None:
        ws_bytes = plan.workspace_bytes(D, P)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=where) if ws_bytes else None
    else:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous tensor on {where}")
        ws_bytes = ws.numel() * ws.element_size()
    return P, o, lse, ws, ws_bytes


def _prefix_q(plan, q, kv_dtype):
    dev = q.get_device()
    if q.dim() != 3:
        raise ValueError(f"q: need [{plan.header['T']}, Hq, D], got {tuple(q.shape)}")
    D = q.shape[2]
    _need("q", q, _f32 if kv_dtype == CP_FP32 else _bf16, (plan.header["T"], plan.heads[0], D), dev)
    return dev, D


def cp_prefix_attn(plan: PrefixPlan, q, shard_k, shard_v, shard_scale=None, sm_scale=None, o_part=None, lse_part=None,
                   out_dtype=torch.bfloat16, o=None, lse=None, ws=None):
    """Attention of the groups' query rows q [N, Hq, D] over the prefix of their
    group, in C shards shard_k[r], shard_v[r] [rows_r, Hkv, D] (and, for E4M3 codes,
    shard_scale[r] [rows_r]), joined with P partial results of the rows' own
    tokens (o_part [P, N, Hq, D], lse_part [P, N, Hq] fp32, as cp_decode_attn
    returns them).  Returns (o [N, Hq, D] out_dtype, lse [N, Hq] fp32)."""
    C, Hkv = plan.header["C"], plan.heads[1]
    if len(shard_k) != C or len(shard_v) != C or (shard_scale is not None and len(shard_scale) != C):
        raise ValueError(f"need one tensor for each of {C} shards")
    dtype = shard_k[0].dtype
    kv_dtype = _dtype_code(shard_k[0])
    dev, D = _prefix_q(plan, q, kv_dtype)
    rows, tail = plan._shard_rows, (Hkv, D)
    kp, vp = (ctypes.c_void_p * C)(), (ctypes.c_void_p * C)()
    sp = None if shard_scale is None else (ctypes.c_void_p * C)()
    for r in range(C):
        shape = (rows[r], *tail)
        kp[r] = _need(f"shard_k[{r}]", shard_k[r], dtype, shape, dev).data_ptr()
        vp[r] = _need(f"shard_v[{r}]", shard_v[r], dtype, shape, dev).data_ptr()
        if sp is not None:
            sp[r] = _need(f"shard_scale[{r}]", shard_scale[r], _f32, (rows[r],), dev).data_ptr()
    if dev != _device_index():
        return _on(dev, cp_prefix_attn, plan, q, shard_k, shard_v, shard_scale, sm_scale, o_part, lse_part, out_dtype, o, lse, ws)
    P, o, lse, ws, ws_bytes = _prefix_call(plan, q, D, o_part, lse_part, out_dtype, o, lse, ws, dev)
    st = lib.cp_prefix_attn(plan.host_ptr, plan.dev.data_ptr(), kv_dtype, q.data_ptr(), kp, vp, sp, plan.heads[0], Hkv, D,
                            1.0 / math.sqrt(D) if sm_scale is None else sm_scale, P, o_part.data_ptr() if P else None,
                            lse_part.data_ptr() if P else None, o.data_ptr(), CP_BF16 if out_dtype is _bf16 else CP_FP32,
                            lse.data_ptr(), None if ws is None else ws.data_ptr(), ws_bytes, _raw_stream(dev))
    if st:
        _check(st)
    return o, lse


def cp_prefix_attn_paged(plan: PrefixPlan, pages: PageTable, q, k_pool, v_pool, scale_pool=None, sm_scale=None, o_part=None,
                         lse_part=None, out_dtype=torch.bfloat16, o=None, lse=None, ws=None):
    """cp_prefix_attn over prefixes in the pages of one pool (k_pool, v_pool
    [pool_rows, Hkv, D]; ``pages`` has a row for every pair r * R + g)."""
    kv_dtype = _dtype_code(k_pool)
    dev, D = _prefix_q(plan, q, kv_dtype)
    Hkv, rows = plan.heads[1], k_pool.shape[0]
    table = _host_table(pages, plan, k_pool=k_pool, v_pool=v_pool, scale_pool=scale_pool)
    if _dtype_code(v_pool) != kv_dtype:
        raise TypeError("v_pool must have k_pool's dtype")
    _need("k_pool", k_pool, k_pool.dtype, (rows, Hkv, D), dev)
    _need("v_pool", v_pool, v_pool.dtype, (rows, Hkv, D), dev)
    if scale_pool is not None:
        _need("scale_pool", scale_pool, _f32, (rows,), dev)
    if pages.dev is None or pages.dev.get_device() != dev:
        raise ValueError(f"the page table has no device copy on {q.device}")
    if dev != _device_index():
        return _on(dev, cp_prefix_attn_paged, plan, pages, q, k_pool, v_pool, scale_pool, sm_scale, o_part, lse_part, out_dtype,
                   o, lse, ws)
    P, o, lse, ws, ws_bytes = _prefix_call(plan, q, D, o_part, lse_part, out_dtype, o, lse, ws, dev)
    _check(lib.cp_prefix_attn_paged(plan.host_ptr, plan.dev.data_ptr(), kv_dtype, q.data_ptr(), k_pool.data_ptr(),
                                    v_pool.data_ptr(), _ptr(scale_pool), table, _ptr(pages.dev), pages.max_pages,
                                    pages.page_size, pages.num_pages, plan.heads[0], Hkv, D,
                                    1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), P, _ptr(o_part),
                                    _ptr(lse_part), o.data_ptr(), _dtype_code(o), lse.data_ptr(), _ptr(ws), ws_bytes,
                                    _raw_stream(dev)))
    return o, lse


# ---------------------------------------------------------------- accumulated weights, eviction

def cp_prefill_weights(plan: PrefillPlan, q, k, lse, sm_scale=None, window: int = 0, out=None, ws=None):
    """The attention weight of every key of a prompt batch: out [KV] fp32, the sum
    over the queries that read it (``window``: over the last so many new tokens of
    each request) and all heads of exp(score - lse).  q [T, Hq, D], k [KV, Hkv, D]
    as given to cp_prefill_attn, lse [T, Hq] as it returned it for all ranks.  In the order
    of k; eviction wants pool rows: weights[slots.long()] = out, with the slots that
    cp_page_slots gave these tokens (+= for a prefix that has weights already)."""
    dev, dtype = q.get_device(), q.dtype
    T, KV = plan.header["T"], plan.header["KV"]
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError(f"q: need bf16 or fp32, got {dtype}")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"need q [{T}, Hq, D] and k [{KV}, Hkv, D], got {tuple(q.shape)} and {tuple(k.shape)}")
    Hq, D, Hkv = q.shape[1], q.shape[2], k.shape[1]
    _need("q", q, dtype, (T, Hq, D), dev)
    _need("k", k, dtype, (KV, Hkv, D), dev)
    _need("lse", lse, _f32, (T, Hq), dev)
    if plan.dev is None or plan.dev.get_device() != dev:
        raise ValueError(f"the plan has no device part on {q.device}")
    if not 0 <= window <= _MAX_COUNT:
        raise ValueError(f"window={window}: need 0 .. 2^31 - 1")
    if dev != _device_index():
        return _on(dev, cp_prefill_weights, plan, q, k, lse, sm_scale, window, out, ws)
    out = torch.empty(KV, dtype=_f32, device=q.device) if out is None else _need("out", out, _f32, (KV,), dev)
    code, b = _dtype_code(q), ctypes.c_size_t()
    _check(lib.cp_prefill_weights_workspace_size(plan.host_ptr, code, Hq, D, window, ctypes.byref(b)))
    if ws is None and b.value:
        ws = torch.empty(b.value, dtype=torch.uint8, device=q.device)
    elif ws is not None and (ws.get_device() != dev or not ws.is_contiguous()):
        raise ValueError(f"ws must be a contiguous tensor on {q.device}")
    _check(lib.cp_prefill_weights(plan.host_ptr, plan.dev.data_ptr(), code, q.data_ptr(), k.data_ptr(), lse.data_ptr(), Hq,
                                  Hkv, D, 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), window, out.data_ptr(),
                                  _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(dev)))
    return out


def cp_decode_weights(plan: DecodePlan, pages: PageTable, mode: int, q, k_pool, lse, weights, scale_pool=None, sm_scale=None):
    """Adds a decode step's attention weights to ``weights`` [pool_rows] fp32, in
    place: for every cached row of the plan's requests the sum over their query
    rows and heads of exp(score - lse).  The plan, pages, q and k_pool as given to
    cp_decode_attn_paged, lse [B, (s_q,) Hq] the merged one.  Returns weights."""
    lead, H, Dqk = _decode_shapes(plan, q)
    dev, rows = q.get_device(), k_pool.shape[0]
    kv_dtype = _dtype_code(k_pool)
    Hkv = 1 if mode == CP_DECODE_MLA else k_pool.shape[1]
    _need("q", q, _f32 if kv_dtype == CP_FP32 else _bf16, (plan.R, *lead[1:], H, Dqk), dev)
    _need("k_pool", k_pool, k_pool.dtype, (rows, Dqk) if mode == CP_DECODE_MLA else (rows, Hkv, Dqk), dev)
    _need("lse", lse, _f32, (*lead, H), dev)
    _need("weights", weights, _f32, (rows,), dev)
    if scale_pool is not None:
        _need("scale_pool", scale_pool, _f32, (rows,), dev)
    table = _host_table(pages, plan, k_pool=k_pool)
    for what, t in (("plan", plan.dev), ("page table", pages.dev)):
        if t is None or t.get_device() != dev:
            raise ValueError(f"the {what} has no device copy on {q.device}")
    if dev != _device_index():
        return _on(dev, cp_decode_weights, plan, pages, mode, q, k_pool, lse, weights, scale_pool, sm_scale)
    _check(lib.cp_decode_weights(plan.host_ptr, plan.dev.data_ptr(), mode, kv_dtype, q.data_ptr(), k_pool.data_ptr(),
                                 _ptr(scale_pool), table, pages.dev.data_ptr(), pages.max_pages, pages.page_size,
                                 pages.num_pages, H, Hkv, Dqk, 1.0 / math.sqrt(Dqk) if sm_scale is None else float(sm_scale),
                                 lse.data_ptr(), weights.data_ptr(), _raw_stream(dev)))
    return weights


def _evict_table(pages, C, ctx_len, keep_len):
    table = pages.dev
    if table is None:
        raise ValueError("the page table has no device copy")
    dev, B = table.get_device(), ctx_len.shape[0]
    _need("page table", table, _i32t, (C * B, pages.max_pages), dev)
    _need("ctx_len", ctx_len, _i32t, (B,), dev)
    _need("keep_len", keep_len, _i32t, (B,), dev)
    return table, dev, B


def cp_evict_select(pages: PageTable, C: int, ctx_len, keep_len, weights, max_moves: int, pos=None, keep_below: int = 0,
                    keep_from=None, src=None, dst=None, count=None):
    """Which rows every pair (shard, request) keeps when its request goes from
    ctx_len[b] to keep_len[b] cached tokens ([B] int32 on the GPU): rows of
    position in [0, keep_below) or >= keep_from[b], then the heaviest by ``weights``
    [pool_rows].  ``pos`` [pool_rows] is the caller's: appended tokens' positions go to
    their slots; a negative one protects nothing.  Returns the moves that bring the kept rows together, for
    cp_cache_move: (src, dst [C B, max_moves] pool rows, -1 behind the last;
    count [C B], -1 for a pair that does not fit: see cpattn.h)."""
    table, dev, B = _evict_table(pages, C, ctx_len, keep_len)
    rows = pages.pool_rows
    _need("weights", weights, _f32, (rows,), dev)
    if pos is not None:
        _need("pos", pos, _i32t, (rows,), dev)
    if keep_from is not None:
        _need("keep_from", keep_from, _i32t, (B,), dev)
    if not 1 <= max_moves <= _MAX_COUNT or not -_MAX_COUNT <= keep_below <= _MAX_COUNT:
        raise ValueError(f"max_moves={max_moves}: need 1 .. 2^31 - 1; keep_below={keep_below}: need an int32")
    if dev != _device_index():
        return _on(dev, cp_evict_select, pages, C, ctx_len, keep_len, weights, max_moves, pos, keep_below, keep_from, src, dst, count)
    shape, where = (C * B, max_moves), table.device
    src = torch.empty(shape, dtype=_i32t, device=where) if src is None else _need("src", src, _i32t, shape, dev)
    dst = torch.empty(shape, dtype=_i32t, device=where) if dst is None else _need("dst", dst, _i32t, shape, dev)
    count = torch.empty(C * B, dtype=_i32t, device=where) if count is None else _need("count", count, _i32t, (C * B,), dev)
    st = lib.cp_evict_select(C, B, ctx_len.data_ptr(), keep_len.data_ptr(), table.data_ptr(), pages.max_pages, pages.page_size,
                             pages.num_pages, weights.data_ptr(), None if pos is None else pos.data_ptr(), keep_below,
                             None if keep_from is None else keep_from.data_ptr(), max_moves, src.data_ptr(), dst.data_ptr(),
                             count.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    return src, dst, count


def cp_cache_move(src, dst, count, k_pool, v_pool=None, scale_pool=None, weights=None, pos=None, C: int = 0):
    """The moves of cp_evict_select on a pool's rows, in place: k_pool and v_pool
    [pool_rows, ...], and scale_pool, weights (fp32) and pos (int32) [pool_rows]
    where they are given.  With the number of shards ``C`` requests move whole: where a
    pair's choice did not fit (count -1) its request stays as it is on all
    shards; without it such pairs alone are skipped."""
    dev, rows = k_pool.get_device(), k_pool.shape[0]
    pairs, most = src.shape
    _need("src", src, _i32t, (pairs, most), dev)
    _need("dst", dst, _i32t, (pairs, most), dev)
    _need("count", count, _i32t, (pairs,), dev)
    _need("k_pool", k_pool, k_pool.dtype, k_pool.shape, dev)
    if v_pool is not None:
        _need("v_pool", v_pool, k_pool.dtype, k_pool.shape, dev)
    for name, t, dtype in (("scale_pool", scale_pool, _f32), ("weights", weights, _f32), ("pos", pos, _i32t)):
        if t is not None:
            _need(name, t, dtype, (rows,), dev)
    if dev != _device_index():
        return _on(dev, cp_cache_move, src, dst, count, k_pool, v_pool, scale_pool, weights, pos, C)
    if C:
        if C < 0 or pairs % C:
            raise ValueError(f"{pairs} pairs are no multiple of C={C}")
        shape, call = (C, pairs // C), lib.cp_cache_move_ex
    else:
        shape, call = (pairs,), lib.cp_cache_move
    st = call(*shape, most, src.data_ptr(), dst.data_ptr(), count.data_ptr(), k_pool.data_ptr(),
                           None if v_pool is None else v_pool.data_ptr(), k_pool.shape[1:].numel() * k_pool.element_size(),
                           None if scale_pool is None else scale_pool.data_ptr(), None if weights is None else weights.data_ptr(),
                           None if pos is None else pos.data_ptr(), rows, _raw_stream(dev))
    if st:
        _check(st)


def cp_page_release(pages: PageTable, C: int, ctx_len, keep_len, free_ids, free_pos, weights=None, pos=None, info=None,
                    count=None):
    """Hands the pages that shorter requests no longer need back to free_ids, below
    free_pos ([1] int32, or an earlier call's info[1:2]), clears their table entries
    and the weights and positions of the rows behind the new lengths.  With the
    ``count`` of cp_evict_select a request one of whose pairs did not fit (count -1)
    stays as it is.  Returns info [4] = status, next free_pos, pages released, requests
    that stay as they are.  Like cp_page_slots it drops the table's host copy
    (``pages.sync_host()``)."""
    table, dev, B = _evict_table(pages, C, ctx_len, keep_len)
    n_free, rows = free_ids.shape[0], pages.pool_rows
    if n_free > _MAX_COUNT:
        raise ValueError(f"n_free={n_free}: at most 2^31 - 1")
    _need("free_ids", free_ids, _i32t, (n_free,), dev)
    _need("free_pos", free_pos, _i32t, (1,), dev)
    if weights is not None:
        _need("weights", weights, _f32, (rows,), dev)
    if count is not None:
        _need("count", count, _i32t, (C * B,), dev)
    if pos is not None:
        _need("pos", pos, _i32t, (rows,), dev)
    if dev != _device_index():
        return _on(dev, cp_page_release, pages, C, ctx_len, keep_len, free_ids, free_pos, weights, pos, info, count)
    info = torch.empty(4, dtype=_i32t, device=table.device) if info is None else _need("info", info, _i32t, (4,), dev)
    st = lib.cp_page_release_ex(C, B, ctx_len.data_ptr(), keep_len.data_ptr(), table.data_ptr(), pages.max_pages, pages.page_size,
                                pages.num_pages, free_ids.data_ptr(), n_free, free_pos.data_ptr(),
                                None if count is None else count.data_ptr(), None if weights is None else weights.data_ptr(),
                                None if pos is None else pos.data_ptr(), info.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    pages.host = None
    return info


# ---------------------------------------------------------------- NVTX ranges
# With CPATTN_NVTX=1 every public entry point runs inside an NVTX range of
# its own name, so a timeline profiler shows the path's steps (plan, prefill,
# pack, decode, merge, ...) on the host and the launch rows they issue.
if os.environ.get("CPATTN_NVTX") == "1":
    import functools

    def _ranged(fn):
        @functools.wraps(fn)
        def wrapper(*args, **kwargs):
            torch.cuda.nvtx.range_push(fn.__name__)
            try:
                return fn(*args, **kwargs)
            finally:
                torch.cuda.nvtx.range_pop()
        return wrapper

    for _n, _f in list(globals().items()):
        if _n.startswith("cp_") and callable(_f):
            globals()[_n] = _ranged(_f)
