"""Refusals of the calls that evict whole requests, answered on the host (no GPU needed)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def cp():
    import __graft_entry__
    __graft_entry__.ensure_built()
    import context_long_attention_gb300 as cp
    return cp


P, ODD, INFO = ctypes.c_void_p(256), ctypes.c_void_p(264), ctypes.c_void_p(512)  # never dereferenced
INVALID, UNSUPPORTED = -1, -2


def refuse(lib, status, words, got):
    assert got == status and words in lib.cp_last_error(), (got, lib.cp_last_error())


def test_move(cp):
    lib = cp.lib

    def move(C=2, B=2, most=9, src=P, count=P, k=P, v=None, rb=256, rows=512):
        return lib.cp_cache_move_ex(C, B, most, src, P, count, k, v, rb, None, None, None, rows, None)

    refuse(lib, INVALID, b"C=0", move(C=0))
    refuse(lib, INVALID, b"C=65", move(C=65))
    refuse(lib, INVALID, b"B=0", move(B=0))
    refuse(lib, INVALID, b"B=8193", move(B=8193))
    refuse(lib, INVALID, b"max_moves", move(C=64, B=8192, most=1 << 20))
    refuse(lib, UNSUPPORTED, b"row_bytes", move(rb=24))
    refuse(lib, INVALID, b"pool_rows", move(rows=0))
    for kw in (dict(src=None), dict(count=None), dict(k=None)):
        refuse(lib, INVALID, b"NULL", move(**kw))
    refuse(lib, INVALID, b"aligned", move(v=ODD))


def test_release(cp):
    lib = cp.lib

    def release(C=2, B=2, ctx=P, n=5, at=P, count=P, info=INFO):
        return lib.cp_page_release_ex(C, B, ctx, P, P, 3, 64, 8, P, n, at, count, None, None, info, None)

    refuse(lib, INVALID, b"C=65", release(C=65))
    refuse(lib, INVALID, b"n_free", release(n=-1))
    refuse(lib, INVALID, b"NULL", release(ctx=None))
    refuse(lib, INVALID, b"info is not", release(info=ODD))
    refuse(lib, INVALID, b"free_pos lies", release(at=ctypes.c_void_p(516)))
