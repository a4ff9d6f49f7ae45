"""Values that are no numbers over E4M3 caches: a NaN code of a row that is read
and a query element that is infinite reach the results, as they do in the other
forms of the same calls, and nothing else."""

import math

import pytest
import torch

from test_gpu_evict import Pool
from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import Case, gen, randn

pytestmark = pytest.mark.gpu


def repack(cp, c):
    """The case's values again, where its cache has them."""
    if c.pages:
        cp.cp_kv_shard_pack_paged(c.dplan, c.pages, c.v, None, c.pool[1])
    else:
        c.sv = cp.cp_kv_shard_pack(c.dplan, c.v)[0]


@pytest.mark.parametrize("D", [128, 64])  # the tensor cores, the CUDA cores
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("members", [1, 9, 25, 70])  # blocks of up to 64, 128 and 256 rows
@pytest.mark.parametrize("workers", [1, 7])
def test_prefix_value_code_that_is_nan(cp, D, page, members, workers):
    """The dim of that kv head is NaN for every query of the group; all others
    and the LSE keep their bits.  Tokens at both ends of tiles, whole and cut ones."""
    C, lens = 2, [700, 130]
    c = Case(cp, C, lens, [members, members], 8, 2, D, "fp8", page=page, workers=workers)
    o, lse = c.run(out_dtype=torch.float32)
    codes = c.v.view(torch.uint8)
    at = [(0, 0, 0, 0x7F), (255, 1, D - 1, 0xFF), (256, 0, 17, 0x7F), (699, 1, 16, 0x7F), (698, 0, 63, 0xFF), (700 + 129, 1, 33, 0xFF)]
    want = o.clone()
    for t, g, d, code in at:
        codes[t, g, d] = code
        rows = slice(0, members) if t < 700 else slice(members, None)
        want[rows, 4 * g:4 * g + 4, d] = math.nan
    repack(cp, c)
    o2, lse2 = c.run(out_dtype=torch.float32)
    cp.cp_device_error_check()
    assert torch.equal(lse, lse2)
    assert torch.equal(want.isnan(), o2.isnan())
    assert torch.equal(want.nan_to_num(9.0), o2.nan_to_num(9.0))


@pytest.mark.parametrize("kv,D", [("fp8", 128), ("fp8", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("members,workers", [(20, 1), (20, 9), (70, 3)])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_prefix_of_a_query_that_is_infinite(cp, kv, D, members, workers, value):
    """Among 600 keys some have either sign there: scores of +inf, so the
    weights are NaN, and no LSE is a number."""
    c = Case(cp, 1, [600], [members], 8, 2, D, kv, workers=workers)
    o, lse = c.run()
    c.q[3, 5, 7] = value
    o2, lse2 = c.run()
    cp.cp_device_error_check()
    assert o2[3, 5].isnan().all() and not lse2[3, 5].isfinite()
    o2[3, 5], lse2[3, 5] = o[3, 5], lse[3, 5]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_weights_of_a_query_that_is_infinite(cp, latent, value):
    """Its request's weights are NaN (its elements as E4M3 numbers have no
    infinity, so a score's sign is lost); other requests' keep their bits."""
    ctx, C, H, D = [300, 150], 2, 8, 576 if latent else 128
    p = Pool(cp, C, ctx, (D,) if latent else (2, D), dtype=torch.float8_e4m3fn)
    q, lse = randn(gen(3), (2, H, D)), torch.full((2, H), 5.0, device=DEV)
    mode = cp.CP_DECODE_MLA if latent else cp.CP_DECODE_GQA
    run = lambda: cp.cp_decode_weights(p.plan, p.pages, mode, q, p.k, lse, torch.zeros_like(p.w), scale_pool=p.scale, sm_scale=0.05)  # noqa: E731
    want = run()
    q[1, 3, 5] = value
    got = run()
    cp.cp_device_error_check()
    spoilt = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
    for r in range(C):
        spoilt[torch.from_numpy(p.rows(1, r)).to(DEV)] = True
    assert got[spoilt].isnan().all() and torch.equal(got[~spoilt], want[~spoilt])
