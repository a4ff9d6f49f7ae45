"""Queries with a dim far larger than the others, over E4M3 caches.

A query row enters the E4M3 products as hi + lo of the row times a power of two that
brings its largest element to [128, 256), where an E4M3 number's step is at least 2^-9:
an element is off by at most 2^-10 there, 2^-17 of the row's largest (shared
prefixes), or by 2^-14, 2^-21 of it (decode weights, which hold lo times 16).  Elements
down to 2^-9 and 2^-13 of the largest keep all of bf16's 8 bits.  A score is off by that
times the sum of the key's magnitudes and, its products summed in fp32, by 2^-20 of
theirs; everything else as for ordinary queries.
"""

import math

import pytest
import torch

from test_gpu_evict import Pool
from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import Case, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [4, 9, 14])
@pytest.mark.parametrize("members", [9, 70])
def test_prefix(cp, power, members):
    c = Case(cp, 2, [700], [members], 8, 2, 128, "fp8", workers=5)
    c.q[..., 5] *= 2.0**power
    c.k.view(torch.uint8)[..., 5] &= 0x83  # key elements under 2^-6 there
    (c.sk, c.sc) = cp.cp_kv_shard_pack(c.dplan, c.k, c.scale)
    o, lse = c.run(out_dtype=torch.float32)
    cp.cp_device_error_check()
    K, V = (x.float().double() * c.scale.double()[:, None, None] for x in (c.k, c.v))
    for h in range(8):
        q, k, v = c.q[:, h].double(), K[:, h // 4], V[:, h // 4]
        x = q @ k.T / math.sqrt(128)
        off = 2.0**-17 * q.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] + 2.0**-20 * (q.abs() @ k.abs().T)
        off = off.amax(1) / math.sqrt(128)
        p = torch.softmax(x, 1)
        assert ((lse[:, h].double() - torch.logsumexp(x, 1)).abs() <= off + 2.0**-20 * (1 + torch.logsumexp(x, 1).abs())).all()
        # a weight is off by less than e^(2 off) - 1 of itself, and rounded to bf16
        tol = (2.0**-8 + torch.expm1(2 * off) * (1 + 2.0**-8))[:, None] * (p @ v.abs()) + 2.0**-20
        assert ((o[:, h].double() - p @ v).abs() <= tol).all()


@pytest.mark.parametrize("power", [4, 9, 14])
@pytest.mark.parametrize("latent", [False, True])
def test_weights(cp, power, latent):
    ctx, C, H, D = [300, 129], 2, 8, 576 if latent else 128
    p = Pool(cp, C, ctx, (D,) if latent else (2, D), dtype=torch.float8_e4m3fn)
    q, scale = randn(gen(3), (2, H, D), std=0.5), 1 / math.sqrt(192)
    q[..., 5] *= 2.0**power
    p.k.view(torch.uint8)[..., 5] &= 0x83
    lse = torch.randn((2, H), generator=gen(4), device=DEV) + 4
    k = p.k.float().double().reshape(p.k.shape[0], -1, D) * p.scale.double()[:, None, None]
    w = torch.zeros_like(p.w)
    cp.cp_decode_weights(p.plan, p.pages, cp.CP_DECODE_MLA if latent else cp.CP_DECODE_GQA, q, p.k, lse, w, scale_pool=p.scale, sm_scale=scale)
    cp.cp_device_error_check()
    for b in range(2):
        for r in range(C):
            at = torch.from_numpy(p.rows(b, r)).to(DEV)
            want = tol = 0
            for h in range(H):
                kk, qq = k[at, h // (H // k.shape[1])], q[b, h].double()
                off = (2.0**-21 * qq.abs().max() * kk.abs().sum(1) + 2.0**-20 * (kk.abs() @ qq.abs())) * scale
                x = kk @ qq * scale - lse[b, h].double()
                # the score, the LSE in other units and the exponential, which rounds its argument to fp32
                want = want + x.exp()
                tol = tol + x.exp() * torch.expm1(off + 2.0**-22 * (4 + x.abs() + 2 * lse[b, h].abs()))
            assert ((w[at].double() - want).abs() <= tol + 2.0**-18 * want).all()
