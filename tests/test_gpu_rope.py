"""Rotary positions against the formula in 64 bits.

Tolerances, before any run: an angle is off by at most 2^-32 turn, its
conversion to fp32 by 2^-25 half turn, sine and cosine by 2 units in the last
place, and the two products and their sum round three times: together less than
2^-20 (|a| + |b|) times the factor.  A bf16 result is rounded once more, by at
most 2^-8 of itself.
"""

import math

import numpy as np
import pytest
import torch

from test_gpu_parity import DEV, cp  # noqa: F401

pytestmark = pytest.mark.gpu


def randn(seed, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def rotated(x, pos, inv_freq, scale, rot, half, tail, inverse=False):
    """(result in 64 bits, |a| + |b| of every element's pair; 0 where it is copied)."""
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] * torch.from_numpy(inv_freq).to(x.device)
    cos, sin = (f(angle)[:, None] * scale for f in (torch.cos, torch.sin))
    sin = -sin if inverse else sin
    part = lambda t: t[..., t.shape[-1] - rot:] if tail else t[..., :rot]  # noqa: E731
    first = slice(0, rot // 2) if half else slice(0, rot, 2)
    second = slice(rot // 2, rot) if half else slice(1, rot, 2)
    a, b = part(y)[..., first].clone(), part(y)[..., second].clone()
    part(y)[..., first], part(y)[..., second] = a * cos - b * sin, b * cos + a * sin
    part(size)[..., first] = part(size)[..., second] = a.abs() + b.abs()
    return y, size


def check(got, want, size, scale, what):
    tol = size * scale * 2.0**-20 + (want.abs() * 2.0**-8 if got.dtype == torch.bfloat16 else 0)
    bad = (got.double() - want).abs() > torch.where(size > 0, tol, torch.zeros_like(tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, first {bad.nonzero()[0].tolist()}"


SCALINGS = [None, dict(kind="linear", factor=8.0), dict(kind="ntk", factor=4.0),
            dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0), dict(kind="yarn", factor=40.0, original=4096)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,Hq,Dq,Hk,Dk,rot,tail", [
    (1, 32, 128, 8, 128, 128, False), (3, 1, 16, 1, 16, 16, False), (37, 5, 96, 5, 96, 96, True), (130, 64, 192, 1, 64, 64, True),
    (2500, 2, 24, 1, 40, 16, False), (700, 8, 256, 2, 256, 64, False), (9, 12, 200, 3, 104, 80, True), (4000, 1, 64, 0, 0, 64, False)])
def test_rope(cp, T, Hq, Dq, Hk, Dk, rot, tail, half, dtype):
    q = randn(T, (T, Hq, Dq), dtype)
    k = randn(T + 1, (T, Hk, Dk), dtype) if Hk else None
    pos = torch.randint(-50, 2**31 - 1, (T,), generator=torch.Generator().manual_seed(2), dtype=torch.int64).to(torch.int32).to(DEV)
    f = cp.cp_rope_freqs(rot, 10000.0, SCALINGS[T % 5], device=DEV)
    got = cp.cp_rope(q, k, pos, f, cp.CP_ROPE_HALF if half else cp.CP_ROPE_INTERLEAVED, tail)
    for g, x, what in zip(got, (q, k), "qk"):
        if x is None:
            assert g is None
            continue
        # a frequency is within 2^-64 turn a position: 2^-33 turn at the farthest
        check(g, *rotated(x, pos, f.inv_freq, f.scale, rot, half, tail), f.scale, what)


@pytest.mark.parametrize("half", [True, False])
def test_rope_in_place_and_views(cp, half):
    """The last columns of wider rows, in place: the other columns stay."""
    T, wide = 77, randn(1, (77, 640))
    keep, lat = wide.clone(), wide[:, 512:576].unsqueeze(1)
    q = randn(2, (T, 4, 192))
    want = [rotated(x, torch.arange(T, device=DEV) + 5, cp.cp_rope_freqs(64).inv_freq, 1.0, 64, half, True) for x in (q, lat)]
    pos = torch.arange(5, T + 5, dtype=torch.int32, device=DEV)
    f, layout = cp.cp_rope_freqs(64, device=DEV), cp.CP_ROPE_HALF if half else cp.CP_ROPE_INTERLEAVED
    out = cp.cp_rope(q, lat, pos, f, layout, tail=True, q_out=q, k_out=lat)
    assert out[0] is q and out[1] is lat
    check(q, *want[0], 1.0, "q")
    check(lat, *want[1], 1.0, "k")
    keep[:, 512:576] = wide[:, 512:576]
    assert torch.equal(keep, wide)
    # strided output of a strided input
    big = torch.zeros((T, 5, 64), dtype=torch.bfloat16, device=DEV)
    cp.cp_rope(lat, None, pos, f, layout, q_out=big[:, 2:3])
    assert not big[:, :2].any() and not big[:, 3:].any()
    check(big[:, 2:3], *rotated(lat, pos, f.inv_freq, 1.0, 64, half, False), 1.0, "strided")


@pytest.mark.parametrize("half", [True, False])
def test_rope_inverse_is_the_gradient(cp, half):
    """<rope(x), y> = <x, rope_inverse(y)>: by the formula, and by a difference
    of the (linear) map itself along random directions."""
    T, H, D = 33, 3, 64
    f = cp.cp_rope_freqs(D, scaling=SCALINGS[4], device=DEV)
    layout = cp.CP_ROPE_HALF if half else cp.CP_ROPE_INTERLEAVED
    x, y = randn(1, (T, H, D), torch.float32), randn(2, (T, H, D), torch.float32)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 99991
    grad, _ = cp.cp_rope(y, None, pos, f, layout, inverse=True)
    check(grad, *rotated(y, pos, f.inv_freq, f.scale, D, half, False, inverse=True), f.scale, "gradient")
    fwd = cp.cp_rope(x, None, pos, f, layout)[0].double()
    for seed in range(3):
        d = randn(10 + seed, x.shape, torch.float32)
        diff = cp.cp_rope(x + d, None, pos, f, layout)[0].double() - fwd
        lhs, rhs = float((diff * y.double()).sum()), float((grad.double() * d.double()).sum())
        size = float((y.double().abs() * (x.abs().double() + d.abs().double()).sum(-1, keepdim=True)).sum())
        assert abs(lhs - rhs) <= 2.0**-19 * f.scale * size


def test_rope_of_a_plan_captured_and_on_another_stream(cp):
    new = [70, 33]
    plan = cp.cp_shard_plan(cp.CP_INTERLEAVE, 4, new, [100, 0], device=DEV)
    _, qpos, _ = plan.device_maps()
    q = randn(1, (103, 4, 64))
    f = cp.cp_rope_freqs(64, device=DEV)
    want = rotated(q, qpos, f.inv_freq, 1.0, 64, True, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = torch.empty_like(q)
        cp.cp_rope(q, None, qpos, f, q_out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cp.cp_rope(q, None, qpos, f, q_out=out)
        out.zero_()
        g.replay()
    s.synchronize()
    check(out, *want, 1.0, "replayed")


def test_rope_refusals(cp):
    q, pos = randn(1, (4, 2, 64)), torch.zeros(4, dtype=torch.int32, device=DEV)
    f = cp.cp_rope_freqs(64, device=DEV)
    with pytest.raises(ValueError, match="pos"):
        cp.cp_rope(q, None, pos[:3], f)
    with pytest.raises(TypeError, match="pos"):
        cp.cp_rope(q, None, pos.long(), f)
    with pytest.raises(TypeError, match="bf16 or fp32"):
        cp.cp_rope(q.half(), None, pos, f)
    with pytest.raises(ValueError, match="dense"):
        cp.cp_rope(q.transpose(1, 2), None, pos, cp.cp_rope_freqs(16, device=DEV))
    with pytest.raises(cp.CpError, match="head dim"):
        cp.cp_rope(q[..., :48].contiguous(), None, pos, f)
    with pytest.raises(cp.CpError, match="stride"):
        wide = torch.zeros((4, 130), dtype=torch.bfloat16, device=DEV)
        cp.cp_rope(wide[:, :64].unsqueeze(1), None, pos, f)
    with pytest.raises(ValueError, match="frequencies"):
        cp.cp_rope(q, None, pos, cp.cp_rope_freqs(64))
    assert cp.cp_rope(q[:0], None, pos[:0], f)[0].shape == (0, 2, 64)


def test_rope_past_31_bits_of_elements(cp):
    """Rows behind 2^31 elements."""
    T, H, D = 2**31 // (64 * 128) + 3, 64, 128
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV)
    q[-2:] = randn(1, (2, H, D))
    pos = torch.full((T,), 12345, dtype=torch.int32, device=DEV)
    f = cp.cp_rope_freqs(D, device=DEV)
    out, _ = cp.cp_rope(q, None, pos, f)
    check(out[-2:], *rotated(q[-2:], pos[-2:], f.inv_freq, 1.0, D, True, False), 1.0, "last rows")
    assert not out[:-2].any()
