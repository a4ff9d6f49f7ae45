"""Prompt weights of prompts whose queries are past the L2: the workers go over
them kv head by kv head, and a key's sum grows from pass to pass."""

import math

import pytest
import torch

from test_gpu_evict import prompt_weights, rows_of_plan
from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv,new,pre,zigzag", [
    (128, 64, 1, [12000, 600], [300, 40], True), (128, 64, 2, [300, 12800], [0, 129], False),
    (64, 32, 2, [12900], [70], True)])  # the heads inside the key blocks, at such a length
def test_long_prompts(cp, D, Hq, Hkv, new, pre, zigzag):
    g, T, KV = gen(D + Hkv), sum(new), sum(new) + sum(pre)
    q, k = randn(g, (T, Hq, D)), randn(g, (KV, Hkv, D))
    plan = cp.cp_shard_plan(cp.CP_ZIGZAG if zigzag else cp.CP_INTERLEAVE, 4, new, pre, device=DEV)
    lse = cp.cp_prefill_attn(plan, q, k, k)[1]
    got = cp.cp_prefill_weights(plan, q, k, lse)
    again = cp.cp_prefill_weights(plan, q, k, lse)
    cp.cp_device_error_check()
    assert torch.equal(got, again)
    want, rel = prompt_weights(rows_of_plan(plan), new, pre, q, k, lse, 1 / math.sqrt(D), 0)
    assert ((got.double() - want).abs() <= rel * want).all()
