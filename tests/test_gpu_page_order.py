"""Calls that read a page table straight behind the cp_page_slots that fills it,
in one captured step without a wait between them: every replay takes other
pages, and each result equals that of a call long after the table is there.
Old and new entries are valid pages, so that a stale one would be seen in the
results and nowhere else."""

import numpy as np
import pytest
import torch

from test_gpu_parity import DEV, cp  # noqa: F401
from test_gpu_prefix import gen, randn

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)
PAGE, HQ, HKV = 64, 8, 2


class Step:
    """Requests of `lens` tokens over C shards whose pages a replayed step takes."""

    def __init__(self, cp, C, lens, row, kv):
        g = gen(7)
        self.cp, self.C, self.lens = cp, C, lens
        pages = [-(-len(range(r, L, C)) // PAGE) for r in range(C) for L in lens]
        self.num = 3 * sum(pages)
        self.free = torch.arange(self.num, **I32)
        # as another step left it: pages that are there
        self.table = torch.arange(len(pages) * (max(pages) + 1), **I32).reshape(len(pages), -1) % self.num
        self.pages = cp.PageTable.on_device(self.table, PAGE, self.num)
        # a host copy that names each page once: what the host checks; the ids of a replay are the GPU's
        self.checked = np.arange(self.table.numel(), dtype=np.int32).reshape(self.table.shape) % self.num
        rows = self.num * PAGE
        if kv == "fp8":
            self.k, self.v = (randn(g, (rows, *row), torch.float32, 20.0).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
            self.scale = torch.rand(rows, generator=g, device=DEV) * 0.04 + 0.01
        else:
            self.k, self.v, self.scale = randn(g, (rows, *row)), randn(g, (rows, *row)), None
        self.zero, self.new = torch.zeros(len(lens), **I32), torch.tensor(lens, **I32)
        self.at = torch.zeros(1, **I32)

    def take(self):
        self.cp.cp_page_slots(self.pages, self.C, self.zero, self.new, self.free, self.at, sum(self.lens))
        self.pages.host = self.checked

    def replays(self, call, reset=lambda: None):
        """`call` behind `take`, captured; replays with other pages against the same call on its own."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.take()
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                self.take()
                out = call()
            for turn in range(12):
                self.free.copy_(torch.from_numpy(np.random.default_rng(turn).permutation(self.num).astype(np.int32)))
                reset()
                before = self.table.clone()
                graph.replay()
                got = [x.clone() for x in out]
                side.synchronize()
                assert not torch.equal(before, self.table)
                self.pages.sync_host()
                reset()
                want = call()
                side.synchronize()
                self.cp.cp_device_error_check()
                for x, y in zip(got, want):
                    assert torch.equal(x, y), turn
        side.synchronize()


@pytest.mark.parametrize("kv,members", [("bf16", 3), ("bf16", 70), ("fp8", 3), ("fp8", 70)])
def test_prefix_behind_the_slots(cp, kv, members):
    lens = [700, 129, 64, 300]
    s = Step(cp, 2, lens, (HKV, 128), kv)
    q = randn(gen(8), (members * len(lens), HQ, 128))
    plan = cp.cp_prefix_plan(2, lens, [members] * len(lens), HQ, HKV, device=DEV)
    s.replays(lambda: cp.cp_prefix_attn_paged(plan, s.pages, q, s.k, s.v, s.scale))


@pytest.mark.parametrize("kv,latent", [("bf16", False), ("fp8", False), ("fp8", True)])
def test_weights_behind_the_slots(cp, kv, latent):
    lens, H, D = [700, 129, 64, 300], HQ, 576 if latent else 128
    s = Step(cp, 2, lens, (D,) if latent else (HKV, D), kv)
    q, lse, w = randn(gen(8), (len(lens), H, D)), torch.full((len(lens), H), 6.0, device=DEV), torch.zeros(s.num * PAGE, device=DEV)
    plan = cp.cp_decode_plan(2, lens, device=DEV)
    mode = cp.CP_DECODE_MLA if latent else cp.CP_DECODE_GQA
    s.replays(lambda: (cp.cp_decode_weights(plan, s.pages, mode, q, s.k, lse, w, scale_pool=s.scale, sm_scale=0.05).clone(),), w.zero_)
