"""Kernels that may start before the one before them in their stream ends read
global memory through the L2 or by plain loads, never through the read-only path:
what another kernel has just written (a page table, say) may stand there as it was.
Checked in the sources (no GPU needed)."""

import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "context_long_attention_gb300" / "csrc"
EARLY = sorted(p.name for p in CSRC.glob("*.cu") if "wait_for_earlier_kernels();" in p.read_text())
# __ldg, a pointer that promises it, the load itself, and the row map that uses it
READ_ONLY = re.compile(r"\b__ldg\(|\b__restrict__\b|ld\.global\.nc|\bmap_row\(")


def early_code(text):
    """The parts of a file that run in such kernels: all of it where all of its
    kernels are, else each one's own text up to the next kernel."""
    text = re.sub(r"//[^\n]*", "", text)
    parts = text.split("__global__")
    waits = [p for p in parts[1:] if "wait_for_earlier_kernels();" in p]
    return [text] if len(waits) == len(parts) - 1 else waits


def test_there_are_such_kernels():
    assert {"cache_kernels.cu", "prefix_tc.cu", "decode_weights_tc.cu", "evict_kernels.cu"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_no_read_only_loads(name):
    found = [m.group(0) for part in early_code((CSRC / name).read_text()) for m in READ_ONLY.finditer(part)]
    assert not found, f"{name}: {found}"
