"""What the sources of the 8-bit operators must not hold, read as text: faults that no run on one
GPU need show."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "cached_masked_decoding_gb300" / "csrc"
ALL = sorted(p for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh", ".h"))


def code(path):
    """The text without comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)


@pytest.mark.parametrize("path", ALL, ids=lambda p: p.name)
def test_every_copy_lands_in_one_cta_only(path):
    """The library also runs on several GPUs, where a copy to many CTAs may not be used; no operand
    of the 8-bit product is known to lie on this GPU."""
    assert "multi" + "cast" not in path.read_text()


OPS8 = [p for p in ALL if p.name in ("gemm8.cu", "kv8.cu", "rope.cu", "attn_kv8.cu", "attn_kv8_rows.cuh", "attn_kv8_tiles.cuh",
                                     "q8.cuh", "ptx8.cuh", "ops8.h")]


@pytest.mark.parametrize("path", OPS8, ids=lambda p: p.name)
def test_loads_are_coherent(path):
    """The operators' kernels are resident while the one before writes what they read: the non-coherent
    path is not defined for such data."""
    assert not re.search(r"__ldg|ld\.global(\.\w+)*\.nc|__restrict__", code(path))


KERNELS = [(p, i, body) for p in ALL for i, body in enumerate(code(p).split("__global__")[1:]) if "tmem_alloc(" in body]


@pytest.mark.parametrize("path,i,body", KERNELS, ids=lambda v: v.name if isinstance(v, Path) else str(v)[:3])
def test_dependents_start_once_tensor_memory_is_held(path, i, body):
    """The first thread that triggers the dependents does so for its CTA.  A dependent that took the columns
    for which this CTA still waits would wait for this grid in turn: a barrier lies between the two."""
    if "griddep_launch_dependents()" not in body:
        return
    alloc, trigger = body.index("tmem_alloc("), body.index("griddep_launch_dependents()")
    assert alloc < body.find("__syncthreads()", alloc) < trigger
