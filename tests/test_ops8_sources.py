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
