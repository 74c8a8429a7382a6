"""A rule of the block-scaled FP8 kernels that no run on one GPU would show broken."""
import re
from pathlib import Path

import pytest

import block_scaled_fp4_sigmoid_gb300 as fm

SOURCES = sorted((Path(fm.__file__).parent / "csrc").glob("fp8_*.cu*"))


@pytest.mark.parametrize("path", SOURCES, ids=lambda p: p.name)
def test_no_read_only_loads(path):
    """Each kernel is launched while the one that may write its inputs still runs, so that they are
    not read-only for its whole life: loads of the read-only path may return what was there before."""
    code = re.sub(r"//[^\n]*", "", path.read_text())
    assert len(SOURCES) >= 5
    assert not re.search(r"\.nc\b|__ldg|__restrict__", code)
