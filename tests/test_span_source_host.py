"""Rules of the span kernels (csrc/span*) that a run cannot show without a fault, held by reading
their source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_compress_gb300", "csrc")
SPAN = sorted(glob.glob(os.path.join(CSRC, "span*.cu*")))


def _code(path):
    """A source without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("path", SPAN, ids=os.path.basename)
def test_products_are_committed_by_the_lane_that_issued_them(path):
    """A commit covers the products of the executing thread alone.  Products are issued by the lane that
    elect() names, so no commit (of a slot, a result or the drain after a timeout) may come from
    a lane chosen in another way."""
    code = _code(path)
    assert "tc::commit(" not in code
    for args in re.findall(r"(?<![\w:])commit\(((?:[^()]|\([^()]*\))*)\)", code):
        lead = args.rsplit(",", 1)[-1].strip()
        assert lead in ("lead", "elect()", "uint32_t lead"), args
    if "lead = elect()" in code:
        assert re.search(r"commit\(bar\((?:B::)?DRAIN\), elect\(\)\)", code)
