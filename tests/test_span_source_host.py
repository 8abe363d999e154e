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


def test_results_of_the_kernel_before_are_not_read_as_read_only():
    """Kernels that start before the one ahead of them has ended (launch_second) read its results after
    wait_primary().  The read-only path (__ldg, const __restrict__) is for data that no one writes
    while the kernel lives, so it must not serve them."""
    written = {"span_bwd.cu": ("nlse2", "ndsum", "near", "part"), "paged_cache.cu": ("keep", "list")}
    for name, fields in written.items():
        code = _code(os.path.join(CSRC, name))
        assert "launch_second(" in code
        for f in fields:
            assert not re.search(rf"__ldg\([^;]*\b{f}\b", code), (name, f)
            assert not re.search(rf"const (?:float|int32_t)\* __restrict__ {f}\b", code), (name, f)
