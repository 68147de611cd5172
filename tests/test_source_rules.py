"""What PTX and CUDA ask of a kernel and no run can show: read from the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_int8_gb300", "csrc")


def source(name):
    """A file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu"))))
def test_the_warps_of_a_warpgroup_execute_the_same_setmaxnreg(name):
    """Two statements of one kind in a kernel would be two instructions for warps that may share a warpgroup."""
    text = source(name)
    for kind in ("inc", "dec"):
        assert len(re.findall(r"setmaxnreg\." + kind, text)) <= 1
    if "setmaxnreg" in text:
        # the branch between the two is between whole warpgroups
        assert re.search(r"if \(warp (<|>=) C::kSoftmax\) \{\s*asm volatile\(\"setmaxnreg\.", text)
        assert "static_assert(kSoftmax % 4 == 0" in text


@pytest.mark.parametrize("name,others", [("q8_chunk.cu", 0), ("q8_norm.cu", 2), ("q8_rope.cu", 0), ("q8_plan.cu", 0), ("q8_rows.cuh", 0)])
def test_what_may_be_written_in_place_is_read_by_ordinary_loads(name, others):
    """The non-coherent loads are for memory that nobody writes while the kernel runs: of these files' operands the norm's gains alone."""
    loads = re.findall(r"__ldg\(([^;]*);", source(name))
    assert len(loads) == others and all("p.weight" in x for x in loads)
    assert not re.search(r"\.nc\.|__restrict__", source(name))
