"""Orders that the kernels' sources have to keep and no run can show: read from the sources (CPU only)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_self_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def code(path):
    """A source without its comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_comparison_reads_what_its_other_operand_writes(path):
    """`search(..., left, at) != left` compares with `left` as it was or as the search leaves it: C++ does not say
    which operand is evaluated first.  The search's result is kept in a variable, and compared then."""
    text = code(path)
    changed = {name for args in re.findall(r"\[&\]\(([^()]*)\)", text) for name in re.findall(r"\w+ ?&(\w+)", args)}
    for statement in re.split(r"[;{}]", text):
        for name in changed:
            for m in re.finditer(rf"\)\s*[!=<>]=?\s*{name}\b", statement):
                assert not re.search(rf"[(,]\s*{name}\s*[,)]", statement[:m.start() + 1]), statement.strip()
