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


def kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        head = re.search(r"(\w+_kernel)\(", text[m.end():])
        at = text.index("{", m.end() + head.start())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield head.group(1), text[at + 1:end - 1]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_tensor_memory_is_taken_between_the_wait_and_the_release_of_followers(path):
    """A CTA that took tensor memory while it waits for the kernels in front could be what one of them waits for, and
    tcgen05.alloc has no limit.  Likewise a follower that is let go before this CTA has its own."""
    for name, body in kernels(code(path)):
        if "tmem_alloc(" not in body:
            continue
        body = re.sub(r"\{[^{}]*return;\s*\}", "", body)        # ways out at once
        alloc = [m.start() for m in re.finditer(r"tmem_alloc\(", body)]
        wait = [m.start() for m in re.finditer(r"pdl_wait\(\)", body)]
        go = [m.start() for m in re.finditer(r"pdl_trigger\(\)", body)]
        assert len(alloc) == len(wait) == len(go) == 1 and wait[0] < alloc[0] < go[0], name
