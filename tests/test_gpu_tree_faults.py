"""The paged-cache and tree operators where an order between threads, a value in a masked place
or a size could go wrong: each against a plain form."""
import pytest
import torch

from long_context_self_gb300 import binding as mb
from tree_util import accept_ref, gen, make_tree

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_self_gb300 import build
    build.build()
    mb.lib()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert mb.magicdec_device_error() == 0


def i32(x):
    return None if x is None else torch.tensor(x, dtype=I32, device=DEV)


def randn(shape, seed):
    return torch.randn(shape, generator=gen(seed)).to(BF16).to(DEV)


# ---------------------------------------------------------------------- accept
@pytest.mark.parametrize("B", [1, 19, 20, 38, 76, 152, 153])        # clusters of 16, 16, 8 ... 1 CTAs on 152 SMs
@pytest.mark.parametrize("V", [1, 3, 64, 1030])
def test_accept_small_vocabulary(B, V):
    """Rows that leave most CTAs of a cluster nothing to read, so that each is at its first store to the
    others at once; sequences without nodes among them, whose CTAs store nothing."""
    n = 5
    g = gen(201)
    target = torch.randn((B, n, V), generator=g)
    counts = [(b * 3) % (n + 1) for b in range(B)]
    parent = make_tree(B, n, "random", 202)
    tok = target.argmax(-1).gather(1, parent.clamp(min=0).long()).to(I32)
    ref = accept_ref(target, tok, parent, counts)
    args = (target.to(DEV), tok.to(DEV), parent.to(DEV), i32(counts))
    for _ in range(20):
        for a, r in zip(mb.magicdec_tree_accept(*args), ref):
            assert torch.equal(a.cpu(), r)
