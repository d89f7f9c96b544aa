"""The paged-cache and tree operators where an order between threads, a value in a masked place
or a size could go wrong: each against a plain form."""
import pytest
import torch

from long_context_self_gb300 import binding as mb
from tree_util import accept_ref, attn_ref, gen, make_cache, make_tree, rows_of

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


def within(got, ref, tol):
    assert torch.isfinite(got).all()
    over = ((got.double() - ref).abs() - tol).max().item()
    assert over <= 0, f"off by {over:.3e} more than the bound"


# ------------------------------------------------------------------- attention
@pytest.mark.parametrize("page", [16, 130])      # 130: every other tile has two keys
@pytest.mark.parametrize("H_q,H_kv,d,n", [(1, 1, 128, 1), (3, 1, 64, 1), (31, 1, 128, 1), (33, 1, 64, 1), (5, 1, 128, 13),
                                          (97, 1, 128, 1), (127, 1, 64, 1), (3, 1, 128, 43), (5, 1, 64, 51),
                                          (2, 2, 128, 129), (1, 1, 64, 161)])
def test_attention_rows_that_leave_warps_part_empty(H_q, H_kv, d, n, page):
    """Warps some of whose rows have no node, whose rows' maxima grow at different tiles; a sequence
    that one CTA has whole and one that several join."""
    lens = [9, 4001]
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 211, DEV, poison=True)
    # Every 97th key is 3 times as long, so maxima move late and for some rows only.  Scores reach
    # 3 * |q| |k| / sqrt(d), about 40: fp32 products of that size are off by less than
    # 128 * 2^-24 * 3 * sum |q k| / sqrt(d) < 2^-12, inside the bound's 2^-10.
    for b in range(2):
        at = torch.arange(0, lens[b], 97)
        x = kp.view(-1, H_kv, d)
        x[rows_of(table, b, at, page).to(DEV)] *= 3
    q, parent = randn((2, n, H_q, d), 212), make_tree(2, n, "random", 213)
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=parent.to(DEV))
    within(got, *attn_ref(q, kp, vp, table, lens, parent, None))


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
