"""The append that norms its heads, and that takes positions of several axes, against plain 64-bit forms
(tests/heavy_util.py)."""
import pytest
import torch

from heavy_util import norm_rope_ref
from long_context_self_gb300 import binding as mb
from tree_util import ancestors, gen, make_cache, make_tree, rows_of

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


def within(got, ref, tol, what=""):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got.double() - ref).abs() - tol).max().item()
    assert over <= 0, f"{what}: off by {over:.3e} more than the bound"


def freqs(rot, base=500000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV) if rot else None


# (H_q, H_kv, d, rot, interleaved, n, lens, page, tree, counts, axes, weights)
CASES = [
    (4, 1, 64, 64, False, 1, [0], 16, None, None, 0, "qk"),
    (32, 8, 128, 128, False, 1, [5, 31999, 0], 16, None, None, 0, "qk"),
    (32, 8, 128, 128, True, 7, [5, 100, 0], 16, "random", None, 0, "qk"),
    (8, 2, 128, 64, False, 9, [5, 100, 17], 48, "star", [9, 0, 3], 0, "qk"),
    (8, 2, 128, 32, True, 9, [5, 100, 17], 100, "forest", [1, 9, 2], 0, "q"),
    (6, 3, 64, 16, False, 33, [250, 1], 1, "chain", None, 0, "k"),
    (8, 8, 64, 0, False, 5, [60, 3], 16, None, None, 0, "qk"),
    (8, 2, 128, 128, False, 1000, [3, 60], 64, None, [1000, 777], 0, "qk"),
    (5, 5, 128, 128, False, 256, [3], 256, "random", None, 0, "qk"),
    # positions given, of one axis and of several
    (8, 2, 128, 128, False, 6, [5, 100], 16, None, None, 1, "qk"),
    (8, 2, 64, 64, True, 6, [5, 100], 16, None, [6, 2], 2, "qk"),
    (28, 4, 128, 128, False, 300, [5, 100], 16, None, None, 3, "qk"),
    (28, 4, 128, 96, False, 40, [5, 100], 16, None, None, 3, ""),
    (7, 7, 64, 32, True, 3, [1, 2, 3], 16, None, None, 5, "k"),
    # many tokens of few rows
    (15, 5, 128, 128, False, 700, [5, 0, 100, 7], 16, None, [700, 3, 0, 699], 3, "qk"),
    (16, 1, 64, 64, True, 700, [5, 0, 100], 48, None, None, 0, "q"),
    (8, 2, 128, 64, True, 200, [5, 100, 17, 0, 1, 2, 3, 4, 5, 6], 64, "random", None, 0, "qk"),
    (3, 3, 64, 64, False, 1000, [5, 1], 1, None, None, 1, "k"),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("H_q,H_kv,d,rot,inter,n,lens,page,tree,counts,axes,weights", CASES)
def test_append(H_q, H_kv, d, rot, inter, n, lens, page, tree, counts, axes, weights, fused):
    B, eps = len(lens), 1e-5
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 41, DEV)
    k0, v0 = kp.clone(), vp.clone()
    if fused:       # views of one projection's output
        q, k, v = randn((B, n, H_q + 2 * H_kv, d), 42).split([H_q, H_kv, H_kv], dim=2)
    else:
        q, k, v = randn((B, n, H_q, d), 43), randn((B, n, H_kv, d), 44), randn((B, n, H_kv, d), 45)
    qw, kw = (randn((d,), s) if x in weights else None for s, x in ((46, "q"), (47, "k")))
    inv, parent = freqs(rot), None if tree is None else make_tree(B, n, tree, 48)
    pos = axis = None
    if axes:
        pos = torch.randint(-50, 1 << 20, (B, n, axes), generator=gen(49), dtype=I32).to(DEV)
        axis = torch.randint(0, axes, (rot // 2,), generator=gen(50), dtype=I32).to(DEV) if axes > 1 else None
    q_out = torch.full((B, n, H_q, d), 7.0, dtype=BF16, device=DEV)
    given = pos[..., 0].contiguous() if axes == 1 else pos
    got = mb.magicdec_norm_append(k, v, kp, vp, table, i32(lens), inv, q=q, q_weight=qw, k_weight=kw, eps=eps,
                                  n_new=i32(counts), parent=None if parent is None else parent.to(DEV), pos=given,
                                  axis=axis, interleaved=inter, q_out=q_out)
    assert got is q_out
    touched = torch.zeros(kp.shape[0] * page, dtype=torch.bool, device=DEV)
    for b in range(B):
        m = n if counts is None else counts[b]
        if axes:
            at = pos[b, :m, axis.long() if axis is not None else [0] * (rot // 2)]
        else:
            pr = None if parent is None else parent[b].tolist()
            at = torch.tensor([lens[b] + (i if pr is None else len(ancestors(pr, i)) - 1) for i in range(m)],
                              dtype=torch.long, device=DEV)[:, None].expand(m, max(1, rot // 2))
        rows = rows_of(table, b, lens[b] + torch.arange(m), page).to(DEV)
        touched[rows] = True
        assert (q_out[b, m:] == 7.0).all()
        if m:
            within(q_out[b, :m], *norm_rope_ref(q[b, :m], qw, eps, at, inv, inter), "q")
            within(kp.view(-1, H_kv, d)[rows], *norm_rope_ref(k[b, :m], kw, eps, at, inv, inter), "k")
            assert torch.equal(vp.view(-1, H_kv, d)[rows], v[b, :m])
    for x, x0 in ((kp, k0), (vp, v0)):
        assert torch.equal(x.view(-1, H_kv, d)[~touched], x0.view(-1, H_kv, d)[~touched])


def test_without_weights_it_is_the_plain_append():
    """Bit for bit: the same angles, products and rounding."""
    B, n, d, page, lens = 3, 20, 128, 16, [7, 0, 500]
    q, k, v = randn((B, n, 8, d), 61), randn((B, n, 2, d), 62), randn((B, n, 2, d), 63)
    parent = make_tree(B, n, "random", 64).to(DEV)
    for inter in (False, True):
        a, b = make_cache(lens, n, page, 2, d, 65, DEV), make_cache(lens, n, page, 2, d, 65, DEV)
        x = mb.magicdec_paged_append(k, v, *a, i32(lens), freqs(d), q=q, parent=parent, interleaved=inter)
        y = mb.magicdec_norm_append(k, v, *b, i32(lens), freqs(d), q=q, parent=parent, interleaved=inter)
        assert torch.equal(x, y) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_in_place_without_queries_and_axes_out_of_range():
    B, n, H, d, page, lens = 2, 5, 8, 128, 16, [30, 7]
    q, k, v = randn((B, n, H, d), 71), randn((B, n, 2, d), 72), randn((B, n, 2, d), 73)
    qw, kw, inv = randn((d,), 74), randn((d,), 75), freqs(d)
    a, b = make_cache(lens, n, page, 2, d, 76, DEV), make_cache(lens, n, page, 2, d, 76, DEV)
    apart = mb.magicdec_norm_append(k, v, *a, i32(lens), inv, q=q, q_weight=qw, k_weight=kw)
    assert mb.magicdec_norm_append(k, v, *b, i32(lens), inv, k_weight=kw) is None
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    mine = q.clone()
    assert mb.magicdec_norm_append(k, v, *b, i32(lens), inv, q=mine, q_weight=qw, k_weight=kw, q_out=mine) is mine
    assert torch.equal(mine, apart)
    pos = torch.randint(0, 9999, (B, n, 2), generator=gen(77), dtype=I32).to(DEV)
    good = torch.tensor([0, 1] * (d // 4), dtype=I32, device=DEV)
    bad = torch.where(good == 0, torch.tensor([-1, 2, 1 << 30, -(1 << 31)], dtype=I32, device=DEV).repeat(d // 8), good)
    got = [mb.magicdec_norm_append(k, v, *a, i32(lens), inv, q=q, q_weight=qw, k_weight=kw, pos=pos, axis=x)
           for x in (good, bad)]
    assert torch.equal(*got)


def test_large_small_and_zero_heads():
    """Heads whose squares leave fp32, heads far below eps, and heads of zeros."""
    B, n, d, page = 1, 6, 64, 16
    q, k, v = randn((B, n, 4, d), 81), randn((B, n, 2, d), 82), randn((B, n, 2, d), 83)
    for i, f in enumerate((1.0, 1e18, 1e25, 7e37, 1e-12, 0.0)):
        q[:, i] = (q[:, i].float().clamp(-4, 4) * f).to(BF16)
        k[:, i] = (k[:, i].float().clamp(-4, 4) * f).to(BF16)
    qw, kw, eps = randn((d,), 84), randn((d,), 85), 1e-6
    kp, vp, table = make_cache([0], n, page, 2, d, 86, DEV)
    got = mb.magicdec_norm_append(k, v, kp, vp, table, i32([0]), freqs(d), q=q, q_weight=qw, k_weight=kw, eps=eps)
    at = torch.arange(n, device=DEV)[:, None].expand(n, d // 2)
    within(got[0], *norm_rope_ref(q[0], qw, eps, at, freqs(d), False), "q")
    rows = rows_of(table, 0, torch.arange(n), page).to(DEV)
    within(kp.view(-1, 2, d)[rows], *norm_rope_ref(k[0], kw, eps, at, freqs(d), False), "k")


def test_slots_past_the_capacity_and_pages_outside_the_pool():
    B, n, d, page = 1, 4, 64, 4
    q, k, v = randn((B, n, 4, d), 91), randn((B, n, 2, d), 92), randn((B, n, 2, d), 93)
    kw = randn((d,), 94)
    kp, vp, table = make_cache([0], 8, page, 2, d, 95, DEV)
    k0 = kp.clone()
    out = mb.magicdec_norm_append(k, v, kp, vp, table, i32([6]), freqs(d), q=q, q_weight=kw, k_weight=kw)
    assert mb.magicdec_device_error() == 3
    want = mb.magicdec_norm_append(k, v, *make_cache([6], n, page, 2, d, 96, DEV), i32([6]), freqs(d), q=q, q_weight=kw)
    assert torch.equal(out, want)
    wrong = table.clone()
    wrong[0, 0] = kp.shape[0]
    kp.copy_(k0)
    mb.magicdec_norm_append(k, v, kp, vp, wrong, i32([0]), freqs(d), k_weight=kw)
    assert mb.magicdec_device_error() == 5
    assert torch.equal(kp, k0)
