"""The normed append, the attention behind shared prefixes and the calls on a heavy-hitter draft cache where values that
are not finite, sizes or an order of calls could go wrong: each against a plain form."""
import pytest
import torch

from heavy_util import heavy_ref, norm_rope_ref
from long_context_self_gb300 import binding as mb
from tree_util import gen, make_cache, rows_of

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


def cache(B, H_kv, cap, d, seed):
    pos = torch.arange(cap, dtype=I32, device=DEV).expand(B, H_kv, cap).contiguous()
    return (randn((B, H_kv, cap, d), seed), randn((B, H_kv, cap, d), seed + 1),
            torch.rand((B, H_kv, cap), generator=gen(seed + 2)).to(DEV), pos)


# Query rows of a KV head: fewer than the rows of a product and as many, by mma.sync and, with 9 rows and more or
# stretches whose scores do not fit shared memory, on tcgen05; one CTA and clusters.  (H_q, H_kv, d, n, cap)
ROWS = [(8, 2, 128, 1, 300), (8, 2, 64, 2, 12001), (12, 2, 128, 2, 300), (10, 2, 64, 5, 300), (32, 2, 64, 1, 300),
        (8, 1, 128, 1, 60001), (16, 2, 64, 1, 30001), (32, 1, 128, 1, 700), (4, 2, 128, 9, 700)]


@pytest.mark.parametrize("H_q,H_kv,d,n,cap", ROWS)
def test_keys_whose_scores_are_minus_infinity(H_q, H_kv, d, n, cap):
    """A key of an infinity whose scores are minus infinity for every query row has no part in anything: weights grow
    by nothing there, and by what the 64-bit form says elsewhere."""
    B, G = 2, H_q // H_kv
    kc, vc, weight, pos = cache(B, H_kv, cap, d, 5)
    lens = [cap, cap - 13]
    q = randn((B, n, H_q, d), 9)
    q[..., 3] = -q[..., 3].abs() - 0.25
    hit = torch.zeros((B, H_kv, cap), dtype=torch.bool, device=DEV)
    hit[:, :, [0, 7, 100]] = True
    hit[:, 0, 150:170] = True
    if n > 1:
        for b, ln in enumerate(lens):
            hit[b, :, ln - 1] = True                   # of the last token's own
    kc[..., 3] = torch.where(hit, float("inf"), kc[..., 3].float()).to(BF16)
    w0 = weight.clone()
    got = mb.magicdec_heavy_attn(q, kc, vc, weight, i32(lens), pos=pos, next_pos=i32([cap, cap]))
    (ref, tol), (w, wt), _ = heavy_ref(q, kc, vc, w0, pos, lens, [cap, cap])
    within(got, ref, tol, "out")
    for b, ln in enumerate(lens):
        within(weight[b, :, :ln], w[b, :, :ln], wt[b, :, :ln], "weight")
        old = hit[b] & (torch.arange(cap, device=DEV) < ln - n)
        assert torch.equal(weight[b][old], w0[b][old])
        if n > 1:
            assert (weight[b, :, ln - 1] == 0).all()


@pytest.mark.parametrize("H_q,H_kv,d,n,cap", [r for r in ROWS if r[3] > 1] + [(4, 1, 128, 2, 24001), (2, 2, 64, 8, 300),
                                                                            (8, 2, 128, 2, 300), (4, 2, 128, 2, 5000)])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_weights_that_a_token_does_not_see(H_q, H_kv, d, n, cap, value):
    """A query row that is not finite makes the weights of the rows that it sees NaN, and leaves those of the later
    tokens' own rows as they are without it."""
    B, G = 2, H_q // H_kv
    kc, vc, weight, pos = cache(B, H_kv, cap, d, 25)
    lens = [cap, n]
    q = randn((B, n, H_q, d), 29)
    w0, w1 = weight.clone(), weight.clone()
    call = lambda q, w: mb.magicdec_heavy_attn(q, kc, vc, w, i32(lens), pos=pos.clone(), next_pos=i32([cap, cap]))  # noqa: E731
    clean = call(q, w0)
    # the first query head of every KV head, of an early token
    for token in sorted({0, n // 2 - 1 if n > 2 else 0}):
        q1, w = q.clone(), w1.clone()
        q1.view(B, n, H_kv, G, d)[:, token, :, 0] = float(value)
        got = call(q1, w).view(B, n, H_kv, G, d)
        bad = torch.zeros((B, n, H_kv, G), dtype=torch.bool, device=DEV)
        bad[:, token, :, 0] = True
        assert got[bad].isnan().all() and torch.equal(got[~bad], clean.view(B, n, H_kv, G, d)[~bad])
        for b, ln in enumerate(lens):
            sees = ln - n + 1 + token
            assert w[b, :, :sees].isnan().all()
            assert torch.equal(w[b, :, sees:], w0[b, :, sees:])


def test_own_slots_up_to_the_largest_capacity():
    """2^31 - 256 own slots, of two pages over and over: tiles are looked up some steps ahead, and positions behind the
    last one pass 2^31."""
    page, d = 47 * 256, 64
    most = ((1 << 31) - 256) // page
    assert page * most == (1 << 31) - 256
    kp = randn((2, page, 1, d), 71)
    # queries of zeros: every key has the same weight, and sums of powers of two are exact as long as the keys of a
    # thread are fewer than 2^24 (a warp's 2^26, 4 of 16 a thread)
    v = torch.tensor([(-1.0) ** c * 2.0 ** (c % 7 - 3) for c in range(d)], device=DEV).to(BF16)
    vp = v.expand(2, page, 1, d).contiguous()
    table = (torch.arange(most, device=DEV) % 2).to(I32).view(1, most)
    q = torch.zeros((1, 1, 1, d), dtype=BF16, device=DEV)
    got = mb.magicdec_prefix_attn(q, kp, vp, i32([[1]]), i32([3]), table, i32([page * most - 1]))
    assert torch.equal(got.view(d), v)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("size,weight,eps", [(2.0 ** -62, 2.0 ** 70, 2.0 ** -126), (2.0 ** 59, 2.0 ** -100, 1e-6),
                                             (2.0 ** -40, 2.0 ** 90, 2.0 ** -126), (2.0 ** 80, 2.0 ** -60, 1e-6)])
def test_norms_whose_weight_and_root_are_far_from_one(size, weight, eps, inter):
    """x / rms(x) is of the order of one whatever x and its root are; only its product with the weight has to be a number."""
    B, n, H_q, H_kv, d, page = 2, 3, 4, 2, 128, 16
    q, k, v = (randn((B, n, H, d), 51 + H) for H in (H_q, H_kv, H_kv))
    q, k = ((x.float() * size).to(BF16) for x in (q, k))
    qw, kw = ((randn((d,), s).float() * weight).to(BF16) for s in (61, 62))
    kp, vp, table = make_cache([5, 0], n, page, H_kv, d, 63, DEV)
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    got = mb.magicdec_norm_append(k, v, kp, vp, table, i32([5, 0]), inv, q=q, q_weight=qw, k_weight=kw, eps=eps,
                                  interleaved=inter)
    for b, ln in enumerate([5, 0]):
        at = torch.arange(ln, ln + n, device=DEV)[:, None].expand(n, d // 2)
        rows = rows_of(table, b, ln + torch.arange(n), page).to(DEV)
        within(got[b], *norm_rope_ref(q[b], qw, eps, at, inv, inter), "q")
        within(kp.view(-1, H_kv, d)[rows], *norm_rope_ref(k[b], kw, eps, at, inv, inter), "k")
