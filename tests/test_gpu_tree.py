"""The paged-cache and tree operators against plain 64-bit forms (tests/tree_util.py):
append with rotation, attention of a tree of drafted tokens, greedy acceptance down the
tree, commit of the accepted path, and a step of all four.  Integer results are exact;
floating ones are held, element by element, to bounds counted from their roundings."""
import pytest
import torch

from long_context_self_gb300 import binding as mb
from tree_util import accept_ref, ancestors, attn_ref, gen, make_cache, make_tree, rope_ref, rows_of

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


# ------------------------------------------------------------------- attention
# (H_q, H_kv, d, n, lens, page, tree, counts)
ATTN = [
    # the smallest calls
    (4, 4, 128, 1, [1], 16, "chain", None),
    (4, 1, 64, 1, [0, 1, 5], 16, None, None),
    # one row tile: lengths around the tile of 128 keys, every kind of tree
    (32, 8, 128, 8, [0, 1, 119, 120, 121, 127, 128, 129, 300], 16, "random", None),
    (32, 8, 128, 32, [1000, 777], 64, "star", None),
    (8, 2, 64, 25, [513, 0, 64], 32, "forest", None),
    (40, 8, 128, 5, [400, 33], 16, None, None),
    # long enough that a sequence is cut over many CTAs and joined
    (8, 2, 128, 4, [30000], 16, "random", None),
    (2, 1, 64, 16, [9999, 20000], 256, "random", None),
    # two row tiles, the second one part full; several pairs of row tiles
    (32, 8, 128, 33, [500, 128, 0], 16, "random", None),
    (32, 8, 128, 64, [2000, 90], 16, "random", None),
    (16, 2, 64, 40, [130, 1000], 64, "chain", None),
    (16, 4, 128, 256, [700, 5], 128, "random", None),
    (8, 8, 64, 256, [300], 16, None, None),
    (8, 2, 128, 100, [12000], 64, "random", None),
    # trees of different sizes, some empty
    (32, 8, 128, 13, [200, 0, 3000, 64, 5], 16, "random", [13, 0, 1, 7, 5]),
    (32, 8, 128, 80, [200, 0, 3000, 64, 0], 16, "random", [80, 0, 1, 33, 5]),
    # page sizes: longer than a tile, not a multiple of 8 or of anything, single rows
    (24, 8, 64, 13, [700, 9], 48, "random", None),
    (8, 2, 128, 6, [999, 128, 256], 256, "random", None),
    (8, 2, 128, 6, [999, 70], 200, "random", None),
    (8, 2, 128, 6, [999, 70], 100, "random", None),
    (8, 2, 64, 70, [301, 70], 24, "random", None),
    (8, 2, 128, 6, [500, 3], 12, "random", None),
    (8, 2, 128, 6, [500, 3], 7, "random", None),
    (8, 2, 64, 40, [301, 2], 1, "random", None),
    # group sizes that do not divide a row tile, one KV head, one query head each
    (21, 3, 128, 19, [411, 20], 16, "random", None),
    (20, 4, 64, 60, [411, 20], 16, "random", None),
    (128, 1, 64, 3, [411, 20], 16, "random", None),
    (100, 1, 128, 4, [411, 20], 16, "random", None),
    (7, 7, 128, 2, [411, 20], 16, "chain", None),
]


@pytest.mark.parametrize("H_q,H_kv,d,n,lens,page,tree,counts", ATTN)
def test_attention(H_q, H_kv, d, n, lens, page, tree, counts):
    B = len(lens)
    # every pool row that no node sees or is holds NaN
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 5, DEV, poison=True, counts=counts)
    q = randn((B, n, H_q, d), 6)
    parent = None if tree is None else make_tree(B, n, tree, 7)
    ws = torch.full((mb.magicdec_tree_attn_workspace_size(mb.paged_shape(B, H_q, H_kv, d, page, kp.shape[0],
                                                                         table.shape[1]), n),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, float("nan"))
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=None if parent is None else parent.to(DEV),
                                n_nodes=i32(counts), out=out, ws=ws)
    assert got is out
    ref, tol = attn_ref(q, kp, vp, table, lens, parent, counts)
    within(got, ref, tol)
    for b, m in enumerate(counts or []):
        assert (got[b, m:] == 0).all()
    again = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=None if parent is None else parent.to(DEV),
                                  n_nodes=i32(counts))
    assert torch.equal(got, again)            # the order of the sums does not depend on the run


def test_attention_many_sequences():
    """More sequences than a CTA has threads, most of them short or empty."""
    B, n, H_q, H_kv, d, page = 700, 3, 8, 2, 64, 16
    lens = [(b * 37) % 90 for b in range(B)]
    counts = [b % 4 for b in range(B)]
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 15, DEV, poison=True, counts=counts)
    q, parent = randn((B, n, H_q, d), 16), make_tree(B, n, "random", 17)
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=parent.to(DEV), n_nodes=i32(counts))
    within(got, *attn_ref(q, kp, vp, table, lens, parent, counts))


def test_attention_dense_cache():
    """A dense cache [B, L_cap, H_kv, d] is a pool of B pages; same values as the verification call
    on the same cache for a causal block, within both calls' bounds."""
    B, n, H_q, H_kv, d, L_cap = 4, 4, 32, 8, 128, 1003
    k, v, q = randn((B, L_cap, H_kv, d), 21), randn((B, L_cap, H_kv, d), 22), randn((B, n, H_q, d), 23)
    lens = [999, 0, 517, 128]
    table = torch.arange(B, dtype=I32, device=DEV)[:, None].contiguous()
    got = mb.magicdec_tree_attn(q, k, v, table, i32(lens))
    ref, tol = attn_ref(q, k, v, table, lens, None, None)
    within(got, ref, tol)
    block = mb.magicdec_verify_attn(q, k, v, i32([x + n for x in lens]))
    within(block, got.double(), 2 * tol)


def test_attention_shared_prefix_pages_and_bad_parents():
    """Sequences whose tables share their prefix pages; parents that are not before their node
    count as none."""
    B, n, H_q, H_kv, d, page = 3, 6, 8, 2, 128, 16
    kp, vp, table = make_cache([64] * B, n, page, H_kv, d, 25, DEV)
    table[:, :4] = table[0, :4]
    parent = torch.tensor([[-1, 0, 5, 9, -7, 2147483647], [0, 0, 1, 2, 3, 4], [-1, 1, 2, 3, 4, 5]], dtype=I32)
    q = randn((B, n, H_q, d), 26)
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32([64] * B), parent=parent.to(DEV))
    within(got, *attn_ref(q, kp, vp, table, [64] * B, parent, None))


def test_attention_at_and_past_the_capacity():
    """Nodes whose slots are past the capacity hold nothing; lengths are clamped to it."""
    B, n, H_q, H_kv, d, page = 4, 5, 8, 2, 128, 16
    kp, vp, table = make_cache([60] * B, 0, page, H_kv, d, 27, DEV)          # 64 slots
    q, parent = randn((B, n, H_q, d), 28), make_tree(B, n, "random", 29)
    lens = [60, 62, 64, 63]
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=parent.to(DEV))
    within(got, *attn_ref(q, kp, vp, table, lens, parent, None))
    far = mb.magicdec_tree_attn(q, kp, vp, table, i32([64, 2**31 - 1, 1000, -3]), parent=parent.to(DEV),
                                n_nodes=i32([5, 5, 99, 5]))
    within(far, *attn_ref(q, kp, vp, table, [64, 64, 64, 0], parent, None))


def test_attention_growing_scores():
    """Keys whose scores grow along the cache, and fall: the running maximum moves at many tiles,
    and tiles far below it weigh nothing."""
    B, n, H_q, H_kv, d, page, L = 2, 40, 8, 2, 128, 64, 3000
    kp, vp, table = make_cache([L] * B, n, page, H_kv, d, 31, DEV)
    q = randn((B, n, H_q, d), 32)
    for b, (lo, hi) in enumerate(((0.05, 12.0), (12.0, 0.05))):
        rows = rows_of(table, b, torch.arange(L + n), page).to(DEV)
        scale = torch.linspace(lo, hi, L + n, device=DEV)[:, None, None]
        x = kp.view(-1, H_kv, d)
        x[rows] = (x[rows].float() * scale).to(BF16)
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32([L] * B), parent=make_tree(B, n, "random", 33).to(DEV))
    ref, tol = attn_ref(q, kp, vp, table, [L] * B, make_tree(B, n, "random", 33), None)
    # scores reach 12 * |q| |k| / sqrt(d), some 200: fp32 products of that size are off by
    # 128 * 2^-24 * 12 * sum |q k| / sqrt(d) < 1e-3, which the exponential turns into a relative error
    within(got, ref, tol * (1 + 1e-3 / 2.0 ** -8))


def test_attention_page_outside_the_pool():
    """A table entry outside the pool reads as zeros and is reported; other sequences are not touched."""
    B, n, H_q, H_kv, d = 2, 3, 8, 2, 128
    for page, bad in ((16, 3), (256, 0)):
        lens = [300, 300]
        kp, vp, table = make_cache(lens, n, page, H_kv, d, 35, DEV, spare=0)
        q = randn((B, n, H_q, d), 36)
        wrong = table.clone()
        wrong[0, bad] = kp.shape[0]
        got = mb.magicdec_tree_attn(q, kp, vp, wrong, i32(lens))
        assert mb.magicdec_device_error() == 5
        zk, zv = (torch.cat((x, torch.zeros_like(x[:1]))) for x in (kp, vp))
        within(got, *attn_ref(q, zk, zv, wrong, lens, None, None))
        wrong[0, bad] = -1
        assert torch.equal(mb.magicdec_tree_attn(q, kp, vp, wrong, i32(lens)), got)
        assert mb.magicdec_device_error() == 5


# ---------------------------------------------------------------------- append
# (H_q, H_kv, d, rot, interleaved, n, lens, page, tree, counts)
APPEND = [
    (4, 1, 64, 64, False, 1, [0], 16, None, None),
    (32, 8, 128, 128, False, 1, [5, 31999, 0], 16, None, None),
    (32, 8, 128, 128, True, 7, [5, 100, 0], 16, "random", None),
    (8, 2, 128, 64, False, 9, [5, 100, 17], 48, "star", [9, 0, 3]),
    (8, 2, 128, 32, True, 9, [5, 100, 17], 100, "forest", [1, 9, 2]),
    (6, 3, 64, 16, False, 33, [250, 1], 1, "chain", None),
    (8, 8, 64, 0, False, 5, [60, 3], 16, None, None),
    (8, 2, 128, 128, False, 1000, [3, 60], 64, None, [1000, 777]),
    (5, 5, 128, 128, False, 256, [3], 256, "random", None),
    (8, 1, 128, 128, False, 130, [0, 1, 2], 7, "random", [130, 129, 1]),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("H_q,H_kv,d,rot,inter,n,lens,page,tree,counts", APPEND)
def test_append(H_q, H_kv, d, rot, inter, n, lens, page, tree, counts, fused):
    B = len(lens)
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 41, DEV)
    k0, v0 = kp.clone(), vp.clone()
    if fused:       # views of one projection's output
        qkv = randn((B, n, H_q + 2 * H_kv, d), 42)
        q, k, v = qkv.split([H_q, H_kv, H_kv], dim=2)
    else:
        q, k, v = randn((B, n, H_q, d), 43), randn((B, n, H_kv, d), 44), randn((B, n, H_kv, d), 45)
    inv = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV) if rot else None
    parent = None if tree is None else make_tree(B, n, tree, 46)
    q_out = torch.full((B, n, H_q, d), 7.0, dtype=BF16, device=DEV)
    got = mb.magicdec_paged_append(k, v, kp, vp, table, i32(lens), inv, q=q, n_new=i32(counts),
                                   parent=None if parent is None else parent.to(DEV), interleaved=inter, q_out=q_out)
    assert got is q_out
    touched = torch.zeros(kp.shape[0] * page, dtype=torch.bool, device=DEV)
    for b in range(B):
        m = n if counts is None else counts[b]
        pr = None if parent is None else parent[b].tolist()
        pos = torch.tensor([lens[b] + (i if pr is None else len(ancestors(pr, i)) - 1) for i in range(m)],
                           dtype=torch.long, device=DEV)
        rows = rows_of(table, b, lens[b] + torch.arange(m), page).to(DEV)
        touched[rows] = True
        within(q_out[b, :m], *rope_ref(q[b, :m], pos, inv, inter), "q") if m else None
        assert (q_out[b, m:] == 7.0).all()
        if m:
            within(kp.view(-1, H_kv, d)[rows], *rope_ref(k[b, :m], pos, inv, inter), "k")
            assert torch.equal(vp.view(-1, H_kv, d)[rows], v[b, :m])
    for x, x0 in ((kp, k0), (vp, v0)):
        assert torch.equal(x.view(-1, H_kv, d)[~touched], x0.view(-1, H_kv, d)[~touched])


def test_append_in_place_and_without_queries():
    B, n, H, d, page = 2, 5, 8, 128, 16
    lens = [30, 7]
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    q, k, v = randn((B, n, H, d), 51), randn((B, n, 2, d), 52), randn((B, n, 2, d), 53)
    a, b = make_cache(lens, n, page, 2, d, 54, DEV), make_cache(lens, n, page, 2, d, 54, DEV)
    apart = mb.magicdec_paged_append(k, v, *a, i32(lens), inv, q=q)
    assert mb.magicdec_paged_append(k, v, *b, i32(lens), inv) is None
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for inter in (False, True):
        apart = mb.magicdec_paged_append(k, v, *a, i32(lens), inv, q=q, interleaved=inter)
        mine = q.clone()
        assert mb.magicdec_paged_append(k, v, *b, i32(lens), inv, q=mine, interleaved=inter, q_out=mine) is mine
        assert torch.equal(mine, apart)


def test_append_far_positions():
    """Angles of a million radians keep the accuracy of the sine."""
    n, d = 4, 128
    lens = [1 << 20, (1 << 30) + 12345]
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    for b, ln in enumerate(lens):
        q, k = randn((1, n, 2, d), 55 + b), randn((1, n, 1, d), 57 + b)
        kp = torch.zeros((1, 64, 1, d), dtype=BF16, device=DEV)
        table = torch.zeros((1, -(-(ln + n) // 64)), dtype=I32, device=DEV)
        got = mb.magicdec_paged_append(k, k, kp, torch.zeros_like(kp), table, i32([ln]), inv, q=q)
        pos = ln + torch.arange(n, device=DEV)
        within(got[0], *rope_ref(q[0], pos, inv, False))


def test_append_past_the_capacity_and_outside_the_pool():
    B, n, H, d, page = 2, 6, 2, 64, 16
    k, v, q = randn((B, n, H, d), 61), randn((B, n, H, d), 62), randn((B, n, 4, d), 63)
    kp, vp, table = make_cache([30] * B, 2, page, H, d, 64, DEV)              # 32 slots
    k0 = kp.clone()
    out = mb.magicdec_paged_append(k, v, kp, vp, table, i32([28, 3]), None, q=q)
    assert mb.magicdec_device_error() == 3
    assert torch.equal(out, q)                                               # nothing to rotate: copied
    rows = torch.cat((rows_of(table, 0, 28 + torch.arange(4), page), rows_of(table, 1, 3 + torch.arange(n), page)))
    assert torch.equal(kp.view(-1, H, d)[rows.to(DEV)], torch.cat((k[0, :4], k[1])))
    rest = torch.ones(kp.shape[0] * page, dtype=torch.bool)
    rest[rows] = False
    assert torch.equal(kp.view(-1, H, d)[rest.to(DEV)], k0.view(-1, H, d)[rest.to(DEV)])
    bad = table.clone()
    bad[1, 0] = kp.shape[0]
    k1 = kp.clone()
    mb.magicdec_paged_append(k, v, kp, vp, bad, i32([32, 3]), None)          # all of 0 past, all of 1 outside
    assert mb.magicdec_device_error() in (3, 5)
    assert torch.equal(kp, k1)


# ---------------------------------------------------------------------- accept
@pytest.mark.parametrize("B,n,V,tree,counts", [
    (1, 1, 1, None, None), (1, 1, 7, None, None), (3, 9, 5, "random", None), (5, 32, 3, "random", [32, 0, 1, 20, 31]),
    (2, 40, 1003, "random", None), (4, 64, 128257, "star", None), (130, 12, 4099, "random", None),
    (2, 256, 6, "random", None), (3, 256, 2, "chain", None), (2, 256, 2, None, [256, 100]), (300, 5, 33, "forest", None),
])
def test_accept(B, n, V, tree, counts):
    g = gen(71)
    # few different logits, so that rows have ties; tokens that follow them often
    target = torch.randint(0, 4, (B, n, V), generator=g).float() * 0.5 - 1.0
    target[target == 0] = -0.0
    tok = torch.randint(0, V, (B, n), generator=g, dtype=I32)
    parent = None if tree is None else make_tree(B, n, tree, 72)
    top = torch.where(target == target.amax(-1, keepdim=True), torch.arange(V), V).amin(-1)
    pr = (torch.arange(n) - 1).expand(B, n) if parent is None else parent.long()
    follow = torch.rand((B, n), generator=g) < 0.7
    tok = torch.where(follow, top.gather(1, pr.clamp(min=0)), tok).to(I32)
    got = mb.magicdec_tree_accept(target.to(DEV), tok.to(DEV), parent=None if parent is None else parent.to(DEV),
                                  n_nodes=i32(counts))
    for a, r in zip(got, accept_ref(target, tok, parent, counts)):
        assert torch.equal(a.cpu(), r)


@pytest.mark.parametrize("B,V", [(130, 10007), (320, 4098)])
def test_accept_full_depth_in_large_batches(B, V):
    """Every level of a chain, with few CTAs a row."""
    n = 7
    g = gen(73)
    target = torch.randn((B, n, V), generator=g)
    tok = torch.zeros((B, n), dtype=I32)
    tok[:, 1:] = target.argmax(-1)[:, :-1].to(I32)
    tok[::5, 4] = -1                                  # some end at level 3
    got = mb.magicdec_tree_accept(target.to(DEV), tok.to(DEV))
    for a, r in zip(got, accept_ref(target, tok, None, None)):
        assert torch.equal(a.cpu(), r)
    assert got[0][:6].tolist() == [3, 6, 6, 6, 6, 3]


def test_accept_infinite_logits_and_chain():
    B, n, V = 2, 4, 37
    target = torch.full((B, n, V), -float("inf"))
    target[1, :, 36] = -1e30
    target[1, 2, 35] = 3e38
    tok = torch.tensor([[9, 0, 0, 0], [9, 36, 36, 35]], dtype=I32)
    got = mb.magicdec_tree_accept(target.to(DEV), tok.to(DEV))
    for a, r in zip(got, accept_ref(target, tok, None, None)):
        assert torch.equal(a.cpu(), r)
    assert got[0].tolist() == [3, 3]


# ---------------------------------------------------------------------- commit
@pytest.mark.parametrize("layers,H_kv,d,page,n", [(1, 8, 128, 16, 20), (3, 1, 64, 7, 9), (2, 5, 128, 100, 33),
                                                  (2, 2, 64, 1, 256), (1, 40, 128, 16, 40)])
def test_commit(layers, H_kv, d, page, n):
    lens = [0, 45, 100, 3, 17]
    B = len(lens)
    _, _, table = make_cache(lens, n, page, H_kv, d, 81, DEV)
    g = gen(82)
    shape = (layers, B * table.shape[1] + 3, page, H_kv, d)
    kp, vp = (torch.randn(shape, generator=g).to(BF16).to(DEV) for _ in range(2))
    n_acc, path = [-1, 0, n - 1, min(n - 1, 8), n // 2], torch.full((B, n), -1, dtype=I32)
    for b, a in enumerate(n_acc):        # ascending from node 0, with and without gaps
        if a >= 0:
            path[b, 0] = 0
            path[b, 1:a + 1] = 1 + torch.randperm(n - 1, generator=g)[:a].sort().values.to(I32)
    ref = [kp.clone(), vp.clone()]
    for x, x0 in zip(ref, (kp, vp)):
        for b in range(B):
            rows = rows_of(table, b, lens[b] + torch.arange(n), page).to(DEV)
            y, y0 = x.view(layers, -1, H_kv, d), x0.view(layers, -1, H_kv, d)
            m = n_acc[b] + 1
            y[:, rows[:m]] = y0[:, rows[path[b, :m].long().to(DEV)]]
    args = (kp, vp) if layers > 1 else (kp[0], vp[0])
    mb.magicdec_tree_commit(*args, table, i32(lens), path.to(DEV), i32(n_acc))
    assert torch.equal(kp, ref[0]) and torch.equal(vp, ref[1])


def test_commit_skips_what_it_cannot_reach():
    B, n, H_kv, d, page = 2, 8, 2, 64, 16
    kp, vp, table = make_cache([24] * B, n, page, H_kv, d, 84, DEV)           # 32 slots
    k0 = kp.clone()
    path = torch.tensor([[0, 3, 99, -4, 7, -1, -1, -1], [0, 2, 5, 6, -1, -1, -1, -1]], dtype=I32)
    bad = table.clone()
    bad[1, 1] = -1
    mb.magicdec_tree_commit(kp, vp, bad, i32([26, 14]), path.to(DEV), i32([4, 3]))
    assert mb.magicdec_device_error() in (3, 5)
    # sequence 0: slot 27 <- 29; entries 99 and -4 and slot 33 are skipped.  1: slots 16.. are outside
    ref = k0.clone().view(-1, H_kv, d)
    r = rows_of(table, 0, torch.arange(32), page)
    ref[r[27]] = k0.view(-1, H_kv, d)[r[29]]
    assert torch.equal(kp.view(-1, H_kv, d), ref)


# --------------------------------------------------------------- streams, graphs
def _step_inputs(seed, B=3, n=24, H_q=32, H_kv=8, d=128, V=5003, page=16, L=700, layers=2):
    g = gen(seed)
    lens = [L, L // 3, 0][:B]
    _, _, table = make_cache(lens, n, page, H_kv, d, seed, DEV, extra_slots=64)
    shape = (layers, B * table.shape[1] + 3, page, H_kv, d)
    kp, vp = (torch.randn(shape, generator=g).to(BF16).to(DEV) for _ in range(2))
    qkv = torch.randn((layers, B, n, H_q + 2 * H_kv, d), generator=g).to(BF16).to(DEV)
    parent = make_tree(B, n, "random", seed)
    target = torch.randn((B, n, V), generator=g)
    tok = torch.randint(0, V, (B, n), generator=g, dtype=I32)
    pr = parent.long().clamp(min=0)
    tok = torch.where(torch.rand((B, n), generator=g) < 0.5, target.argmax(-1).gather(1, pr).to(I32), tok)
    inv = (500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    return dict(lens=lens, table=table, kp=kp, vp=vp, qkv=qkv, parent=parent.to(DEV), target=target.to(DEV),
                tok=tok.to(DEV), inv=inv, len=i32(lens), H=(H_q, H_kv, H_kv), layers=layers, n=n)


def _step(s, stream=None):
    outs = []
    for layer in range(s["layers"]):
        q, k, v = s["qkv"][layer].split(s["H"], dim=2)
        kp, vp = s["kp"][layer], s["vp"][layer]
        q = mb.magicdec_paged_append(k, v, kp, vp, s["table"], s["len"], s["inv"], q=q, parent=s["parent"],
                                     stream=stream)
        outs.append(mb.magicdec_tree_attn(q, kp, vp, s["table"], s["len"], parent=s["parent"], stream=stream))
    n_acc, path, tok = mb.magicdec_tree_accept(s["target"], s["tok"], parent=s["parent"], stream=stream)
    mb.magicdec_tree_commit(s["kp"], s["vp"], s["table"], s["len"], path, n_acc, stream=stream)
    return outs, n_acc, path, tok


def test_a_step_of_all_four():
    """Append, attention in two layers, acceptance, commit and the next lengths, against the plain
    forms chained the same way; the committed cache then serves a chain of one token."""
    s = _step_inputs(91)
    B, n, layers, page = 3, s["n"], s["layers"], s["kp"].shape[2]
    H_q, H_kv, _ = s["H"]
    d = s["kp"].shape[-1]
    parent, lens = s["parent"].cpu(), s["lens"]
    k_ref, v_ref = s["kp"].clone(), s["vp"].clone()
    outs, n_acc, path, tok = _step(s)
    depth = torch.tensor([[len(ancestors(parent[b].tolist(), i)) - 1 for i in range(n)] for b in range(B)])
    na, pt, tk = accept_ref(s["target"].cpu(), s["tok"].cpu(), parent, None)
    assert torch.equal(n_acc.cpu(), na) and torch.equal(path.cpu(), pt) and torch.equal(tok.cpu(), tk)
    assert int(na.max()) >= 1
    for layer in range(layers):
        q, k, v = s["qkv"][layer].split(s["H"], dim=2)
        qr = torch.empty((B, n, H_q, d), dtype=BF16, device=DEV)
        for b in range(B):
            pos = (lens[b] + depth[b]).to(DEV)
            rows = rows_of(s["table"], b, lens[b] + torch.arange(n), page).to(DEV)
            # the kernel's own rotated rows, once checked, go on: attention is compared on equal inputs
            keys, tol = rope_ref(k[b], pos, s["inv"], False)
            kr = k_ref[layer].view(-1, H_kv, d)
            kr[rows] = keys.to(BF16)
            v_ref[layer].view(-1, H_kv, d)[rows] = v[b]
            qr[b] = rope_ref(q[b], pos, s["inv"], False)[0].to(BF16)
        ref, tol = attn_ref(qr, k_ref[layer], v_ref[layer], s["table"], lens, parent, None)
        # a rotated row rounded the other way by a last-place difference of the fp32 sine moves a
        # score by up to 2^-7 of one product of 128: 2^-8 more per probability
        within(outs[layer], ref, 2 * tol)
        for b in range(B):
            m = int(na[b]) + 1
            rows = rows_of(s["table"], b, lens[b] + torch.arange(n), page).to(DEV)
            for x in (k_ref, v_ref):
                y = x[layer].view(-1, H_kv, d)
                y[rows[:m]] = y[rows[pt[b, :m].long().to(DEV)]].clone()
            got = s["vp"][layer].view(-1, H_kv, d)[rows[:m]]
            assert torch.equal(got, v_ref[layer].view(-1, H_kv, d)[rows[:m]])
    nxt, _ = mb.magicdec_step_lengths(s["len"], 0, s["table"].shape[1] * page, n_acc=n_acc)
    assert nxt.tolist() == [ln + int(a) + 1 for ln, a in zip(lens, na)]
    q = randn((B, 1, H_q, d), 92)
    got = mb.magicdec_tree_attn(q, s["kp"][0], s["vp"][0], s["table"], nxt)
    within(got, *attn_ref(q, s["kp"][0], s["vp"][0], s["table"], nxt.tolist(), None, None))


def test_step_captured_in_a_graph_and_on_side_streams():
    """A captured step replays to the bits of the eager one; two steps on two streams at once do
    not disturb each other."""
    ref = [_step(_step_inputs(93 + i)) for i in range(2)]
    s = _step_inputs(93)
    keep = (s["kp"].clone(), s["vp"].clone())
    graph = torch.cuda.CUDAGraph()
    _step(s)
    s["kp"].copy_(keep[0])
    s["vp"].copy_(keep[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = _step(s)
    for _ in range(2):
        s["kp"].copy_(keep[0])
        s["vp"].copy_(keep[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got[0] + list(got[1:]), ref[0][0] + list(ref[0][1:])):
            assert torch.equal(a, b)
    states = [_step_inputs(93 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [_step(st, stream=sm) for st, sm in zip(states, streams)]
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(both[i][0] + list(both[i][1:]), ref[i][0] + list(ref[i][1:])):
            assert torch.equal(a, b)
    handle = _step(_step_inputs(93), stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(handle[0][1], ref[0][0][1])


# ------------------------------------------------------------- far pages, debug build
def test_pages_past_32_bit_offsets():
    """A pool of more than 2^31 elements: the last pages are appended to, attended to and moved."""
    H_q, H_kv, d, page, n = 8, 8, 128, 64, 5
    n_pages = (1 << 31) // (page * H_kv * d) + 40
    kp, vp = (torch.empty((n_pages, page, H_kv, d), dtype=BF16, device=DEV) for _ in range(2))
    lens = [100, 30]
    table = torch.tensor([[n_pages - 1, n_pages - 7], [n_pages - 3, n_pages - 2]], dtype=I32, device=DEV)
    for pg in table.flatten().tolist():
        kp[pg], vp[pg] = randn((page, H_kv, d), pg), randn((page, H_kv, d), pg + 1)
    q, k, v = randn((2, n, H_q, d), 101), randn((2, n, H_kv, d), 102), randn((2, n, H_kv, d), 103)
    mb.magicdec_paged_append(k, v, kp, vp, table, i32(lens), None)
    small = torch.cat((kp[table.flatten().long()], torch.zeros_like(kp[:1]))), torch.cat(
        (vp[table.flatten().long()], torch.zeros_like(vp[:1])))
    near = torch.arange(4, dtype=I32, device=DEV).view(2, 2)
    for b in range(2):
        rows = rows_of(near, b, lens[b] + torch.arange(n), page).to(DEV)
        assert torch.equal(small[0].view(-1, H_kv, d)[rows], k[b]) and torch.equal(small[1].view(-1, H_kv, d)[rows], v[b])
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens))
    within(got, *attn_ref(q, *small, near, lens, None, None))
    mb.magicdec_tree_commit(kp, vp, table, i32(lens), i32([[0, 2, 4, -1, -1], [0, 3, -1, -1, -1]]), i32([2, 1]))
    for b, (dst, src) in enumerate((((1, 2), (2, 4)), ((1,), (3,)))):
        at = rows_of(table, b, lens[b] + torch.tensor(dst), page).to(DEV)
        assert torch.equal(vp.view(-1, H_kv, d)[at], v[b, list(src)])


@pytest.mark.parametrize("page,H_q,H_kv,d,n", [(2, 8, 2, 128, 40), (3, 16, 2, 64, 5), (1, 8, 1, 128, 20),
                                               (4, 8, 2, 128, 9), (5, 8, 2, 64, 33), (128, 8, 2, 128, 33),
                                               (136, 8, 2, 128, 33), (40, 4, 4, 128, 129)])
def test_attention_more_page_sizes(page, H_q, H_kv, d, n):
    lens = [515, 0, 129]
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 111, DEV, poison=True)
    q, parent = randn((3, n, H_q, d), 112), make_tree(3, n, "random", 113)
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=parent.to(DEV))
    within(got, *attn_ref(q, kp, vp, table, lens, parent, None))
    table[1, 0] = kp.shape[0]                       # outside the pool: zeros, and reported
    mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=parent.to(DEV))
    assert mb.magicdec_device_error() == 5


@pytest.mark.parametrize("page", [8, 24, 56, 72, 80, 96, 104, 125, 129, 192, 250, 264, 1000])
@pytest.mark.parametrize("H_q,H_kv,d,n", [(6, 2, 64, 7), (8, 2, 128, 40)])
def test_attention_tiles_over_pages(page, H_q, H_kv, d, n):
    """Tiles that run on over the pages' ends, and those that begin anew with each page."""
    lens, counts = [1207, 1, 2 * page, 129], [n, n, n, 1]
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 121, DEV, poison=True, counts=counts)
    q, parent = randn((4, n, H_q, d), 122), make_tree(4, n, "random", 123)
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=parent.to(DEV), n_nodes=i32(counts))
    within(got, *attn_ref(q, kp, vp, table, lens, parent, counts))
    assert mb.magicdec_device_error() == 0


DEBUG_CHILD = """
import json, sys, torch
sys.path.insert(0, {tests!r}); sys.path.insert(0, {root!r})
from long_context_self_gb300 import binding as mb
from tree_util import make_cache, make_tree
D = torch.device("cuda:0")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=D)
B, n, H, d, page = 2, 6, 2, 64, 16
kp, vp, table = make_cache([60, 60], 4, page, H, d, 1, D)             # 64 slots
q = torch.ones((B, n, 4, d), dtype=torch.bfloat16, device=D)
k = torch.ones((B, n, H, d), dtype=torch.bfloat16, device=D)
good = make_tree(B, n, "forest", 2).to(D)
bad = good.clone(); bad[1, 3] = 5
target = torch.randn((B, n, 50), device=D)
tok = torch.zeros((B, n), dtype=torch.int32, device=D)
path = i32([[0, 2, -1, -1, -1, -1], [0, -1, -1, -1, -1, -1]])
err = mb.magicdec_device_error
def tell(f):
    f(); return err()
res = dict(lib=mb.lib()._name.rsplit("/", 1)[-1])
res["in"] = [tell(lambda: mb.magicdec_paged_append(k, k, kp, vp, table, i32([10, 20]), parent=good, n_new=i32([6, 0]))),
             tell(lambda: mb.magicdec_tree_attn(q, kp, vp, table, i32([10, 20]), parent=good, n_nodes=i32([6, 0]))),
             tell(lambda: mb.magicdec_tree_accept(target, tok, parent=good, n_nodes=i32([6, 0]))),
             tell(lambda: mb.magicdec_tree_commit(kp, vp, table, i32([10, 20]), path, i32([1, -1])))]
res["out"] = [tell(lambda: mb.magicdec_paged_append(k, k, kp, vp, table, i32([10, 20]), parent=bad)),
              tell(lambda: mb.magicdec_paged_append(k, k, kp, vp, table, i32([10, -1]), n_new=i32([1, 7]))),
              tell(lambda: mb.magicdec_tree_attn(q, kp, vp, table, i32([10, 65]))),
              tell(lambda: mb.magicdec_tree_attn(q, kp, vp, table, i32([10, 20]), n_nodes=i32([7, 1]))),
              tell(lambda: mb.magicdec_tree_attn(q, kp, vp, table, i32([10, 20]), parent=bad)),
              tell(lambda: mb.magicdec_tree_accept(target, tok, parent=bad)),
              tell(lambda: mb.magicdec_tree_accept(target, tok, n_nodes=i32([-1, 6]))),
              tell(lambda: mb.magicdec_tree_commit(kp, vp, table, i32([10, 20]), path, i32([6, 0]))),
              tell(lambda: mb.magicdec_tree_commit(kp, vp, table, i32([10, 20]), path - 9, i32([1, 0])))]
print(json.dumps(res))
"""


def test_range_checking_build_records_and_release_build_does_not():
    import json
    import os
    import subprocess
    import sys
    from long_context_self_gb300 import build
    build.build(debug=True)
    tests = os.path.dirname(os.path.abspath(__file__))
    code = DEBUG_CHILD.format(tests=tests, root=os.path.dirname(tests))
    for library, name, out in (("debug", "libmagicdec_debug.so", 4), (None, "libmagicdec.so", 0)):
        env = {k: v for k, v in os.environ.items() if k != "MAGICDEC_LIBRARY"}
        if library:
            env["MAGICDEC_LIBRARY"] = library
        r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-3000:]
        res = json.loads(r.stdout.strip().splitlines()[-1])
        assert res["lib"] == name
        assert res["in"] == [0] * 4, res
        assert res["out"] == [out] * 9, res
