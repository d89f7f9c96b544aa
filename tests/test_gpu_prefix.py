"""Attention behind shared prefixes against a plain 64-bit form (tests/heavy_util.prefix_ref), and a step of append,
attention, acceptance and commit behind one."""
import pytest
import torch

from heavy_util import prefix_ref
from long_context_self_gb300 import binding as mb
from tree_util import gen, make_tree, rows_of

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


def make(plens, first, lens, n, page, H_kv, d, seed, counts=None, poison=True):
    """A pool with shuffled pages for the prefixes and the sequences' own slots; rows that nobody sees are NaN."""
    g = gen(seed)
    B, P = len(lens), len(plens)
    mp, pp = -(-(max(lens) + n) // page), max(1, -(-max(plens) // page))
    pages = B * mp + P * pp + 2
    perm = torch.randperm(pages, generator=g).to(I32)
    table, ptable = perm[: B * mp].view(B, mp), perm[B * mp: B * mp + P * pp].view(P, pp)
    kp, vp = (torch.randn((pages, page, H_kv, d), generator=g).to(BF16) for _ in range(2))
    if poison:
        used = torch.zeros((pages * page,), dtype=torch.bool)
        for b in range(B):
            m = n if counts is None else counts[b]
            if m:
                used[rows_of(table, b, torch.arange(lens[b] + m), page)] = True
        for x in range(P):
            if first[x + 1] > first[x] and plens[x]:
                used[rows_of(ptable, x, torch.arange(plens[x]), page)] = True
        kp.view(-1, H_kv, d)[~used] = float("nan")
        vp.view(-1, H_kv, d)[~used] = float("nan")
    return kp.to(DEV), vp.to(DEV), ptable.contiguous().to(DEV), table.contiguous().to(DEV)


# (H_q, H_kv, d, n, plens, first, lens, page, tree, counts)
CASES = [
    # the smallest calls
    (4, 4, 128, 1, [1], None, [0], 16, None, None),
    (4, 1, 64, 1, [0], None, [0, 1, 5], 16, None, None),
    (8, 2, 128, 1, [300], None, [0, 40, 3], 16, None, None),
    # prefixes around the tile of 128 keys
    (32, 8, 128, 1, [127], None, [5, 130], 16, None, None),
    (32, 8, 128, 2, [128], None, [5, 130], 16, "chain", None),
    (32, 8, 128, 2, [129], None, [127, 126], 16, "chain", None),
    # one row tile for all, two, several pairs; nodes of one sequence in two row tiles and blocks
    (32, 8, 128, 4, [1000], None, [10] * 8, 16, "random", None),
    (32, 8, 128, 5, [1000], None, [10, 0, 300, 7, 9, 64, 11, 12, 13], 16, "random", None),
    (32, 8, 128, 7, [777], None, [20] * 40, 16, "random", None),
    (8, 2, 64, 33, [900], None, [50, 2, 17], 64, "random", None),
    (16, 4, 128, 100, [500], None, [130, 7, 0], 64, "random", None),
    (8, 8, 64, 256, [260], None, [40, 3], 128, None, None),
    # long enough that a prefix is cut over many CTAs
    (8, 2, 128, 1, [20000], None, [100, 50, 7], 16, None, None),
    (8, 2, 128, 3, [9000], None, [100] * 50, 64, "random", None),
    # few rows, each in many parts: clusters that share them, and own slots in the list
    (16, 1, 128, 1, [16000], None, [10, 300, 0], 16, None, None),
    (16, 1, 64, 2, [9000, 7000], [0, 1, 2], [10, 3], 64, "chain", None),
    (5, 1, 128, 1, [12000], None, [33], 16, None, None),
    (16, 1, 128, 5, [6000], None, [10, 65], 16, "random", None),
    # groups: empty ones, of one sequence, sequences in none, prefixes of no length
    (8, 2, 128, 2, [300, 500, 77], [0, 2, 2, 5], [10, 20, 0, 40, 50], 16, "random", None),
    (8, 2, 64, 3, [300, 0, 77, 1200], [1, 3, 4, 4, 6], [10, 20, 0, 40, 50, 300, 8, 9], 16, "forest", None),
    (32, 8, 128, 9, [300, 140, 1], [0, 30, 31, 40], [11] * 40, 16, "random", None),
    (24, 8, 64, 5, [701, 9, 333], [0, 6, 13, 20], [(b * 31) % 90 for b in range(20)], 48, "random",
     [b % 6 for b in range(20)]),
    (8, 2, 128, 4, [64] * 30, list(range(31)), [(b * 7) % 40 for b in range(30)], 16, "random", None),
    # trees of different sizes, some without nodes, whole groups without
    (32, 8, 128, 13, [200, 100], [0, 3, 5], [200, 0, 30, 64, 5], 16, "random", [13, 0, 1, 0, 0]),
    (32, 8, 128, 80, [300], None, [20, 0, 5], 16, "random", [80, 0, 33]),
    # page sizes: longer than a tile, not a multiple of 8 or of anything, of few rows
    (8, 2, 128, 3, [999], None, [128, 256, 1], 256, "random", None),
    (8, 2, 128, 3, [999], None, [70, 9], 200, "random", None),
    (8, 2, 128, 30, [999, 30], [0, 2, 3], [70, 9, 30], 100, "random", None),
    (8, 2, 64, 6, [301], None, [70, 3], 7, "random", None),
    (8, 2, 64, 40, [301, 64], [0, 1, 2], [20, 2], 1, "random", None),
    (8, 2, 128, 2, [150], None, [20, 2], 3, "random", None),
    # group sizes that do not divide a row tile
    (21, 3, 128, 19, [411], None, [20, 20, 7], 16, "random", None),
    (100, 1, 128, 2, [411], None, [20, 3], 16, "random", None),
    (128, 1, 64, 1, [411], None, [20, 3, 5], 16, None, None),
    (7, 7, 128, 2, [411], None, [20] * 70, 16, "chain", None),
]


@pytest.mark.parametrize("n,H_q,d", [(1, 8, 128), (4, 8, 64), (8, 8, 128), (20, 8, 128), (70, 8, 64)])
def test_scores_that_are_not_numbers(n, H_q, d):
    """A row that sees a NaN, in its prefix or among its own positions, is NaN; all others are as without."""
    H_kv, page, first, plens, lens = 2, 16, [0, 3, 5], [900, 300], [40, 130, 20, 0, 300]
    B, G = len(lens), H_q // H_kv
    kp, vp, ptable, table = make(plens, first, lens, n, page, H_kv, d, 25)
    q = randn((B, n, H_q, d), 26)
    args = (ptable, i32(plens), table, i32(lens), i32(first))
    clean = mb.magicdec_prefix_attn(q, kp, vp, *args)
    hit = torch.zeros((B, n, H_kv, G), dtype=torch.bool, device=DEV)
    kp[int(ptable[1, 5]), 3, 0, 7] = float("nan")      # a prefix's row: both sequences behind it
    hit[3:, :, 0] = True
    kp[table[0, :2].long(), :, 1] = float("nan")       # most of a sequence's own positions
    hit[0, :, 1] = True
    q[1, n - 1, 2, 1] = float("nan")                   # a query row
    hit[1, n - 1, 2 // G, 2 % G] = True
    got = mb.magicdec_prefix_attn(q, kp, vp, *args)
    hit = hit.view(B, n, H_q)
    assert got[hit].isnan().all()
    assert torch.equal(got[~hit], clean[~hit])
    kp[ptable[0].long(), :, 1] = float("nan")          # all of a prefix
    got = mb.magicdec_prefix_attn(q, kp, vp, *args)
    assert got[:3, :, G:].isnan().all() and torch.equal(got[:2, :n - 1, :G], clean[:2, :n - 1, :G])


@pytest.mark.parametrize("H_q,H_kv,d,n,plens,first,lens,page,tree,counts", CASES)
def test_attention(H_q, H_kv, d, n, plens, first, lens, page, tree, counts):
    B, P = len(lens), len(plens)
    groups = first or [0, B]
    kp, vp, ptable, table = make(plens, groups, lens, n, page, H_kv, d, 5, counts)
    q = randn((B, n, H_q, d), 6)
    parent = None if tree is None else make_tree(B, n, tree, 7)
    shape = mb.paged_shape(B, H_q, H_kv, d, page, kp.shape[0], table.shape[1])
    ws = torch.full((mb.magicdec_prefix_attn_workspace_size(shape, P, n),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, float("nan"))
    args = dict(first=i32(first), parent=None if parent is None else parent.to(DEV), n_nodes=i32(counts))
    got = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32(plens), table, i32(lens), out=out, ws=ws, **args)
    assert got is out
    within(got, *prefix_ref(q, kp, vp, ptable, plens, groups, table, lens, parent, counts))
    for b, m in enumerate(counts or []):
        assert (got[b, m:] == 0).all()
    again = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32(plens), table, i32(lens), **args)
    assert torch.equal(got, again)


def test_many_sequences_and_prefixes():
    """More entries of the list than a CTA has threads."""
    B, P, n, H_q, H_kv, d, page = 900, 300, 2, 8, 2, 64, 16
    lens, plens = [(b * 37) % 50 for b in range(B)], [(g * 53) % 200 for g in range(P)]
    first = [g * 3 for g in range(P + 1)]
    counts = [b % 3 for b in range(B)]
    kp, vp, ptable, table = make(plens, first, lens, n, page, H_kv, d, 15, counts)
    q, parent = randn((B, n, H_q, d), 16), make_tree(B, n, "random", 17)
    got = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32(plens), table, i32(lens), first=i32(first),
                                  parent=parent.to(DEV), n_nodes=i32(counts))
    within(got, *prefix_ref(q, kp, vp, ptable, plens, first, table, lens, parent, counts))


def test_same_values_as_the_tree_attention_of_whole_contexts():
    """Tables that begin with the prefix's pages, within both calls' bounds."""
    B, n, H_q, H_kv, d, page, Lp = 6, 5, 32, 8, 128, 16, 640
    kp, vp, ptable, table = make([Lp], [0, B], [50] * B, n, page, H_kv, d, 25)
    q, parent, lens = randn((B, n, H_q, d), 26), make_tree(B, n, "random", 27).to(DEV), i32([50, 3, 0, 17, 49, 22])
    mine = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32([Lp]), table, lens, parent=parent)
    whole = torch.cat((ptable.expand(B, -1), table), 1).contiguous()
    other = mb.magicdec_tree_attn(q, kp, vp, whole, lens + Lp, parent=parent)
    ref, tol = prefix_ref(q, kp, vp, ptable, [Lp], [0, B], table, lens.tolist(), parent.cpu(), None)
    within(mine, ref, tol)
    within(other, ref, tol)


def test_lengths_and_groups_out_of_range():
    """Lengths are clamped to the capacities, groups to the batch; bad parents count as none."""
    B, n, H_q, H_kv, d, page = 4, 5, 8, 2, 128, 16
    kp, vp, ptable, table = make([160, 160], [0, 2, 4], [59] * B, n, page, H_kv, d, 35, poison=False)   # 64 own slots
    q = randn((B, n, H_q, d), 36)
    parent = torch.tensor([[-1, 0, 5, 9, -7], [0, 0, 1, 2, 3], [-1, 1, 2, 3, 4], [-1, 0, 0, 2147483647, -2147483648]],
                          dtype=I32)
    lens = [64, 2**31 - 1, 62, -3]
    got = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32([1 << 30, -5]), table, i32(lens), first=i32([-9, 2, 99]),
                                  parent=parent.to(DEV), n_nodes=i32([5, 99, 5, 5]))
    within(got, *prefix_ref(q, kp, vp, ptable, [160, 0], [0, 2, 4], table, [64, 64, 62, 0], parent, None))


def test_what_other_nodes_hold():
    """Infinities and NaN in a node's own rows reach it and its descendants only."""
    B, n, H_q, H_kv, d, page, Lp = 3, 6, 8, 2, 128, 16, 300
    for lens in ([40] * B, [125] * B):
        kp, vp, ptable, table = make([Lp], [0, B], lens, n, page, H_kv, d, 45)
        q, parent = randn((B, n, H_q, d), 46), torch.tensor([[-1, 0, 0, 1, 2, 4]] * B, dtype=I32, device=DEV)
        args = (ptable, i32([Lp]), table, i32(lens))
        clean = mb.magicdec_prefix_attn(q, kp, vp, *args, parent=parent)
        for b in range(B):
            row = rows_of(table, b, torch.tensor([lens[b] + 2]), page).to(DEV)
            vp.view(-1, H_kv, d)[row] = float("nan") if b else float("inf")
        got = mb.magicdec_prefix_attn(q, kp, vp, *args, parent=parent)
        assert torch.equal(got[:, [0, 1, 3]], clean[:, [0, 1, 3]])
        assert not torch.isfinite(got[:, [2, 4, 5]]).any()


def test_page_outside_the_pool():
    B, n, H_q, H_kv, d, page = 2, 3, 8, 2, 128, 16
    kp, vp, ptable, table = make([300], [0, B], [40, 40], n, page, H_kv, d, 55, poison=False)
    q = randn((B, n, H_q, d), 56)
    wrong = ptable.clone()
    for bad in (kp.shape[0], -1):
        wrong[0, 3] = bad
        got = mb.magicdec_prefix_attn(q, kp, vp, wrong, i32([300]), table, i32([40, 40]))
        assert mb.magicdec_device_error() == 5
        zk, zv = (torch.cat((x, torch.zeros_like(x[:1]))) for x in (kp, vp))
        wrong[0, 3] = kp.shape[0]
        within(got, *prefix_ref(q, zk, zv, wrong, [300], [0, B], table, [40, 40], None, None))


def test_growing_scores():
    """The prefix far above a sequence's own keys, and far below."""
    B, n, H_q, H_kv, d, page, Lp = 2, 9, 8, 2, 128, 64, 2000
    for lo, hi, own in ((0.05, 12.0, 1.0), (1.0, 0.05, 12.0)):
        kp, vp, ptable, table = make([Lp], [0, B], [300] * B, n, page, H_kv, d, 65)
        x = kp.view(-1, H_kv, d)
        rows = rows_of(ptable, 0, torch.arange(Lp), page).to(DEV)
        x[rows] = (x[rows].float() * torch.linspace(lo, hi, Lp, device=DEV)[:, None, None]).to(BF16)
        for b in range(B):
            rows = rows_of(table, b, torch.arange(300 + n), page).to(DEV)
            x[rows] = (x[rows].float() * own).to(BF16)
        q, parent = randn((B, n, H_q, d), 66), make_tree(B, n, "random", 67)
        got = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32([Lp]), table, i32([300] * B), parent=parent.to(DEV))
        ref, tol = prefix_ref(q, kp, vp, ptable, [Lp], [0, B], table, [300] * B, parent, None)
        # scores reach 12 * |q| |k| / sqrt(d), some 200: fp32 products of that size are off by
        # 128 * 2^-24 * 12 * sum |q k| / sqrt(d) < 1e-3, which the exponential turns into a relative error
        within(got, ref, tol * (1 + 1e-3 / 2.0 ** -8))


def test_steps_behind_a_shared_prompt():
    """A prompt appended once, then steps of trees behind it, normed and rotated by positions that count the prompt:
    every step's attention against the 64-bit form over what the cache holds, captured in a graph and not."""
    B, n, H_q, H_kv, d, page, Lp, V = 5, 7, 8, 2, 64, 16, 333, 50
    pp, mp = -(-Lp // page), 6
    pages = pp + B * mp
    kp, vp = (torch.zeros((pages, page, H_kv, d), dtype=BF16, device=DEV) for _ in range(2))
    perm = torch.randperm(pages, generator=gen(81)).to(I32).to(DEV)
    ptable, table = perm[:pp].view(1, pp).contiguous(), perm[pp:].view(B, mp).contiguous()
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    qw, kw = randn((d,), 82), randn((d,), 83)
    k, v = randn((1, Lp, H_kv, d), 84), randn((1, Lp, H_kv, d), 85)
    mb.magicdec_norm_append(k, v, kp, vp, ptable, i32([0]), inv, k_weight=kw)
    lens = i32([0] * B)
    for step in range(4):
        parent = make_tree(B, n, "random", 90 + step).to(DEV)
        depth = torch.zeros((B, n), dtype=I32)
        for b in range(B):
            for i in range(1, n):
                p = int(parent[b, i])
                depth[b, i] = depth[b, p] + 1 if p >= 0 else 0
        pos = (lens[:, None] + Lp + depth.to(DEV)).to(I32).contiguous()
        q, k, v = randn((B, n, H_q + 2 * H_kv, d), 100 + step).split([H_q, H_kv, H_kv], dim=2)
        q_out, out = (torch.empty((B, n, H_q, d), dtype=BF16, device=DEV) for _ in range(2))
        plen = i32([Lp])

        def layer():
            mb.magicdec_norm_append(k, v, kp, vp, table, lens, inv, q=q, q_weight=qw, k_weight=kw, pos=pos, q_out=q_out)
            mb.magicdec_prefix_attn(q_out, kp, vp, ptable, plen, table, lens, parent=parent, out=out)
        layer()
        first = out.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer()
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
        within(out, *prefix_ref(q_out, kp, vp, ptable, [Lp], [0, B], table, lens.tolist(), parent.cpu(), None))
        target = torch.randn((B, n, V), generator=gen(110 + step)).to(DEV)
        tok = torch.randint(0, V, (B, n), generator=gen(120 + step), dtype=I32).to(DEV)
        for b in range(B):                                     # some of the first children are accepted
            if b % 2 and n > 1:
                target[b, 0, tok[b, 1]] = 9.0
        n_acc, path, _ = mb.magicdec_tree_accept(target, tok, parent=parent)
        mb.magicdec_tree_commit(kp, vp, table, lens, path, n_acc)
        lens = (lens + n_acc + 1).to(I32)


def test_on_a_stream_of_its_own():
    B, n, H_q, H_kv, d, page = 3, 2, 8, 2, 128, 16
    kp, vp, ptable, table = make([300], [0, B], [40] * B, n, page, H_kv, d, 75)
    q, plen, lens = randn((B, n, H_q, d), 76), i32([300]), i32([40] * B)
    want = mb.magicdec_prefix_attn(q, kp, vp, ptable, plen, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mb.magicdec_prefix_attn(q, kp, vp, ptable, plen, table, lens, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
