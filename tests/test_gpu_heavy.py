"""The heavy-hitter draft cache against plain 64-bit forms (tests/heavy_util.py): attention that adds every row's
weight up, and eviction of the rows of least weight."""
import pytest
import torch

from heavy_util import evict_ref, heavy_ref
from long_context_self_gb300 import binding as mb
from tree_util import gen

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


def cache(B, H_kv, cap, d, lens, seed):
    """Random rows, weights and positions; rows at or past the length NaN, with marks in weight and pos."""
    kc, vc = randn((B, H_kv, cap, d), seed), randn((B, H_kv, cap, d), seed + 1)
    weight = torch.rand((B, H_kv, cap), generator=gen(seed + 2)).to(DEV)
    pos = torch.randint(0, 1 << 20, (B, H_kv, cap), generator=gen(seed + 3), dtype=I32).to(DEV)
    for b, ln in enumerate(lens):
        ln = min(max(ln, 0), cap)
        kc[b, :, ln:] = float("nan")
        vc[b, :, ln:] = float("nan")
        weight[b, :, ln:] = float("nan")
        pos[b, :, ln:] = -5
    return kc, vc, weight, pos


# ------------------------------------------------------------------ attention
# (H_q, H_kv, d, n, cap, lens)
ATTN = [
    # the smallest calls
    (1, 1, 64, 1, 1, [1, 0]),
    (4, 4, 128, 1, 16, [1]),
    (4, 1, 64, 1, 16, [0, 1, 5, 16]),
    # lengths around a warp's 16 keys and a CTA's share, an odd capacity
    (32, 8, 128, 1, 601, [15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 513, 600, 601]),
    (8, 2, 64, 1, 70, [70, 69, 1]),
    # every number of row tiles, and groups that do not divide them
    (32, 8, 128, 2, 300, [300, 2, 111]),
    (12, 4, 128, 3, 333, [333, 40]),
    (32, 8, 128, 4, 300, [300, 5, 111]),
    (40, 8, 128, 5, 300, [300, 7, 111]),
    (32, 8, 64, 8, 300, [300, 9, 111]),
    (28, 4, 64, 4, 300, [300, 9, 111]),
    (16, 1, 128, 2, 300, [300, 9, 111]),
    (32, 1, 128, 1, 300, [300, 9, 0]),
    (5, 5, 64, 32, 300, [300, 32, 40]),
    # fewer rows than tokens: the first see nothing
    (8, 2, 128, 4, 40, [0, 1, 2, 3, 4]),
    (16, 2, 64, 4, 40, [0, 1, 2, 3, 4]),
    # long caches: wide clusters, scores beside one another in shared memory
    (8, 2, 128, 1, 20000, [20000, 1, 7777]),
    (10, 2, 128, 5, 12001, [12001, 3000]),
    (2, 1, 64, 1, 100003, [100003]),
    (4, 1, 128, 1, 300001, [300001, 12345]),
    (16, 2, 64, 4, 30001, [30001, 3]),
    (16, 2, 128, 1, 30001, [29999, 3]),
    (6, 2, 64, 5, 30001, [30001, 6]),
    # more pairs than fill the GPU
    (16, 8, 64, 1, 130, [(b * 37) % 131 for b in range(200)]),
    # lengths out of range are clamped
    (8, 2, 128, 3, 50, [51, 1 << 30, -1, -(1 << 31)]),
]


@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("H_q,H_kv,d,n,cap,lens", ATTN)
def test_attention(H_q, H_kv, d, n, cap, lens, fresh):
    B = len(lens)
    kc, vc, weight, pos = cache(B, H_kv, cap, d, lens, 3)
    q = randn((B, n, H_q, d), 9)
    next_pos = [1000 * b + 7 for b in range(B)] if fresh else None
    w0, p0 = weight.clone(), pos.clone()
    out = torch.full_like(q, float("nan"))
    got = mb.magicdec_heavy_attn(q, kc, vc, weight, i32(lens), pos=pos, next_pos=i32(next_pos), out=out)
    assert got is out
    used = torch.arange(cap, device=DEV) < i32([min(max(x, 0), cap) for x in lens])[:, None, None]
    used = used.expand_as(weight)
    (ref, tol), (w, wt), p = heavy_ref(q, kc, vc, w0, p0, lens, next_pos)
    within(got, ref, tol, "out")
    assert weight[~used].isnan().all()                 # rows behind the last one as they were
    within(weight[used], w[used], wt[used], "weight")
    assert torch.equal(pos, p)
    # the same again: the order of all sums is fixed
    w1, p1 = w0.clone(), p0.clone()
    again = mb.magicdec_heavy_attn(q, kc, vc, w1, i32(lens), pos=p1, next_pos=i32(next_pos))
    assert torch.equal(again, got) and torch.equal(w1[used], weight[used]) and torch.equal(p1, pos)


def test_attention_without_positions():
    kc, vc, weight, _ = cache(2, 2, 40, 128, [40, 17], 13)
    q, w0 = randn((2, 1, 8, 128), 14), weight.clone()
    mb.magicdec_heavy_attn(q, kc, vc, weight, i32([40, 17]))
    _, (w, wt), _ = heavy_ref(q, kc, vc, w0, torch.zeros_like(w0, dtype=I32), [40, 17], None)
    within(weight[0], w[0], wt[0])
    within(weight[1, :, :17], w[1, :, :17], wt[1, :, :17])


def test_weights_of_a_sequence_sum_to_its_query_rows():
    B, n, H_q, H_kv, d, cap = 3, 2, 8, 2, 64, 900
    lens = [900, 2, 130]
    kc, vc, weight, pos = cache(B, H_kv, cap, d, lens, 17)
    weight.zero_()
    mb.magicdec_heavy_attn(randn((B, n, H_q, d), 18), kc, vc, weight, i32(lens), pos=pos, next_pos=i32([0, 0, 0]))
    # n * G probabilities of one each, summed in fp32
    assert (weight.sum(-1) - n * H_q / H_kv).abs().max() < 1e-4


@pytest.mark.parametrize("n,H_q", [(3, 8), (8, 8), (5, 4)])
def test_a_token_behind_others_reaches_none_of_them(n, H_q):
    """Infinities and NaN in a block's own rows reach their token and later ones only."""
    B, H_kv, d, cap = 2, 2, 128, 200
    lens = [150, n]
    kc, vc, weight, pos = cache(B, H_kv, cap, d, lens, 21)
    q = randn((B, n, H_q, d), 22)
    w0, p0 = weight.clone(), pos.clone()
    clean = mb.magicdec_heavy_attn(q, kc, vc, weight, i32(lens), pos=pos, next_pos=i32([5, 6]))
    for b, ln in enumerate(lens):
        for i in range(1, n):
            vc[b, :, ln - n + i] = float("nan" if i % 2 else "inf")
            kc[b, :, ln - n + i] = float("nan")
    got = mb.magicdec_heavy_attn(q, kc, vc, w0, i32(lens), pos=p0, next_pos=i32([5, 6]))
    assert torch.equal(got[:, 0], clean[:, 0])
    assert got[:, 1:].isnan().all()


@pytest.mark.parametrize("n,H_q,d,cap", [(1, 8, 128, 200), (2, 8, 64, 12001), (3, 8, 128, 700), (8, 8, 64, 200), (8, 8, 128, 3000)])
def test_scores_that_are_not_numbers(n, H_q, d, cap):
    """A row that sees a NaN or a score of infinity is NaN, as are the weights of the rows that it sees;
    all others are as without."""
    B, H_kv = 4, 2
    G, lens = H_q // H_kv, [cap, cap - 7, cap - 20, cap]
    kc, vc, weight, pos = cache(B, H_kv, cap, d, lens, 81)
    q = randn((B, n, H_q, d), 82)
    w0, p0 = weight.clone(), pos.clone()
    clean = mb.magicdec_heavy_attn(q, kc, vc, weight, i32(lens), pos=pos, next_pos=i32([5] * B))
    kc[0, 0, 11, 3] = float("nan")                     # a row that all tokens see
    kc[1, 1] = float("nan")                            # every row of a head
    q[2, n - 1, 0, 5] = float("nan")                   # a query row
    kc[3, 0, 40, 9] = float("inf")                     # scores of either infinity: NaN, and nothing for this row
    bad = torch.zeros((B, n, H_kv, G), dtype=torch.bool, device=DEV)
    bad[0, :, 0] = bad[1, :, 1] = bad[2, n - 1, 0, 0] = True
    bad[3, :, 0] = q[3, :, :G, 9] > 0
    got = mb.magicdec_heavy_attn(q, kc, vc, w0, i32(lens), pos=p0, next_pos=i32([5] * B))
    hit = bad.view(B, n, H_q)
    assert got[hit].isnan().all() and not got[~hit].isnan().any()
    assert torch.equal(got[:3][~hit[:3]], clean[:3][~hit[:3]]) and torch.equal(got[3, :, G:], clean[3, :, G:])
    any_row = bad.any(-1).any(1)                       # of a KV head
    for b in range(B):
        for h in range(H_kv):
            if not any_row[b, h]:
                assert torch.equal(w0[b, h, :lens[b]], weight[b, h, :lens[b]])
            else:
                first = int(bad[b, :, h].any(-1).nonzero().max())          # the last token that is NaN sees the most
                assert w0[b, h, :lens[b] - n + 1 + first].isnan().all()


def test_attention_of_growing_scores():
    """Keys whose scores grow, and fall, along the rows: the running maximum moves often."""
    B, n, H_q, H_kv, d, cap = 2, 2, 8, 2, 128, 2000
    kc, vc, weight, pos = cache(B, H_kv, cap, d, [cap] * B, 31)
    for b, (lo, hi) in enumerate(((0.05, 12.0), (12.0, 0.05))):
        kc[b] = (kc[b].float() * torch.linspace(lo, hi, cap, device=DEV)[:, None]).to(BF16)
    q, w0 = randn((B, n, H_q, d), 32), weight.clone()
    got = mb.magicdec_heavy_attn(q, kc, vc, weight, i32([cap] * B), pos=pos, next_pos=i32([0, 0]))
    (ref, tol), (w, wt), _ = heavy_ref(q, kc, vc, w0, pos, [cap] * B, [0, 0])
    # scores reach 12 * |q| |k| / sqrt(d), some 200: fp32 products of that size are off by
    # 128 * 2^-24 * 12 * sum |q k| / sqrt(d) < 1e-3, which the exponential turns into a relative error
    within(got, ref, tol * (1 + 1e-3 / 2.0 ** -8))
    within(weight, w, wt * (1 + 1e-3 / 2.0 ** -12))


# -------------------------------------------------------------------- eviction
# (layers, B, H_kv, d, cap, lens, budget, sink, recent, weights)
EVICT = [
    (1, 1, 1, 64, 2, [2], 1, 0, 0, "random"),
    (1, 1, 8, 128, 528, [517], 512, 4, 64, "random"),
    (3, 2, 2, 64, 100, [100, 37], 36, 2, 5, "random"),
    # nothing to do, exactly full, an empty cache, lengths out of range
    (2, 6, 2, 128, 50, [50, 20, 21, 0, 99, -3], 20, 4, 16, "random"),
    # ties: all alike, few values, zeros of both signs, infinities
    (1, 2, 2, 64, 300, [300, 290], 100, 0, 0, "alike"),
    (2, 2, 2, 64, 300, [300, 290], 100, 3, 40, "few"),
    (1, 2, 1, 64, 300, [300, 290], 299, 0, 299, "few"),
    # positions that are alike too: the lower row stays
    (1, 2, 2, 64, 200, [200, 150], 90, 0, 0, "twins"),
    # every row protected that can be
    (1, 1, 2, 64, 64, [64], 40, 10, 30, "random"),
    # most of the rows go, more moves than are listed at a time
    (1, 2, 2, 128, 4000, [4000, 2100], 2000, 16, 100, "random"),
    (1, 1, 1, 64, 5000, [5000], 3, 1, 1, "few"),
    # few rows to go, of many that are alike, in their positions too
    (2, 3, 4, 64, 300, [300, 295, 285], 284, 2, 20, "few"),
    (1, 2, 8, 64, 1041, [1041, 1035], 1030, 0, 0, "alike"),
    (1, 2, 8, 64, 1041, [1041, 1035], 1025, 5, 7, "twins"),
    (1, 2, 8, 64, 1030, [1030, 1029], 1029, 5, 7, "twins"),
    (1, 3, 2, 128, 77, [77, 70, 64], 61, 0, 9, "twins"),
    # many caches, each of a few rows, of which a few or many go
    (8, 39, 8, 64, 70, [(b * 29) % 72 for b in range(39)], 30, 2, 5, "random"),
    (8, 39, 8, 64, 70, [(b * 29) % 72 for b in range(39)], 20, 0, 0, "few"),
    (8, 39, 8, 64, 70, [(b * 29) % 72 for b in range(39)], 33, 0, 0, "twins"),
    (2, 200, 8, 64, 280, [(b * 29) % 282 for b in range(200)], 130, 5, 20, "random"),
    # more rows than keys in shared memory
    (1, 1, 1, 64, 30001, [30001], 29000, 16, 1000, "random"),
    (1, 1, 1, 64, 30001, [29990], 1000, 16, 100, "few"),
]


@pytest.mark.parametrize("layers,B,H_kv,d,cap,lens,budget,sink,recent,weights", EVICT)
def test_eviction(layers, B, H_kv, d, cap, lens, budget, sink, recent, weights):
    g = gen(41)
    lead = (layers, B, H_kv, cap)
    kc, vc = torch.randn((*lead, d), generator=g).to(BF16), torch.randn((*lead, d), generator=g).to(BF16)
    if weights == "random":
        w = torch.rand(lead, generator=g) ** 4
    elif weights == "few":
        w = torch.tensor([0.0, -0.0, 1.0, 1e-30, float("inf"), 2.5])[torch.randint(0, 6, lead, generator=g)]
    else:
        w = torch.full(lead, 0.25)
    # distinct positions, in any order, of four times as many
    pos = (torch.rand(lead, generator=g).argsort(-1) * 4 + torch.randint(0, 4, lead, generator=g)).to(I32)
    if weights == "twins":
        pos = pos // 16
    total = [4 * cap - 3 * b for b in range(B)]
    ref = evict_ref(kc, vc, w, pos, lens, total, budget, sink, recent)
    x = [t.to(DEV) for t in (kc, vc, w, pos)]
    if layers == 1:
        x = [t[0] for t in x]
    got = mb.magicdec_heavy_evict(*x, i32(lens), i32(total), budget, n_sink=sink, n_recent=recent)
    assert got.tolist() == ref[4]
    for mine, want, what in zip(x, ref, ("k", "v", "weight", "pos")):
        assert torch.equal(mine.cpu().view(want.shape), want), what


def test_steps_follow_the_64_bit_cache():
    """Tokens appended, attended and evicted one after another: the cache holds the rows that the plain
    form holds as long as the weights at the border differ by more than their bound."""
    B, H_q, H_kv, d, cap, budget, sink, recent = 3, 8, 2, 64, 40, 36, 2, 8
    lens = [budget - 3, budget, 10]
    kc, vc, weight, pos = cache(B, H_kv, cap, d, lens, 51)
    for x in (kc, vc, weight):
        x.nan_to_num_(0.0)
    for b, ln in enumerate(lens):
        pos[b, :, :ln] = torch.arange(ln, device=DEV, dtype=I32)
    total = list(lens)
    seen = list(lens)
    shadow = [kc.clone(), vc.clone(), weight.double(), pos.clone()]
    length = i32(lens)
    for step in range(30):
        n = 1 + step % 3
        k, v, q = randn((B, H_kv, n, d), 60 + step), randn((B, H_kv, n, d), 160 + step), randn((B, n, H_q, d), 260 + step)
        for b in range(B):
            for x, y in ((kc, k), (vc, v), (shadow[0], k), (shadow[1], v)):
                x[b, :, seen[b]:seen[b] + n] = y[b]
        length = length + n
        seen = [x + n for x in seen]
        mb.magicdec_heavy_attn(q, kc, vc, weight, length, pos=pos, next_pos=i32(total))
        _, (shadow[2], _), shadow[3] = heavy_ref(q, shadow[0], shadow[1], shadow[2], shadow[3], seen, total)
        total = [x + n for x in total]
        length = mb.magicdec_heavy_evict(kc, vc, weight, pos, length, i32(total), budget, n_sink=sink, n_recent=recent)
        *host, seen = evict_ref(*(x.cpu()[None] for x in shadow), seen, total, budget, sink, recent)
        shadow = [x[0].to(DEV) for x in host]
        assert length.tolist() == seen
        for b, ln in enumerate(seen):
            assert torch.equal(pos[b, :, :ln], shadow[3][b, :, :ln]), step
            assert torch.equal(kc[b, :, :ln], shadow[0][b, :, :ln])
            assert (weight[b, :, :ln].double() - shadow[2][b, :, :ln]).abs().max() < 1e-4


@pytest.mark.parametrize("d", [64, 128])
def test_attention_right_behind_a_selection(d):
    """Kernels of a selection and of the attention that hold tensor memory, many in a row, each let go before the
    one in front has ended: they wait for one another in one order only."""
    B, n, H_q, H_kv, cap, w = 2, 8, 8, 2, 300, 32
    lens = i32([300, 77])
    kc, vc, weight, pos = cache(B, H_kv, cap, d, [300, 77], 91)
    q, q_win, k = randn((B, n, H_q, d), 92), randn((B, w, H_q, d), 93), randn((B, 2000, H_kv, d), 94)
    long = i32([2000, 1500])
    want = mb.magicdec_heavy_attn(q, kc, vc, weight.clone(), lens)
    idx, _ = mb.magicdec_snapkv_select(q_win, k, long, w, 5, 128)
    torch.cuda.synchronize()
    w0, got = weight.clone(), [torch.empty_like(q) for _ in range(20)]
    ws = torch.empty(mb.magicdec_snapkv_workspace_size(mb.kv_shape(B, H_q, H_kv, d, 2000), w), dtype=torch.uint8, device=DEV)
    idx2, n_sel = torch.empty_like(idx), torch.empty((B,), dtype=I32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in got:
            mb.magicdec_snapkv_select(q_win, k, long, w, 5, 128, idx=idx2, n_sel=n_sel, ws=ws)
            mb.magicdec_heavy_attn(q, kc, vc, w0, lens, out=out)
    for _ in range(3):
        for out in got:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx2, idx)
        assert all(torch.equal(out, want) for out in got)


def test_calls_on_a_stream_and_in_a_graph():
    """On a stream of their own, and captured and replayed beside another graph's calls."""
    B, H_q, H_kv, d, cap, budget = 4, 8, 2, 128, 300, 250
    lens, total = i32([300, 251, 250, 7]), i32([900, 901, 902, 903])
    x = cache(B, H_kv, cap, d, lens.tolist(), 71)
    q = randn((B, 2, H_q, d), 72)

    def step(kc, vc, weight, pos, out, left):
        mb.magicdec_heavy_attn(q, kc, vc, weight, lens, pos=pos, next_pos=total, out=out)
        mb.magicdec_heavy_evict(kc, vc, weight, pos, lens, total, budget, n_sink=4, n_recent=32, draft_len_out=left)

    def fresh():
        return [t.clone() for t in x] + [torch.empty_like(q), torch.empty_like(lens)]

    want = fresh()
    step(*want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mine = fresh()
    side.wait_stream(torch.cuda.current_stream())
    mb.magicdec_heavy_attn(q, *mine[:3], lens, pos=mine[3], next_pos=total, out=mine[4], stream=side)
    mb.magicdec_heavy_evict(*mine[:4], lens, total, budget, n_sink=4, n_recent=32, draft_len_out=mine[5], stream=side)
    side.synchronize()
    sets, graphs = [fresh(), fresh()], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(*s)
    for s, g in zip(sets, graphs):
        for t, t0 in zip(s, fresh()):
            t.copy_(t0)
        g.replay()
    torch.cuda.synchronize()
    for got in (mine, *sets):
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
