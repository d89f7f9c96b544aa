"""The paged-cache and tree operators where an order between threads, a value in a masked place
or a size could go wrong: each against a plain form."""
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


@pytest.mark.parametrize("H_q,H_kv,d,n,lens,page,tree,counts", [
    (8, 2, 128, 2, [0, 127, 300], 16, "chain", None),
    (8, 2, 128, 13, [0, 1, 121, 700], 16, "random", [13, 2, 7, 13]),       # one row tile
    (8, 2, 64, 13, [120, 64, 9001], 48, "star", None),
    (8, 2, 64, 20, [250, 3], 100, None, None),                             # a causal block
    (8, 2, 128, 6, [500, 3], 7, "random", None),
    (8, 2, 64, 40, [301, 2], 1, "forest", None),
    (8, 2, 128, 40, [30000, 90], 64, "random", None),                      # two row tiles, joined
    (32, 8, 128, 64, [2000, 64, 0], 16, "random", [64, 33, 50]),
    (16, 4, 128, 256, [700, 5], 256, "random", None),                      # several pairs of row tiles
    (8, 8, 64, 200, [250], 16, None, None),
    # many entries a CTA, with one row tile, and with two of which the second is often empty
    (8, 2, 128, 20, [b * 37 % 300 for b in range(300)], 16, "random", [b * 29 % 21 for b in range(300)]),
    (8, 2, 64, 48, [b * 37 % 300 for b in range(300)], 24, "random", [b * 29 % 49 for b in range(300)]),
])
def test_attention_values_that_a_node_does_not_see(H_q, H_kv, d, n, lens, page, tree, counts):
    """A node's keys and values reach itself and its descendants only, whatever they are: infinities
    in single channels, of both signs, NaN in a whole row, a NaN key."""
    B = len(lens)
    kp, vp, table = make_cache(lens, n, page, H_kv, d, 221, DEV, poison=True, counts=counts)
    q = randn((B, n, H_q, d), 222)
    parent = None if tree is None else make_tree(B, n, tree, 223)
    kx, vx = kp.view(-1, H_kv, d), vp.view(-1, H_kv, d)
    k0, v0 = kp.clone(), vp.clone()                           # the same with zeros in their place
    k0x, v0x = k0.view(-1, H_kv, d), v0.view(-1, H_kv, d)
    more = torch.zeros((B, n, H_kv, d), dtype=torch.float64)  # what each node's own values add
    key = torch.zeros((B, n, H_kv), dtype=torch.bool)
    for b in range(B):
        m = n if counts is None else counts[b]
        rows = rows_of(table, b, lens[b] + torch.arange(m), page)
        picks = torch.randperm(m, generator=gen(224 + b))
        for what, i in enumerate(picks[: max(1, m // 3)].tolist()):
            h = (what // 4) % H_kv
            if what % 4 == 3:
                kx[rows[i], h, 5] = float("nan")
                k0x[rows[i], h, 5] = 0
                key[b, i, h] = True
                continue
            at = slice(None) if what % 4 == 2 else slice(what % 11, None, 17 + what)
            x = (float("inf"), -float("inf"), float("nan"))[what % 4]
            vx[rows[i], h, at] = x
            v0x[rows[i], h, at] = 0
            more[b, i, h, at] = x
    got = mb.magicdec_tree_attn(q, kp, vp, table, i32(lens), parent=None if parent is None else parent.to(DEV),
                                n_nodes=i32(counts)).cpu()
    ref, tol = (x.cpu() for x in attn_ref(q, k0, v0, table, lens, parent, counts))
    G = H_q // H_kv
    for b in range(B):
        for i in range(n if counts is None else counts[b]):
            path = ancestors(None if parent is None else parent[b].tolist(), i)
            ref[b, i] += more[b, path].sum(0).repeat_interleave(G, 0)
            ref[b, i][key[b, path].any(0).repeat_interleave(G)] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    far = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), far) and torch.equal(got[far].double(), ref[far])
    fine = torch.isfinite(ref)
    assert ((got.double() - ref).abs() - tol)[fine].max() <= 0


def test_attention_row_that_sees_nothing_beside_values_that_are_not_finite():
    """Roots past the capacity of an empty sequence: zero, whatever the nodes inside it hold."""
    H_q, H_kv, d, n = 4, 2, 128, 6
    kp, vp = randn((2, 4, H_kv, d), 231), randn((2, 4, H_kv, d), 232)
    vp[0, 1], vp[0, 3] = float("nan"), float("inf")
    table = torch.tensor([[0], [1]], dtype=I32, device=DEV)
    parent = i32([[-1, -1, 0, -1, -1, -1]] * 2)
    got = mb.magicdec_tree_attn(randn((2, n, H_q, d), 233), kp, vp, table, i32([0, 0]), parent=parent)
    assert (got[:, 4:] == 0).all() and torch.isfinite(got[1]).all()
    assert torch.isfinite(got[0, [0, 2]]).all()
    assert torch.isnan(got[0, 1]).all() and (got[0, 3] == float("inf")).all()


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


@pytest.mark.parametrize("B,V", [(3, 37), (40, 4099), (160, 1030)])
def test_accept_infinities_and_nan(B, V):
    """NaN counts as -inf, wherever in a row and in how many of its values; infinities as themselves."""
    n = 6
    g = gen(241)
    target = torch.randn((B, n, V), generator=g)
    inf, nan = float("inf"), float("nan")
    target[0::3, 0, ::2] = nan
    target[0::3, 1] = nan
    target[0::3, 2, 1:] = nan
    target[0::3, 2, 0] = -inf
    target[1::3, 0, V // 2] = inf
    target[1::3, 0, V - 1] = inf
    target[1::3, 1, 0] = nan
    target[1::3, 1, V - 1] = 1e30
    target[2::3, :2] = -inf
    target[2::3, 1, 3] = nan
    target[2::3, 1, V - 2] = -3e38
    plain = torch.where(torch.isnan(target), -inf, target)
    tok = torch.zeros((B, n), dtype=I32)
    tok[:, 1:] = torch.where(plain == plain.amax(-1, keepdim=True), torch.arange(V), V).amin(-1)[:, :-1].to(I32)
    ref = accept_ref(plain, tok, None, None)
    assert (ref[0] == n - 1).all()
    for a, r in zip(mb.magicdec_tree_accept(target.to(DEV), tok.to(DEV)), ref):
        assert torch.equal(a.cpu(), r)


# ----------------------------------------------------------------- steps of all
@pytest.mark.parametrize("page", [None, 16])
def test_steps_from_a_prompt(page):
    """A ragged prompt's append, then steps of append, attention, acceptance, commit and the next
    lengths, over a dense cache (page None: one page a sequence) or pages.  Every row of K and V is
    followed: as the append writes it (against the rotation's 64-bit form), and bit for bit through the
    commits.  Over the dense cache a StreamingLLM draft cache takes the accepted positions in."""
    B, n, H_q, H_kv, d, V, layers, P, steps = 3, 12, 8, 2, 128, 41, 2, 70, 4
    L_cap = P + steps * n
    g = gen(251)
    ps = L_cap if page is None else page
    mp = -(-L_cap // ps)
    pages = torch.arange(B) if page is None else torch.randperm(B * mp + 3, generator=g)[: B * mp]
    table = pages.view(B, mp).to(I32).to(DEV)
    shape = (layers, B if page is None else B * mp + 3, ps, H_kv, d)
    kp, vp = (torch.full(shape, float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    lens = [P, 1, 33]
    rows = [rows_of(table, b, torch.arange(L_cap), ps).to(DEV) for b in range(B)]

    def append(m, length, seed, **kw):
        x = [randn((B, m, H, d), seed + j) for j, H in enumerate((H_q, H_kv, H_kv))]
        out = []
        for layer in range(layers):
            k, v = x[1].roll(layer, -1), x[2].roll(layer, -1)
            q = mb.magicdec_paged_append(k, v, kp[layer], vp[layer], table, i32(length), inv, q=x[0], **kw)
            out.append((q, k, v))
        return out

    def check_rows(new, length, depth, counts):
        for layer, (_, k, v) in enumerate(new):
            for b in range(B):
                at = rows[b][length[b]:length[b] + counts[b]]
                pos = (length[b] + depth[b, :counts[b]]).to(DEV)
                within(kp[layer].view(-1, H_kv, d)[at], *rope_ref(k[b, :counts[b]], pos, inv, False))
                assert torch.equal(vp[layer].view(-1, H_kv, d)[at], v[b, :counts[b]])

    check_rows(append(P, [0] * B, 252, n_new=i32(lens)), [0] * B, torch.arange(P).expand(B, P), lens)
    ring, sinks = 16, 4
    if page is None:
        kc, vc = (torch.full((B, H_kv, sinks + ring, d), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
        origin, zero = i32([sinks] * B), i32([0] * B)
        mb.magicdec_draft_cache_update(kp[0], vp[0], kc, vc, zero, zero, i32(lens), origin, None, ring)
    total = 0
    for step in range(steps):
        parent = make_tree(B, n, "random", 260 + step)
        depth = torch.tensor([[len(ancestors(parent[b].tolist(), i)) - 1 for i in range(n)] for b in range(B)])
        new = append(n, lens, 270 + 10 * step, parent=parent.to(DEV))
        check_rows(new, lens, depth, [n] * B)
        for layer, (q, _, _) in enumerate(new):
            got = mb.magicdec_tree_attn(q, kp[layer], vp[layer], table, i32(lens), parent=parent.to(DEV))
            within(got, *attn_ref(q, kp[layer], vp[layer], table, lens, parent, None))
        target = torch.randn((B, n, V), generator=g)
        tok = target.argmax(-1).gather(1, parent.clamp(min=0).long())
        tok = torch.where(torch.rand((B, n), generator=g) < 0.8, tok, 0).to(I32)
        n_acc, path, out = mb.magicdec_tree_accept(target.to(DEV), tok.to(DEV), parent=parent.to(DEV))
        ref = accept_ref(target, tok, parent, None)
        assert torch.equal(n_acc.cpu(), ref[0]) and torch.equal(path.cpu(), ref[1]) and torch.equal(out.cpu(), ref[2])
        moved = []
        for x in (kp, vp):
            x = x.clone().view(layers, -1, H_kv, d)
            for b in range(B):
                m = int(ref[0][b]) + 1
                x[:, rows[b][lens[b]:lens[b] + m]] = x[:, rows[b][lens[b] + ref[1][b, :m].long()]].clone()
            moved.append(x)
        mb.magicdec_tree_commit(kp, vp, table, i32(lens), path, n_acc)
        for x, y in zip((kp, vp), moved):
            assert torch.equal(x.view(layers, -1, H_kv, d).view(torch.int16), y.view(torch.int16))
        now, _ = mb.magicdec_step_lengths(i32(lens), 0, L_cap, n_acc=n_acc)
        if page is None:
            mb.magicdec_draft_cache_update(kp[0], vp[0], kc, vc, i32(lens), i32(lens), now, origin, None, ring)
        lens = [ln + int(a) + 1 for ln, a in zip(lens, ref[0])]
        total += int(ref[0].sum())
        assert now.tolist() == lens
        if page is None:
            for b, ln in enumerate(lens):
                pos = torch.cat((torch.arange(min(ln, sinks)), torch.arange(max(sinks, ln - ring), ln)))
                slot = torch.where(pos < sinks, pos, sinks + (pos - sinks) % ring)
                assert torch.equal(kc[b][:, slot].transpose(0, 1), kp[0, b, pos])
                assert torch.equal(vc[b][:, slot].transpose(0, 1), vp[0, b, pos])
    assert total > 4
