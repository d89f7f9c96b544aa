"""The calls for batches behind a shared prompt and for a heavy-hitter draft cache, run together as a program uses them,
and where its memory is large, shared or captured."""
import json
import os
import subprocess
import sys

import pytest
import torch

from heavy_util import evict_ref, heavy_ref, prefix_ref
from long_context_self_gb300 import binding as mb
from tree_util import gen, rows_of

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, I32 = torch.bfloat16, torch.int32
HERE = os.path.dirname(os.path.abspath(__file__))


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
    return torch.tensor(x, dtype=I32, device=DEV)


def randn(shape, seed):
    return torch.randn(shape, generator=gen(seed)).to(BF16).to(DEV)


def within(got, ref, tol, what=""):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got.double() - ref).abs() - tol).max().item()
    assert over <= 0, f"{what}: off by {over:.3e} more than the bound"


class Step:
    """One layer of a speculative step of B samples of one prompt: gamma tokens drafted over the heavy-hitter
    cache, the block of gamma + 1 appended to the pages, normed and rotated, and verified behind the prompt,
    then the draft cache cut to its budget.  Every tensor is the step's own, so that it can be captured."""
    B, gamma, H_q, H_kv, d, page, Lp, budget = 6, 3, 8, 2, 64, 16, 500, 48

    def __init__(self, seed):
        B, d, H_kv, n = self.B, self.d, self.H_kv, self.gamma + 1
        pp, mp = -(-self.Lp // self.page), 4
        perm = torch.randperm(pp + B * mp, generator=gen(seed)).to(I32).to(DEV)
        self.ptable, self.table = perm[:pp].view(1, pp).contiguous(), perm[pp:].view(B, mp).contiguous()
        self.kp, self.vp = (randn((pp + B * mp, self.page, H_kv, d), seed + x) for x in (1, 2))
        self.plen, self.lens = i32([self.Lp]), i32([b * 7 % 40 for b in range(B)])
        self.inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
        self.qw, self.kw = randn((d,), seed + 3), randn((d,), seed + 4)
        self.qkv = randn((B, n, self.H_q + 2 * H_kv, d), seed + 5)
        self.pos = (self.lens[:, None] + self.Lp + torch.arange(n, device=DEV)).to(I32).contiguous()
        self.q_out, self.out = (torch.empty((B, n, self.H_q, d), dtype=BF16, device=DEV) for _ in range(2))
        # the draft cache: as many of the context's rows as it keeps
        cap = self.budget + self.gamma
        self.kc, self.vc = randn((B, H_kv, cap, d), seed + 6), randn((B, H_kv, cap, d), seed + 7)
        self.weight = torch.rand((B, H_kv, cap), generator=gen(seed + 8)).to(DEV)
        self.rpos = torch.stack([torch.randperm(self.Lp, generator=gen(seed + 9 + x))[:cap] for x in range(B * H_kv)])
        self.rpos = self.rpos.view(B, H_kv, cap).to(I32).to(DEV)
        self.dl = [i32([self.budget + g + 1] * B) for g in range(self.gamma)]
        self.at = [(self.lens + self.Lp + g).to(I32) for g in range(self.gamma)]
        self.total = (self.lens + self.Lp + self.gamma).to(I32)
        self.dq, self.dout = randn((self.gamma, B, 1, self.H_q, d), seed + 40), torch.empty((self.gamma, B, 1, self.H_q, d), dtype=BF16, device=DEV)
        self.dk, self.dv = randn((self.gamma, B, H_kv, d), seed + 41), randn((self.gamma, B, H_kv, d), seed + 42)
        self.left = torch.empty_like(self.lens)
        self.ws = torch.empty(mb.magicdec_prefix_attn_workspace_size(
            mb.paged_shape(B, self.H_q, H_kv, d, self.page, self.kp.shape[0], mp), 1, n), dtype=torch.uint8, device=DEV)

    def run(self, ws=None):
        for g in range(self.gamma):
            self.kc[:, :, self.budget + g], self.vc[:, :, self.budget + g] = self.dk[g], self.dv[g]
            mb.magicdec_heavy_attn(self.dq[g], self.kc, self.vc, self.weight, self.dl[g], pos=self.rpos, next_pos=self.at[g],
                                   out=self.dout[g])
        q, k, v = self.qkv.split([self.H_q, self.H_kv, self.H_kv], dim=2)
        mb.magicdec_norm_append(k, v, self.kp, self.vp, self.table, self.lens, self.inv, q=q, q_weight=self.qw,
                                k_weight=self.kw, pos=self.pos, q_out=self.q_out)
        mb.magicdec_prefix_attn(self.q_out, self.kp, self.vp, self.ptable, self.plen, self.table, self.lens, out=self.out,
                                ws=self.ws if ws is None else ws)
        mb.magicdec_heavy_evict(self.kc, self.vc, self.weight, self.rpos, self.dl[-1], self.total, self.budget, n_sink=2,
                                n_recent=8, draft_len_out=self.left)

    def results(self):
        return [self.kp, self.vp, self.q_out, self.out, self.kc, self.vc, self.weight, self.rpos, self.dout, self.left]


def test_a_whole_step():
    s = Step(1000)
    kc, vc, weight, rpos = (x.clone() for x in (s.kc, s.vc, s.weight, s.rpos))
    s.run()
    for g in range(s.gamma):
        kc[:, :, s.budget + g], vc[:, :, s.budget + g] = s.dk[g], s.dv[g]
        (ref, tol), (w, wt), rpos = heavy_ref(s.dq[g], kc, vc, weight, rpos, [s.budget + g + 1] * s.B, s.at[g].tolist())
        within(s.dout[g], ref, tol, f"draft {g}")
        weight = w
    host = [x.cpu()[None] for x in (kc, vc, weight, rpos)]
    *host, left = evict_ref(*host, [s.budget + s.gamma] * s.B, s.total.tolist(), s.budget, 2, 8)
    assert s.left.tolist() == left
    used = slice(0, s.budget)
    assert torch.equal(s.rpos[:, :, used].cpu(), host[3][0][:, :, used])
    assert torch.equal(s.kc[:, :, used].cpu(), host[0][0][:, :, used])
    assert (s.weight[:, :, used].cpu().double() - host[2][0][:, :, used]).abs().max() < 1e-4
    within(s.out, *prefix_ref(s.q_out, s.kp, s.vp, s.ptable, [s.Lp], [0, s.B], s.table, s.lens.tolist(), None, None))


def test_graphs_that_share_a_workspace_and_calls_at_once():
    """Two captured steps that share one workspace, replayed one after the other, twice; and two steps with
    workspaces of their own, on two streams at once."""
    want = [Step(2000), Step(3000)]
    for s in want:
        s.run()
    torch.cuda.synchronize()
    mine = [Step(2000), Step(3000)]
    start = [[x.clone() for x in s.results()] for s in mine]
    for s in mine:                                      # first passes outside of a capture
        s.run(mine[0].ws)
    torch.cuda.synchronize()
    graphs = []
    for s in mine:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run(mine[0].ws)
    for _ in range(2):
        for s, old in zip(mine, start):
            for x, y in zip(s.results(), old):
                x.copy_(y)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, t in zip(mine, want):
            for x, y in zip(s.results(), t.results()):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    apart, streams = [Step(2000), Step(3000)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, st in zip(apart, streams):
        with torch.cuda.stream(st):
            s.run()
    torch.cuda.synchronize()
    for s, t in zip(apart, want):
        for x, y in zip(s.results(), t.results()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_rows_past_32_bits():
    """The last sequence's rows lie past element 2^31 of the caches."""
    B, H_kv, d, cap, ln, budget = 17, 1, 128, 1 << 20, 300, 290
    kc, vc = (torch.empty((B, H_kv, cap, d), dtype=BF16, device=DEV) for _ in range(2))
    weight = torch.empty((B, H_kv, cap), dtype=torch.float32, device=DEV)
    pos = torch.empty((B, H_kv, cap), dtype=I32, device=DEV)
    lens, total = [0] * (B - 1) + [ln], [0] * (B - 1) + [900]
    for H_q, n in ((4, 1), (20, 1)):                    # both ways of the attention
        small = randn((1, H_kv, ln, d), 5), randn((1, H_kv, ln, d), 6)
        w0, p0 = torch.rand((1, H_kv, ln), generator=gen(7)).to(DEV), torch.arange(ln, device=DEV, dtype=I32).view(1, 1, ln)
        for x, y in zip((kc, vc, weight, pos), (*small, w0, p0)):
            x[-1:, :, :ln] = y
        q = randn((B, n, H_q, d), 8)
        got = mb.magicdec_heavy_attn(q, kc, vc, weight, i32(lens), pos=pos, next_pos=i32(total))
        (ref, tol), (w, wt), p = heavy_ref(q[-1:], *small, w0, p0.clone(), [ln], [900])
        within(got[-1:], ref, tol)
        assert (got[:-1] == 0).all()
        within(weight[-1:, :, :ln], w, wt)
        before = [x[-1:, :, :ln].cpu()[None] for x in (kc, vc, weight, pos)]
        mb.magicdec_heavy_evict(kc, vc, weight, pos, i32(lens), i32([x + 1 for x in total]), budget, n_sink=2, n_recent=20)
        after = evict_ref(*before, [ln], [901], budget, 2, 20)
        for x, y in zip((kc, vc, weight, pos), after):
            assert torch.equal(x[-1:, :, :ln].cpu(), y[0])


def test_pages_past_32_bits():
    page, H_kv, d, H_q, n = 64, 8, 128, 32, 2
    pages = (1 << 31) // (page * H_kv * d) + 40         # the last ones lie past element 2^31
    kp, vp = (torch.empty((pages, page, H_kv, d), dtype=BF16, device=DEV) for _ in range(2))
    used = torch.arange(pages - 32, pages, device=DEV)
    for x, seed in ((kp, 11), (vp, 12)):
        x[used] = randn((32, page, H_kv, d), seed)
    order = used[torch.randperm(32, generator=gen(13)).to(DEV)].to(I32)
    ptable, table = order[:20].view(1, 20).contiguous(), order[20:32].view(3, 4).contiguous()
    lens, plens = [100, 0, 254], [1270]
    k, v = randn((3, n, H_kv, d), 14), randn((3, n, H_kv, d), 15)
    mb.magicdec_norm_append(k, v, kp, vp, table, i32(lens), None)
    for b in range(3):
        rows = rows_of(table, b, lens[b] + torch.arange(n), page).to(DEV)
        assert torch.equal(kp.view(-1, H_kv, d)[rows], k[b]) and torch.equal(vp.view(-1, H_kv, d)[rows], v[b])
    base = pages - 32                                   # the reference looks at the used pages only
    for heads in (H_q, 20 * H_kv):                      # own slots with the prefix's parts, and in the list of work
        q = randn((3, n, heads, d), 16)
        got = mb.magicdec_prefix_attn(q, kp, vp, ptable, i32(plens), table, i32(lens))
        within(got, *prefix_ref(q, kp[used], vp[used], ptable - base, plens, [0, 3], table - base, lens, None, None))


CHILD = r"""
import json, sys, torch
sys.path[:0] = [sys.argv[1], sys.argv[2]]
from long_context_self_gb300 import binding as mb
dev = torch.device("cuda:0")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
rnd = lambda *s: torch.randn(s, generator=torch.Generator().manual_seed(sum(s))).to(torch.bfloat16).to(dev)
def word():
    return mb.magicdec_device_error()
res = {}
kp, vp = rnd(12, 16, 2, 64), rnd(12, 16, 2, 64)
table, ptable = i32([[0, 1], [2, 3]]), i32([[4, 5, 6]])
q, k = rnd(2, 2, 4, 64), rnd(2, 2, 2, 64)
inv = torch.ones(32, device=dev)
kc, vc, weight = rnd(2, 2, 20, 64), rnd(2, 2, 20, 64), torch.rand((2, 2, 20), device=dev)
pos = torch.arange(20, dtype=torch.int32, device=dev).expand(2, 2, 20).contiguous()
def append(axis):
    mb.magicdec_norm_append(k, k, kp.clone(), vp.clone(), table, i32([3, 4]), inv, pos=i32([[[1, 2]] * 2] * 2), axis=i32(axis))
def prefix(plen, first, lens, parent=None):
    mb.magicdec_prefix_attn(q, kp, vp, ptable, i32([plen]), table, i32(lens), first=i32(first), parent=parent)
def heavy(lens, heads=4):
    mb.magicdec_heavy_attn(rnd(2, 1, heads, 64), kc, vc, weight.clone(), i32(lens))
def evict(lens):
    mb.magicdec_heavy_evict(kc.clone(), vc.clone(), weight.clone(), pos.clone(), i32(lens), i32([30, 30]), 10)
for name, good, bad in (
        ("axis", lambda: append([0, 1] * 16), lambda: append([0, 2] * 16)),
        ("prefix_len", lambda: prefix(48, [0, 2], [3, 4]), lambda: prefix(49, [0, 2], [3, 4])),
        ("first", lambda: prefix(48, [0, 2], [3, 4]), lambda: prefix(48, [0, 3], [3, 4])),
        ("own", lambda: prefix(48, [0, 2], [3, 30]), lambda: prefix(48, [0, 2], [3, 33])),
        ("parent", lambda: prefix(48, [0, 2], [3, 4], i32([[-1, 0]] * 2)), lambda: prefix(48, [0, 2], [3, 4], i32([[-1, 1]] * 2))),
        ("draft_len", lambda: heavy([20, 0]), lambda: heavy([21, 0])),
        ("draft_len, more rows", lambda: heavy([20, 0], 24), lambda: heavy([20, -1], 24)),
        ("evicted", lambda: evict([20, 5]), lambda: evict([20, 21]))):
    good(); a = word(); bad(); res[name] = [a, word()]
print(json.dumps(res))
"""


@pytest.mark.parametrize("library,error", [("debug", 4), (None, 0)])
def test_the_range_checking_build_records_what_is_out_of_range(library, error):
    from long_context_self_gb300 import build
    build.build(debug=library == "debug")
    env = dict(os.environ)
    env.pop("MAGICDEC_LIBRARY", None)
    if library:
        env["MAGICDEC_LIBRARY"] = library
    r = subprocess.run([sys.executable, "-c", CHILD, os.path.dirname(HERE), HERE], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(res) == 8
    for name, words in res.items():
        assert words == [0, error], (name, words)
