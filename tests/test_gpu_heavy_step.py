"""Speculative steps over a heavy-hitter draft cache as the header describes them: rows appended and refreshed by
magicdec_draft_cache_update, attended, evicted; against the plain 64-bit forms."""
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


def randn(shape, seed):
    return torch.randn(shape, generator=gen(seed)).to(BF16).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=I32, device=DEV)


class Cache:
    """A layer's caches: verified and drafted K, V [B, L_cap, H_kv, d], and the draft cache.  What no call has
    written is far from any weight or position."""
    B, H_q, H_kv, d, L_cap, budget, gamma, sink, recent = 5, 8, 2, 64, 200, 24, 3, 2, 6

    def __init__(self):
        B, H_kv, d, cap = self.B, self.H_kv, self.d, self.budget + self.gamma + 1
        self.k, self.v = randn((B, self.L_cap, H_kv, d), 1), randn((B, self.L_cap, H_kv, d), 2)
        self.kd, self.vd = randn((B, self.L_cap, H_kv, d), 3), randn((B, self.L_cap, H_kv, d), 4)
        self.len, self.rows = i32([40, 31, 24, 24, 60]), i32([24, 20, 24, 5, 1])
        self.kc, self.vc = randn((B, H_kv, cap, d), 5), randn((B, H_kv, cap, d), 6)
        self.weight = torch.full((B, H_kv, cap), 1e6, device=DEV)
        self.pos = torch.full((B, H_kv, cap), 1 << 20, dtype=I32, device=DEV)
        for b in range(B):
            r = int(self.rows[b])
            self.weight[b, :, :r] = torch.rand((H_kv, r), generator=gen(7 + b)).to(DEV)
            for h in range(H_kv):
                self.pos[b, h, :r] = torch.randperm(int(self.len[b]), generator=gen(20 + 7 * b + h))[:r].to(I32).to(DEV)
        self.out = torch.empty((self.gamma, B, 1, self.H_q, d), dtype=BF16, device=DEV)
        self.dl, self.left = torch.empty_like(self.len), torch.empty_like(self.len)

    def step(self, q, n_acc):
        """Drafts gamma tokens, keeps n_acc [B] of them and the emitted one, evicts: the header's order of calls."""
        L, g = self.len, self.gamma
        new_len, table = mb.magicdec_step_lengths(L, g, self.L_cap)
        t = table.view(g + 2, self.B)
        for i in range(g):
            mb.magicdec_draft_cache_update(self.kd, self.vd, self.kc, self.vc, t[i], t[i], t[i + 1], L, self.rows, 0,
                                           draft_len=self.dl)
            mb.magicdec_heavy_attn(q[i], self.kc, self.vc, self.weight, self.dl, pos=self.pos, next_pos=t[i], out=self.out[i])
        # the row that the refresh brings in where every drafted token was accepted: no attention has set it
        at = (self.rows + g).long()[:, None, None].expand(self.B, self.H_kv, 1)
        self.weight.scatter_(2, at, 0.0)
        self.pos.scatter_(2, at, t[g][:, None, None].expand(self.B, self.H_kv, 1))
        new_len, _ = mb.magicdec_step_lengths(L, g, self.L_cap, n_acc=n_acc)
        mb.magicdec_draft_cache_update(self.k, self.v, self.kc, self.vc, t[0], t[g], new_len, L, self.rows, 0, draft_len=self.dl)
        mb.magicdec_heavy_evict(self.kc, self.vc, self.weight, self.pos, self.dl, new_len, self.budget, n_sink=self.sink,
                                n_recent=self.recent, draft_len_out=self.left)
        self.len, self.rows = new_len, self.left.clone()


def test_steps_of_appends_refreshes_and_evictions():
    """Between none and all of the drafted tokens accepted: the cache's rows, positions and weights are those of the
    plain form; a rejected token's row goes, what it gave to other rows' weights stays."""
    c = Cache()
    w, p = c.weight.double(), c.pos.clone()
    kc, vc = c.kc.clone(), c.vc.clone()
    rows, L = c.rows.tolist(), c.len.tolist()
    for step in range(12):
        q = randn((c.gamma, c.B, 1, c.H_q, c.d), 100 + step)
        n_acc = [(b + step) % (c.gamma + 1) for b in range(c.B)]
        c.step(q, i32(n_acc))
        for g in range(c.gamma):
            for b in range(c.B):
                kc[b, :, rows[b] + g], vc[b, :, rows[b] + g] = c.kd[b, L[b] + g], c.vd[b, L[b] + g]
            (ref, tol), (w, _), p = heavy_ref(q[g], kc, vc, w, p, [r + g + 1 for r in rows], [x + g for x in L])
            assert ((c.out[g].double() - ref).abs() <= tol).all()
        for b in range(c.B):
            for j in range(n_acc[b] + 1):
                kc[b, :, rows[b] + j], vc[b, :, rows[b] + j] = c.k[b, L[b] + j], c.v[b, L[b] + j]
            if n_acc[b] == c.gamma:
                w[b, :, rows[b] + c.gamma], p[b, :, rows[b] + c.gamma] = 0.0, L[b] + c.gamma
        L = [x + a + 1 for x, a in zip(L, n_acc)]
        *host, rows = evict_ref(*(x.cpu()[None] for x in (kc, vc, w, p)), [r + a + 1 for r, a in zip(rows, n_acc)], L,
                                c.budget, c.sink, c.recent)
        kc, vc, w, p = (x[0].to(DEV) for x in host)
        assert c.rows.tolist() == rows and c.len.tolist() == L
        for b, r in enumerate(rows):
            assert torch.equal(c.pos[b, :, :r], p[b, :, :r]), (step, b)
            assert torch.equal(c.kc[b, :, :r], kc[b, :, :r]) and torch.equal(c.vc[b, :, :r], vc[b, :, :r])
            # sums of some 40 probabilities in fp32, each off by 2^-12 of itself at most
            assert (c.weight[b, :, :r].double() - w[b, :, :r]).abs().max() < 40 * 4 * 2.0 ** -12
            assert int(c.pos[b, :, :r].max()) < L[b]
            assert all(c.pos[b, h, :r].unique().numel() == r for h in range(c.H_kv))
