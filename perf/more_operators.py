"""Workloads of the operators for batches behind a shared prompt and for a heavy-hitter draft cache.

Four operators: appending normed and rotated heads to a paged cache ("append"),
attention of a batch whose sequences share long prefixes ("prefix"), attention
over a compact draft cache that adds every row's attention weight up ("heavy"),
and eviction of the rows of least weight ("evict").  `run` computes each in
elementary torch operations where `own` is false and through
long_context_self_gb300.binding where it is true; `exact` gives the 64-bit values.

Paged cache, as in operators.py: a pool [n_pages, page, H_kv, d], a block table
[B, max_pages] of every sequence's own pages and one [P, max_prefix_pages] of the
prefixes'; own slots are counted from 0 behind the prefix.  Draft cache: rows
[B, H_kv, cap, d] in any order, of each its weight and its position.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one sequence: the latency of a decode step's append
        dict(name="append_token_b1", op="append", B=1, n=1, Hq=32, Hkv=8, d=128, rot=128, inter=False, tree=False,
             axes=0, ragged=False, L=2000, page=16),
        # every node of the drafted trees of a full batch, one layer
        dict(name="append_tree_b128", op="append", B=128, n=32, Hq=32, Hkv=8, d=128, rot=128, inter=False, tree=True,
             axes=0, ragged=False, L=4000, page=16),
        # ragged prompts with images at prefill: positions of three axes
        dict(name="append_images_b4", op="append", B=4, n=8001, Hq=40, Hkv=8, d=128, rot=128, inter=False, tree=False,
             axes=3, ragged=True, L=517, page=64),
        # one token each of a few samples of one prompt: the single-token form, where latency counts
        dict(name="prefix_token_b8_l4k", op="prefix", B=8, n=1, P=1, Hq=32, Hkv=8, d=128, Lp=4000, L=60, page=16,
             branch=0, ragged=False),
        # one token of a full batch behind a 32k prompt: reading and products weigh about the same
        dict(name="prefix_token_b128_l32k", op="prefix", B=128, n=1, P=1, Hq=32, Hkv=8, d=128, Lp=32000, L=500,
             page=16, branch=0, ragged=False),
        # verification of drafted trees behind a 32k prompt: bound by the products
        dict(name="prefix_tree8_b128_l32k", op="prefix", B=128, n=8, P=1, Hq=32, Hkv=8, d=128, Lp=32000, L=300,
             page=64, branch=2, ragged=False),
        # several prompts with their samples, uneven lengths, odd group and page sizes, 64 channels
        dict(name="prefix_groups_b40_d64", op="prefix", B=40, n=5, P=7, Hq=24, Hkv=8, d=64, Lp=9001, L=701, page=48,
             branch=2, ragged=True),
        # one drafted token of one sequence over a 512-row draft cache
        dict(name="heavy_token_b1", op="heavy", B=1, n=1, Hq=32, Hkv=8, d=128, L=517, cap=528, ragged=False),
        # one drafted token of a full batch over 2k rows
        dict(name="heavy_token_b128_l2k", op="heavy", B=128, n=1, Hq=32, Hkv=8, d=128, L=2053, cap=2064,
             ragged=False),
        # a block of five tokens, five query heads a KV head, uneven lengths
        dict(name="heavy_block5_b16_l12k", op="heavy", B=16, n=5, Hq=40, Hkv=8, d=128, L=12001, cap=12001,
             ragged=True),
        # one row of one layer's cache after a token
        dict(name="evict_one_b1", op="evict", layers=1, B=1, Hkv=8, d=128, budget=512, more=1, cap=528, sink=4,
             recent=64, ragged=False),
        # the rows of a speculative step in every layer
        dict(name="evict_step_b16_layers32", op="evict", layers=32, B=16, Hkv=8, d=128, budget=1024, more=5, cap=1040,
             sink=16, recent=256, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "prefix", "prefix", "heavy", "heavy", "evict"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    d = rng.choice([64, 128, 128])
    Hkv, G = rng.choice([(8, 4), (8, 5), (4, 7), (8, 1), (2, 8), (1, 16), (5, 3)])
    ragged = rng.random() < 0.5
    if op == "append":
        axes = rng.choice([0, 0, 1, 2, 3])
        tree = axes == 0 and rng.random() < 0.6
        n = _log(rng, 1, 200) if tree else _log(rng, 1, 6000)
        B = _log(rng, 1, max(1, min(128, 24000 // n)))
        return dict(op=op, B=B, n=n, Hq=Hkv * G, Hkv=Hkv, d=d, rot=rng.choice([d, d // 2]), inter=rng.random() < 0.5,
                    tree=tree, axes=axes, ragged=ragged, L=_log(rng, 1, 5000), page=page)
    if op == "prefix":
        n = _log(rng, 1, 40)
        B = _log(rng, 1, 128)
        Lp = _log(rng, 1, max(2, min(60000, int(1.0e9 / (B * n * Hkv * G)))))
        L = _log(rng, 1, max(2, min(2000, int(2.0e5 / B))))
        return dict(op=op, B=B, n=n, P=_log(rng, 1, min(B, 8)), Hq=Hkv * G, Hkv=Hkv, d=d, Lp=Lp, L=L, page=page,
                    branch=rng.choice([0, 2, 3]), ragged=ragged)
    if op == "heavy":
        n = rng.randint(1, max(1, min(8, 32 // G)))
        L = _log(rng, 1, 12000)
        B = _log(rng, 1, max(1, min(128, int(2.4e6 / (L * Hkv)))))
        return dict(op=op, B=B, n=n, Hq=Hkv * G, Hkv=Hkv, d=d, L=L, cap=L + rng.randint(0, 40), ragged=ragged)
    budget = _log(rng, 2, 4000)
    more = _log(rng, 1, 300)
    layers = _log(rng, 1, 32)
    B = _log(rng, 1, max(1, min(64, int(3.0e6 / ((budget + more) * layers * Hkv)))))
    sink = rng.randint(0, min(16, budget // 2))
    return dict(op=op, layers=layers, B=B, Hkv=Hkv, d=d, budget=budget, more=more,
                cap=budget + more + rng.randint(0, 40), sink=sink, recent=rng.randint(0, budget - sink), ragged=ragged)


# Lengths, counts and groups follow from the case alone, so that work() can count them.
def _spread(B, most, least, k):
    """B whole numbers in [least, most], the first of them `most`."""
    return [most if b == 0 else least + int((most - least) * ((b * k) % 1.0)) for b in range(B)]


def _lens(c):
    least = c["n"] if c["op"] == "heavy" else 0
    return _spread(c["B"], c["L"], min(least, c["L"]), 0.618034) if c["ragged"] else [c["L"]] * c["B"]


def _counts(c):
    return _spread(c["B"], c["n"], 0, 0.414214) if c["ragged"] else [c["n"]] * c["B"]


def _plens(c):
    return _spread(c["P"], c["Lp"], 0, 0.732051) if c["ragged"] else [c["Lp"]] * c["P"]


def _first(c):
    """The first sequence of every group, and the end of the last: cuts at uneven places."""
    B, P = c["B"], c["P"]
    return [min(B, int(B * (g / P) ** 1.3)) for g in range(P)] + [B]


def _rows_in(c):
    """Rows of the draft caches before the eviction."""
    most = c["budget"] + c["more"]
    return _spread(c["B"], most, max(0, c["budget"] - c["more"] // 4), 0.618034) if c["ragged"] else [most] * c["B"]


def _parents(B, n, branch, g, dev):
    """Parents in level order.  branch 0: a chain; otherwise node i hangs, at random, from the
    node that a complete tree of that branching gives it or from an earlier one."""
    i = torch.arange(n, device=dev)
    if branch == 0:
        return (i - 1).to(I32).expand(B, n).contiguous()
    p = (i - 1).clamp(min=0) // branch
    back = (torch.rand((B, n), generator=g, device=dev) < 0.2).long()
    p = torch.minimum((p[None] - back).clamp(min=0), (i - 1).clamp(min=0)[None])
    p[:, 0] = -1
    return p.to(I32)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(c)
    i32 = lambda x: torch.tensor(x, dtype=I32, device=dev)  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=BF16)  # noqa: E731
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] in ("append", "prefix"):
        n, page = c["n"], c["page"]
        mp = -(-(c["L"] + n) // page)
        pp = -(-c["Lp"] // page) if c["op"] == "prefix" else 0
        P = c["P"] if c["op"] == "prefix" else 0
        pages = B * mp + P * pp + 3
        perm = torch.randperm(pages, generator=g, device=dev).to(I32)
        s["table"] = perm[: B * mp].view(B, mp)
        s["kp"], s["vp"] = randn(pages, page, Hkv, d), randn(pages, page, Hkv, d)
        s["len"], s["count"] = i32(_lens(c)), i32(_counts(c)) if c["ragged"] else None
    if c["op"] == "append":
        # one projection's output holds a token's queries, keys and values side by side
        qkv = randn(B, n, c["Hq"] + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], Hkv, Hkv], dim=2)
        s["qw"], s["kw"] = ((1.0 + 0.3 * randn(d).float()).to(BF16) for _ in range(2))
        s["parent"] = _parents(B, n, 2, g, dev) if c["tree"] else None
        base = 500000.0 * (1.0 + 0.1 * float(torch.rand((), generator=g, device=dev)))
        s["inv_freq"] = (base ** (-torch.arange(0, c["rot"], 2, dtype=F64, device=dev) / c["rot"])).to(F32)
        s["pos"] = s["axis"] = None
        if c["axes"]:
            # text counts on all axes alike; of an image's patches each axis counts its own
            i = torch.arange(n, device=dev)
            img = (i // 1024) % 2 == 1
            grid = torch.stack([torch.zeros_like(i), (i % 1024) // 32, i % 32], -1)[:, : c["axes"]]
            at = torch.where(img[:, None], (i // 1024 * 1024)[:, None] + grid, i[:, None])
            s["pos"] = (s["len"].long()[:, None, None] + at).to(I32).contiguous()
            s["axis"] = (torch.arange(c["rot"] // 2, device=dev) * c["axes"] // (c["rot"] // 2)).to(I32)
        s["q_out"] = torch.zeros((B, n, c["Hq"], d), dtype=BF16, device=dev)
    elif c["op"] == "prefix":
        s["ptable"] = perm[B * mp: B * mp + P * pp].view(P, pp)
        # one position in a hundred draws much of the attention
        big = torch.rand(s["kp"].shape[:3], generator=g, device=dev) < 0.01
        s["kp"].mul_(torch.where(big, 4.0, 1.0).to(BF16)[..., None])
        s["q"] = randn(B, n, c["Hq"], d)
        s["plen"], s["first"] = i32(_plens(c)), i32(_first(c)) if P > 1 else None
        s["parent"] = _parents(B, n, c["branch"], g, dev)
        s["out"] = torch.empty_like(s["q"])
    else:
        lead = (c["layers"], B) if c["op"] == "evict" else (B,)
        cap = c["cap"]
        s["kc"], s["vc"] = randn(*lead, Hkv, cap, d), randn(*lead, Hkv, cap, d)
        rows = _lens(c) if c["op"] == "heavy" else _rows_in(c)
        s["len"] = i32(rows)
        # a few rows hold most of the weight, as accumulated attention has it
        s["weight"] = torch.rand((*lead, Hkv, cap), generator=g, device=dev).pow_(8.0).mul_(20.0)
        # positions of a sequence of 4 times the rows, distinct, in the order that evictions leave
        s["total"] = i32([4 * r for r in rows])
        live = torch.arange(cap, device=dev) < s["len"][:, None, None]
        u = torch.rand((*lead, Hkv, cap), generator=g, device=dev).masked_fill_(~live, 2.0)
        # ranks of the live rows, spread over the positions
        rank = u.argsort(-1).argsort(-1)
        s["pos"] = torch.where(live, rank * 4 + (rank % 4), -1).to(I32).contiguous()
        if c["op"] == "heavy":
            big = torch.rand((B, Hkv, cap), generator=g, device=dev) < 0.01
            s["kc"].mul_(torch.where(big, 4.0, 1.0).to(BF16)[..., None])
            s["q"] = randn(B, c["n"], c["Hq"], d)
            s["out"] = torch.empty_like(s["q"])
        else:
            s["len_out"] = torch.empty_like(s["len"])
    return s


# ------------------------------------------------------------------------- run
def run(state):
    if own:
        return _kernels(state)
    return {"append": _append, "prefix": _prefix, "heavy": _heavy, "evict": _evict}[state["op"]](state)


def _kernels(s):
    from long_context_self_gb300 import binding as mb

    if s["op"] == "append":
        mb.magicdec_norm_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["len"], s["inv_freq"], q=s["q"],
                                q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, n_new=s["count"], parent=s["parent"],
                                pos=s["pos"], axis=s["axis"], interleaved=s["inter"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}
    if s["op"] == "prefix":
        return mb.magicdec_prefix_attn(s["q"], s["kp"], s["vp"], s["ptable"], s["plen"], s["table"], s["len"],
                                       first=s["first"], parent=s["parent"], n_nodes=s["count"], out=s["out"])
    if s["op"] == "heavy":
        mb.magicdec_heavy_attn(s["q"], s["kc"], s["vc"], s["weight"], s["len"], pos=s["pos"], next_pos=s["total"],
                               out=s["out"])
        return {"out": s["out"], "weight": s["weight"], "pos": s["pos"]}
    mb.magicdec_heavy_evict(s["kc"], s["vc"], s["weight"], s["pos"], s["len"], s["total"], s["budget"],
                            n_sink=s["sink"], n_recent=s["recent"], draft_len_out=s["len_out"])
    return {"k": s["kc"], "v": s["vc"], "weight": s["weight"], "pos": s["pos"], "len": s["len_out"]}


# -------------------------------------------------------------- the plain form
def _closure(parent):
    """[B, n, n] truth: node j is node i or one of those before it.  With P the 0/1 matrix that
    takes a node to its parent, the closure is I + P + P^2 + ... = (I - P)^-1."""
    B, n = parent.shape
    eye = torch.eye(n, dtype=F32, device=parent.device)
    P = (parent[:, :, None] == torch.arange(n, device=parent.device)).to(F32)
    return torch.linalg.solve_triangular(eye - P, eye.expand(B, n, n), upper=False, unitriangular=True) > 0.5


def _rows(table, pos, page):
    """Pool rows (page * page size + offset) of positions pos [B, m]."""
    return table.long().gather(1, pos // page) * page + pos % page


def _append(s):
    B, n, d, rot = s["B"], s["n"], s["d"], s["rot"]
    dev = s["k"].device
    i = torch.arange(n, device=dev)
    if s["pos"] is not None:
        at = s["pos"].long()[:, :, s["axis"].long()]
    else:
        depth = i.expand(B, n) if s["parent"] is None else _closure(s["parent"]).sum(-1) - 1
        at = (s["len"].long()[:, None] + depth)[..., None]
    ang = at.to(F64) * s["inv_freq"].to(F64)
    cos, sin = ang.cos().to(F32)[:, :, None], ang.sin().to(F32)[:, :, None]

    def turn(x, w):
        x = x.to(F32)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(F32)
        y = x[..., :rot]
        if s["inter"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., : rot // 2], y[..., rot // 2:]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((y, x[..., rot:]), -1).to(BF16)

    live = torch.ones((B, n), dtype=torch.bool, device=dev) if s["count"] is None else i[None] < s["count"][:, None]
    at = _rows(s["table"], s["len"].long()[:, None] + i, s["page"])[live]
    s["kp"].view(-1, s["Hkv"], d)[at] = turn(s["k"], s["kw"])[live]
    s["vp"].view(-1, s["Hkv"], d)[at] = s["v"][live]
    s["q_out"][live] = turn(s["q"], s["qw"])[live]
    return {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}


def _prefix(s):
    B, n, P, Hkv, d, page = s["B"], s["n"], s["P"], s["Hkv"], s["d"], s["page"]
    G, cap, Lp = s["Hq"] // Hkv, s["L"] + n, s["Lp"]
    dev = s["q"].device
    root = 1.0 / math.sqrt(d)
    count = torch.full((B, 1), n, device=dev) if s["count"] is None else s["count"].long()[:, None]
    # The prefixes: the groups' rows side by side, [P, Hkv, m * n * G, Lp].
    first = torch.tensor([0, B], device=dev) if s["first"] is None else s["first"].long()
    m = max(y - x for x, y in zip(_first(s), _first(s)[1:]))
    who = first[:-1, None] + torch.arange(m, device=dev)                     # [P, m]: sequences of a group
    mine = who < first[1:, None]
    who = who.clamp(max=B - 1)
    pos = torch.arange(Lp, device=dev).expand(P, Lp)
    at = _rows(s["ptable"], pos, page)
    q = s["q"].to(F32).view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4)          # [B, Hkv, n, G, d]
    qg = q[who].permute(0, 2, 1, 3, 4, 5).reshape(P, Hkv, m * n * G, d)
    x = torch.matmul(qg, s["kp"].view(-1, Hkv, d)[at].to(F32).permute(0, 2, 3, 1)).mul_(root)
    x.masked_fill_((pos >= s["plen"][:, None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, s["vp"].view(-1, Hkv, d)[at].to(F32).permute(0, 2, 1, 3))
    del x

    def back(y):                                                             # to [B, Hkv, n * G, ...]
        y = y.view(P, Hkv, m, n * G, y.shape[-1]).permute(0, 2, 1, 3, 4)[mine]
        full = torch.zeros((B,) + y.shape[1:], dtype=F32, device=dev)
        full[who[mine]] = y
        return full

    o1, l1 = back(o), back(total)
    m1 = torch.where(l1 > 0, back(torch.where(top == -math.inf, 0.0, top)), -math.inf)
    # The sequences' own slots.
    length = s["len"].long()[:, None]
    pos = torch.arange(cap, device=dev).expand(B, cap)
    at = _rows(s["table"], pos, page)
    node = pos - length
    live = node < count
    i = torch.arange(n, device=dev)
    seen = _closure(s["parent"]).gather(2, node.clamp(0, n - 1)[:, None].expand(B, n, cap)) & (node >= 0)[:, None]
    seen = (seen | (node < 0)[:, None]) & live[:, None] & (i[None] < count)[:, :, None]
    x = torch.matmul(q.reshape(B, Hkv, n * G, d), s["kp"].view(-1, Hkv, d)[at].to(F32).permute(0, 2, 3, 1)).mul_(root)
    x = x.view(B, Hkv, n, G, cap).masked_fill_(~seen[:, None, :, None], -math.inf).view(B, Hkv, n * G, cap)
    m2 = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m2 == -math.inf, 0.0, m2)).exp_()
    v = s["vp"].view(-1, Hkv, d)[at].to(F32).masked_fill_(~live[..., None, None], 0.0).permute(0, 2, 1, 3)
    o2, l2 = torch.matmul(x, v), x.sum(-1, keepdim=True)
    top = torch.maximum(m1, m2)
    top = torch.where(top == -math.inf, 0.0, top)
    w1, w2 = (m1 - top).exp(), (m2 - top).exp()
    total = w1 * l1 + w2 * l2
    o = torch.where(total > 0, (w1 * o1 + w2 * o2) / total, 0.0).view(B, Hkv, n, G, d)
    o = torch.where((i < count)[:, None, :, None, None], o, 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, s["Hq"], d).to(BF16)


def _heavy(s):
    B, n, Hkv, d, cap = s["B"], s["n"], s["Hkv"], s["d"], s["cap"]
    G = s["Hq"] // Hkv
    dev = s["q"].device
    row = torch.arange(cap, device=dev)
    length = s["len"].long()[:, None, None]
    new = (row >= length - n) & (row < length)                               # [B, 1, cap]: the block's own rows
    place = s["total"].long()[:, None, None] + row - (length - n)
    s["pos"].copy_(torch.where(new, place, s["pos"]))
    s["weight"].masked_fill_(new, 0.0)
    q = s["q"].to(F32).view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    x = torch.matmul(q, s["kc"].to(F32).transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, n, G, cap)
    i = torch.arange(n, device=dev)[:, None]
    x.masked_fill_((row >= length - n + 1 + i)[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    x.copy_(torch.where(total > 0, x / total, 0.0))
    s["weight"].add_(x.sum((2, 3)))
    v = s["vc"].to(F32).masked_fill_((row >= length)[..., None], 0.0)
    o = torch.matmul(x.view(B, Hkv, n * G, cap), v).view(B, Hkv, n, G, d).permute(0, 2, 1, 3, 4)
    return {"out": o.reshape(B, n, s["Hq"], d).to(BF16), "weight": s["weight"], "pos": s["pos"]}


def _evict(s):
    cap, budget = s["cap"], s["budget"]
    row = torch.arange(cap, device=s["kc"].device)
    length = s["len"].long()[:, None, None]                                  # [B, 1, 1], under the layers
    total = s["total"].long()[:, None, None]
    live = row < length
    pos, weight = s["pos"].long(), s["weight"]
    safe = (pos < s["sink"]) | (pos >= total - s["recent"])
    key = torch.where(live, torch.where(safe, math.inf, weight), -1.0)
    # by falling weight, then rising position, then rising row: three stable sorts
    order = pos.sort(dim=-1, stable=True).indices
    order = order.gather(-1, key.gather(-1, order).sort(dim=-1, descending=True, stable=True).indices)
    keep = torch.zeros_like(live.expand_as(pos)).scatter_(-1, order, (row < budget).expand_as(pos)) & live
    # kept rows at or past the budget, ascending, into the rows below it that were not kept
    hole = live & ~keep & (row < budget)
    late = keep & (row >= budget)
    where = (~hole).to(torch.int8).sort(dim=-1, stable=True).indices
    come = (~late).to(torch.int8).sort(dim=-1, stable=True).indices
    moves = row < late.sum(-1, keepdim=True)
    lead = torch.arange(pos[..., 0].numel(), device=pos.device).view(*pos.shape[:-1], 1).expand_as(pos)[moves]
    dst, src = lead * cap + where[moves], lead * cap + come[moves]
    for name in ("kc", "vc", "weight", "pos"):
        x = s[name].view(-1, s["d"]) if name in ("kc", "vc") else s[name].view(-1)
        x[dst] = x[src]
    s["len_out"].copy_(s["len"].clamp(max=budget))
    return {"k": s["kc"], "v": s["vc"], "weight": s["weight"], "pos": s["pos"], "len": s["len_out"]}


# ------------------------------------------------------------------------ work
def work(case):
    c = case
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "append":
        tokens = sum(_counts(c))
        return {"bytes": tokens * (4.0 * (c["Hq"] + 2 * Hkv) * d + 4.0 * c["axes"]) + 8.0 * B + 4.0 * B * c["n"] * c["tree"],
                "flops": tokens * (c["Hq"] + Hkv) * (4.0 * d + 3.0 * c["rot"])}
    if c["op"] == "prefix":
        first, n = _first(c), c["n"]
        counts, lens, plens = _counts(c), _lens(c), _plens(c)
        groups = [(plens[g], sum(counts[first[g]:first[g + 1]])) for g in range(c["P"])]
        kv = sum(p for p, m in groups if m) + sum(ln + m for ln, m in zip(lens, counts) if m)
        pairs = sum(p * m for p, m in groups)
        pairs += sum(m * ln + m * (m + 1) / 2 if c["branch"] == 0 else m * (ln + 1) for ln, m in zip(lens, counts))
        return {"bytes": 4.0 * kv * Hkv * d + 2.0 * (sum(counts) + B * n) * c["Hq"] * d + 8.0 * B,
                "flops": 4.0 * pairs * c["Hq"] * d}
    if c["op"] == "heavy":
        rows = sum(_lens(c))
        return {"bytes": rows * Hkv * (4.0 * d + 8.0) + 4.0 * B * c["n"] * c["Hq"] * d,
                "flops": 4.0 * rows * c["n"] * c["Hq"] * d}
    rows = _rows_in(c)
    moved = sum(max(0, r - c["budget"]) for r in rows)
    return {"bytes": c["layers"] * Hkv * (8.0 * sum(r for r in rows if r > c["budget"]) + moved * (8.0 * d + 16.0)) + 12.0 * B,
            "flops": 0.0}


# ----------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "prefix": _exact_prefix, "heavy": _exact_heavy, "evict": _exact_evict}[s["op"]](s)


def _ancestors(parent, i):
    got = []
    while i >= 0:
        got.append(i)
        i = parent[i]
    return got


def _exact_append(s):
    B, rot = s["B"], s["rot"]
    lens, counts = _lens(s), _counts(s)
    out = {"q": s["q_out"].double(), "k": s["kp"].double(), "v": s["vp"].double()}
    table, f = s["table"].long().cpu(), s["inv_freq"].double().cpu()
    par = s["parent"].tolist() if s["parent"] is not None else None
    half = torch.arange(rot // 2)
    first, second = (2 * half, 2 * half + 1) if s["inter"] else (half, half + rot // 2)
    for b in range(B):
        m = counts[b]
        if m == 0:
            continue
        slots = torch.arange(lens[b], lens[b] + m)
        pg, row = table[b, slots // s["page"]], slots % s["page"]
        if s["pos"] is not None:
            w = s["pos"][b, :m].double().cpu()[:, s["axis"].long().cpu()] * f
        elif par is not None:
            w = torch.outer(torch.tensor([lens[b] + len(_ancestors(par[b], i)) - 1 for i in range(m)]).double(), f)
        else:
            w = torch.outer(slots.double(), f)
        turn = torch.polar(torch.ones_like(w), w).to(s["k"].device)
        for name, x, g in (("q", s["q"], s["qw"]), ("k", s["k"], s["kw"])):
            y = x[b, :m].double()
            y = y / (y.square().sum(-1, keepdim=True) / s["d"] + 1e-6).sqrt() * g.double()
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            if name == "q":
                out["q"][b, :m] = y
            else:
                out["k"][pg, row] = y
        out["v"][pg, row] = s["v"][b, :m].double()
    return out


def _exact_prefix(s):
    B, n, Hkv, d, page = s["B"], s["n"], s["Hkv"], s["d"], s["page"]
    G = s["Hq"] // Hkv
    lens, counts, plens, first, par = _lens(s), _counts(s), _plens(s), _first(s), s["parent"].tolist()
    group = [sum(b >= x for x in first[1:-1]) for b in range(B)]
    # empty groups begin where the next does: the last that begins at or before b is its own
    if sum(plens[group[b]] + lens[b] for b in range(B)) * n * s["Hq"] * d > 1.2e12:
        return None
    out = torch.zeros((B, n, s["Hq"], d), dtype=F64, device=s["q"].device)
    for b in range(B):
        lp, ln, m = plens[group[b]], lens[b], counts[b]
        if m == 0:
            continue
        own_pages = s["table"][b, : -(-(ln + m) // page)].long()
        pre_pages = s["ptable"][group[b], : -(-lp // page)].long()
        k, v = (torch.cat((x[pre_pages].flatten(0, 1)[:lp], x[own_pages].flatten(0, 1)[: ln + m])).double()
                .transpose(0, 1) for x in (s["kp"], s["vp"]))
        see = torch.zeros((m, lp + ln + m), dtype=torch.bool)
        see[:, : lp + ln] = True
        for i in range(m):
            see[i, [lp + ln + j for j in _ancestors(par[b], i)]] = True
        see = see.to(k.device)[:, None]
        for h in range(Hkv):
            q = s["q"][b, :m, h * G:(h + 1) * G].double()
            w = (q.reshape(m * G, d) @ k[h].T / math.sqrt(d)).view(m, G, lp + ln + m)
            w = torch.where(see, w, -math.inf).softmax(-1)
            out[b, :m, h * G:(h + 1) * G] = (w.view(m * G, lp + ln + m) @ v[h]).view(m, G, d)
    return out


def _exact_heavy(s):
    B, n, Hkv, d = s["B"], s["n"], s["Hkv"], s["d"]
    G = s["Hq"] // Hkv
    out = torch.zeros((B, n, s["Hq"], d), dtype=F64, device=s["q"].device)
    weight, pos = s["weight"].double(), s["pos"].clone()
    for b, ln in enumerate(_lens(s)):
        at = max(0, ln - n)
        weight[b, :, at:ln] = 0.0
        pos[b, :, at:ln] = torch.arange(at - (ln - n), n, device=pos.device) + 4 * ln
        for i in range(n):
            e = ln - n + 1 + i                                               # rows that token i sees
            if e <= 0:
                continue
            q = s["q"][b, i].double().view(Hkv, G, d)
            w = torch.einsum("hgd,hed->hge", q, s["kc"][b, :, :e].double()).div(math.sqrt(d)).softmax(-1)
            out[b, i] = torch.einsum("hge,hed->hgd", w, s["vc"][b, :, :e].double()).reshape(s["Hq"], d)
            weight[b, :, :e] += w.sum(1)
    return {"out": out, "weight": weight, "pos": pos}


def _exact_evict(s):
    out = {"k": s["kc"].double(), "v": s["vc"].double(), "weight": s["weight"].double(), "pos": s["pos"].clone(),
           "len": s["len"].clamp(max=s["budget"])}
    at, frm = [], []
    cap = s["cap"]
    weight, pos = s["weight"].cpu().flatten(0, 1).tolist(), s["pos"].cpu().flatten(0, 1).tolist()
    for lb in range(s["layers"] * s["B"]):
        r = _rows_in(s)[lb % s["B"]]
        if r <= s["budget"]:
            continue
        for h in range(s["Hkv"]):
            w, p = weight[lb][h], pos[lb][h]
            safe = {j for j in range(r) if p[j] < s["sink"] or p[j] >= 4 * r - s["recent"]}
            rest = sorted((j for j in range(r) if j not in safe), key=lambda j: (-w[j], p[j], j))
            kept = safe | set(rest[: s["budget"] - len(safe)])
            base = (lb * s["Hkv"] + h) * cap
            at += [base + j for j in range(s["budget"]) if j not in kept]
            frm += [base + j for j in range(s["budget"], r) if j in kept]
    at, frm = torch.tensor(at, dtype=torch.long), torch.tensor(frm, dtype=torch.long)
    for name in ("k", "v", "weight", "pos"):
        x = out[name].view(-1, s["d"]) if name in ("k", "v") else out[name].view(-1)
        x[at.to(x.device)] = x[frm.to(x.device)]
    return out
