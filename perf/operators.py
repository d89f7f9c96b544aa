"""Workloads of the tree-speculation operators over a paged KV cache.

Four operators: appending rotated keys and values to a paged cache ("append"),
attention of a tree of drafted tokens over that cache ("attn"), greedy
acceptance down the tree ("accept") and moving the accepted rows to their
final slots ("commit").  `run` computes each in elementary torch operations
where `own` is false and through long_context_self_gb300.binding where it is
true; `exact` gives the 64-bit values.

Shapes, shared by all cases: a sequence b has `len[b]` committed positions; its
drafted node i sits at slot len[b] + i; node 0 is the root (the last emitted
token); parent[b, i] < i names the node before it.  Pages: a pool
[n_pages, page, H_kv, d] and a block table [B, max_pages].
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
             ragged=False, L=2000, page=16),
        # every node of the drafted trees of a full batch, one layer
        dict(name="append_tree_b128", op="append", B=128, n=32, Hq=32, Hkv=8, d=128, rot=128, inter=False, tree=True,
             ragged=False, L=4000, page=16),
        # ragged prompts at prefill, half of each head rotated, pairs interleaved
        dict(name="append_prompt_b4", op="append", B=4, n=8001, Hq=40, Hkv=8, d=128, rot=64, inter=True, tree=False,
             ragged=True, L=517, page=64),
        # one token of one short sequence: the single-token form, where latency counts
        dict(name="attn_token_b1", op="attn", B=1, n=1, Hq=32, Hkv=8, d=128, L=2000, page=16, branch=0, ragged=False),
        # a small tree over a long context: bound by reading the cache
        dict(name="attn_tree8_b16_l100k", op="attn", B=16, n=8, Hq=40, Hkv=8, d=128, L=99991, page=64, branch=2,
             ragged=False),
        # a wide tree over the 32k context: reading and products weigh about the same
        dict(name="attn_tree64_b32_l32k", op="attn", B=32, n=64, Hq=32, Hkv=8, d=128, L=32000, page=16, branch=3,
             ragged=False),
        # uneven batch, odd group and page sizes, 64 channels, trees of different sizes
        dict(name="attn_ragged_b24_d64", op="attn", B=24, n=13, Hq=24, Hkv=8, d=64, L=9001, page=48, branch=2,
             ragged=True),
        # a long linear block: more rows than one verification call of n_q tokens takes
        dict(name="attn_chain200_b8_l8k", op="attn", B=8, n=200, Hq=32, Hkv=8, d=128, L=8000, page=256, branch=0,
             ragged=False),
        # one sequence's tree over the largest vocabulary here
        dict(name="accept_b1", op="accept", B=1, n=40, V=152064, branch=3, acc=3),
        # a full batch
        dict(name="accept_b128", op="accept", B=128, n=32, V=128256, branch=2, acc=4),
        # one layer, one sequence
        dict(name="commit_b1", op="commit", layers=1, B=1, n=32, Hkv=8, d=128, L=2000, page=16, acc=4),
        # every layer of a full batch
        dict(name="commit_b128_layers32", op="commit", layers=32, B=128, n=32, Hkv=8, d=128, L=90, page=16, acc=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "accept", "commit"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    d = rng.choice([64, 128, 128])
    Hkv, G = rng.choice([(8, 4), (8, 5), (4, 7), (8, 1), (2, 8), (1, 16), (5, 3)])
    if op == "append":
        tree = rng.random() < 0.6
        n = _log(rng, 1, 200) if tree else _log(rng, 1, 6000)
        B = _log(rng, 1, max(1, min(128, 24000 // n)))
        rot = rng.choice([d, d // 2])
        return dict(op=op, B=B, n=n, Hq=Hkv * G, Hkv=Hkv, d=d, rot=rot, inter=rng.random() < 0.5, tree=tree,
                    ragged=rng.random() < 0.5, L=_log(rng, 1, 5000), page=page)
    if op == "attn":
        n = _log(rng, 1, 200)
        L = _log(rng, 1, 60000)
        B = _log(rng, 1, max(1, min(128, int(1.0e6 / (L + n)), int(2.0e9 / ((L + 2 * n) * n * Hkv * G)))))
        return dict(op=op, B=B, n=n, Hq=Hkv * G, Hkv=Hkv, d=d, L=L, page=page, branch=rng.choice([0, 2, 3]),
                    ragged=rng.random() < 0.5)
    if op == "accept":
        n = _log(rng, 1, 200)
        V = _log(rng, 500, 150000)
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 500_000_000 // (n * V)))), n=n, V=V,
                    branch=rng.choice([1, 2, 3]), acc=rng.randint(0, 6))
    n = rng.randint(12, 64)
    return dict(op=op, layers=rng.randint(1, 32), B=_log(rng, 1, 100), n=n, Hkv=Hkv, d=d, L=_log(rng, 1, 100),
                page=page, acc=rng.randint(0, 6))


# Lengths and node counts follow from the case alone, so that work() can count them.
def _spread(B, most, least, k):
    """B whole numbers in [least, most], the first of them `most`."""
    return [most if b == 0 else least + int((most - least) * ((b * k) % 1.0)) for b in range(B)]


def _lens(c):
    return _spread(c["B"], c["L"], 0, 0.618034) if c.get("ragged") else [c["L"]] * c["B"]


def _counts(c):
    return _spread(c["B"], c["n"], 0, 0.414214) if c.get("ragged") else [c["n"]] * c["B"]


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


def _pool(c, g, dev, layers=None):
    cap = c["L"] + c["n"]
    mp = -(-cap // c["page"])
    pages = c["B"] * mp + 3
    shape = (pages, c["page"], c["Hkv"], c["d"])
    if layers is not None:
        shape = (layers,) + shape
    table = torch.randperm(pages, generator=g, device=dev)[: c["B"] * mp].view(c["B"], mp).to(I32)
    kp = torch.randn(shape, generator=g, device=dev, dtype=BF16)
    vp = torch.randn(shape, generator=g, device=dev, dtype=BF16)
    return kp, vp, table


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(c)
    i32 = lambda x: torch.tensor(x, dtype=I32, device=dev)  # noqa: E731
    B, n = c["B"], c["n"]
    if c["op"] == "append":
        s["kp"], s["vp"], s["table"] = _pool(c, g, dev)
        # one projection's output holds a token's queries, keys and values side by side
        w = (c["Hq"] + 2 * c["Hkv"])
        qkv = torch.randn((B, n, w, c["d"]), generator=g, device=dev, dtype=BF16)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
        s["len"], s["count"] = i32(_lens(c)), i32(_counts(c)) if c["ragged"] else None
        s["parent"] = _parents(B, n, 2, g, dev) if c["tree"] else None
        base = 500000.0 * (1.0 + 0.1 * float(torch.rand((), generator=g, device=dev)))
        s["inv_freq"] = (base ** (-torch.arange(0, c["rot"], 2, dtype=F64, device=dev) / c["rot"])).to(F32)
        s["q_out"] = torch.zeros((B, n, c["Hq"], c["d"]), dtype=BF16, device=dev)
    elif c["op"] == "attn":
        s["kp"], s["vp"], s["table"] = _pool(c, g, dev)
        # one position in a hundred draws much of the attention
        big = torch.rand(s["kp"].shape[:3], generator=g, device=dev) < 0.01
        s["kp"].mul_(torch.where(big, 4.0, 1.0).to(BF16)[..., None])
        s["q"] = torch.randn((B, n, c["Hq"], c["d"]), generator=g, device=dev, dtype=BF16)
        s["len"], s["count"] = i32(_lens(c)), i32(_counts(c)) if c["ragged"] else None
        s["parent"] = _parents(B, n, c["branch"], g, dev)
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "accept":
        V = c["V"]
        s["target"] = torch.randn((B, n, V), generator=g, device=dev, dtype=F32).mul_(2.0)
        s["tok"] = torch.randint(0, V, (B, n), generator=g, device=dev, dtype=I32)
        par = ((torch.arange(n) - 1).clamp(min=0) // max(1, c["branch"])).tolist()
        par[0] = -1
        s["parent"] = i32(par).expand(B, n).contiguous()
        # the first b % (acc + 1) levels are accepted, along a path taken at random
        rows, nodes, at = [], [], torch.rand((B, 16), generator=g, device=dev).tolist()
        for b in range(B):
            u = 0
            for lvl in range(b % (c["acc"] + 1) if B > 1 else c["acc"]):
                kids = [i for i in range(u * max(1, c["branch"]) + 1, min(n, (u + 1) * max(1, c["branch"]) + 1))]
                if not kids:
                    break
                x = kids[int(at[b][lvl] * len(kids))]
                rows.append((b, u))
                nodes.append(x)
                u = x
        if rows:
            r = torch.tensor(rows, device=dev)
            s["target"][r[:, 0], r[:, 1], s["tok"][r[:, 0], torch.tensor(nodes, device=dev)].long()] = 30.0
    else:
        s["kp"], s["vp"], s["table"] = _pool(c, g, dev, layers=c["layers"])
        s["len"] = i32([c["L"]] * B)
        acc = [b % (c["acc"] + 1) if B > 1 else c["acc"] for b in range(B)]
        # accepted node of level j >= 1: an id past every slot that is written, ascending
        ids = c["acc"] + 1 + torch.rand((B, n - c["acc"] - 1), generator=g, device=dev).argsort(1)[:, : c["acc"]]
        path = torch.full((B, n), -1, dtype=I32, device=dev)
        path[:, 0] = 0
        path[:, 1:c["acc"] + 1] = ids.sort(1).values.to(I32)
        keep = torch.arange(n, device=dev)[None] <= i32(acc)[:, None]
        s["path"], s["n_acc"] = torch.where(keep, path, torch.full_like(path, -1)), i32(acc)
    return s


# ------------------------------------------------------------------------- run
def run(state):
    if own:
        return _kernels(state)
    return {"append": _append, "attn": _attn, "accept": _accept, "commit": _commit}[state["op"]](state)


def _kernels(s):
    from long_context_self_gb300 import binding as mb

    if s["op"] == "append":
        mb.magicdec_paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["len"], s["inv_freq"], q=s["q"],
                                 n_new=s["count"], parent=s["parent"], interleaved=s["inter"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}
    if s["op"] == "attn":
        return mb.magicdec_tree_attn(s["q"], s["kp"], s["vp"], s["table"], s["len"], parent=s["parent"],
                                     n_nodes=s["count"], out=s["out"])
    if s["op"] == "accept":
        n_acc, path, tok = mb.magicdec_tree_accept(s["target"], s["tok"], parent=s["parent"])
        return {"n_acc": n_acc, "path": path, "tok": tok}
    mb.magicdec_tree_commit(s["kp"], s["vp"], s["table"], s["len"], s["path"], s["n_acc"])
    return {"k": s["kp"], "v": s["vp"]}


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
    depth = i.expand(B, n) if s["parent"] is None else _closure(s["parent"]).sum(-1) - 1
    ang = (s["len"].long()[:, None] + depth).to(F64)[..., None] * s["inv_freq"].to(F64)
    cos, sin = ang.cos().to(F32)[:, :, None], ang.sin().to(F32)[:, :, None]

    def turn(x):
        x = x.to(F32)
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
    s["kp"].view(-1, s["Hkv"], d)[at] = turn(s["k"])[live]
    s["vp"].view(-1, s["Hkv"], d)[at] = s["v"][live]
    s["q_out"][live] = turn(s["q"])[live]
    return {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}


def _attn(s):
    B, n, Hkv, d, page = s["B"], s["n"], s["Hkv"], s["d"], s["page"]
    G, cap = s["Hq"] // Hkv, s["L"] + n
    dev = s["q"].device
    length = s["len"].long()[:, None]
    count = torch.full_like(length, n) if s["count"] is None else s["count"].long()[:, None]
    pos = torch.arange(cap, device=dev).expand(B, cap)
    at = _rows(s["table"], pos, page)
    node = pos - length                                                  # [B, cap]: the node at a position
    live = node < count
    anc = _closure(s["parent"])                                          # [B, n, n]
    i = torch.arange(n, device=dev)
    seen = anc.gather(2, node.clamp(0, n - 1)[:, None].expand(B, n, cap)) & (node >= 0)[:, None]
    seen = (seen | (node < 0)[:, None]) & live[:, None] & (i[None] < count)[:, :, None]
    k = s["kp"].view(-1, Hkv, d)[at].to(F32).permute(0, 2, 3, 1)         # [B, Hkv, d, cap]
    q = s["q"].to(F32).view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    x = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(B, Hkv, n, G, cap)
    del k
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["vp"].view(-1, Hkv, d)[at].to(F32).masked_fill_(~live[..., None, None], 0.0).permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, Hkv, n * G, cap), v).view(B, Hkv, n, G, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, s["Hq"], d).to(BF16)


def _accept(s):
    t, tok, parent = s["target"], s["tok"], s["parent"]
    B, n, V = t.shape
    dev = t.device
    best = t.amax(-1, keepdim=True)
    top = torch.where(t == best, torch.arange(V, device=dev, dtype=I32), V).amin(-1).to(I32)     # the lowest index
    i = torch.arange(n, device=dev)
    match = (parent >= 0) & (tok == top.gather(1, parent.clamp(min=0).long()))
    # of the children of one node that match, the lowest goes on
    twin = (parent[:, :, None] == parent[:, None, :]) & match[:, None, :] & (i[None, :] < i[:, None])
    good = (match & ~twin.any(-1)) | (i[None] == 0)
    on = ~(_closure(parent) & ~good[:, None, :]).any(-1)
    n_acc = on.sum(-1).to(I32) - 1
    path = torch.where(on, i[None], n).sort(1).values
    end = path.gather(1, n_acc.long()[:, None])
    took = tok.gather(1, path.roll(-1, 1).clamp(max=n - 1))
    out = torch.where(i[None] < n_acc[:, None], took, torch.where(i[None] == n_acc[:, None], top.gather(1, end), -1))
    path = torch.where(path < n, path, -1).to(I32)
    return {"n_acc": n_acc, "path": path, "tok": out.to(I32)}


def _commit(s):
    layers, page, (B, n) = s["layers"], s["page"], s["path"].shape
    i = torch.arange(n, device=s["path"].device).expand(B, n)
    keep = i <= s["n_acc"][:, None]
    length = s["len"].long()[:, None]
    src = _rows(s["table"], length + s["path"].long().clamp(min=0), page)[keep]
    dst = _rows(s["table"], length + i, page)[keep]
    for x in (s["kp"], s["vp"]):
        x = x.view(layers, -1, s["Hkv"], s["d"])
        x[:, dst] = x[:, src]
    return {"k": s["kp"], "v": s["vp"]}


# ------------------------------------------------------------------------ work
def work(case):
    c = case
    B, n = c["B"], c["n"]
    if c["op"] == "append":
        tokens = sum(_counts(c))
        return {"bytes": 4.0 * tokens * (c["Hq"] + 2 * c["Hkv"]) * c["d"] + 8.0 * B + 4.0 * B * n * c["tree"],
                "flops": 3.0 * tokens * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "attn":
        both = list(zip(_lens(c), _counts(c)))
        kv = sum(ln + m for ln, m in both if m > 0)
        rows = sum(m for _, m in both)
        pairs = sum(m * ln + m * (m + 1) / 2 if c["branch"] == 0 else m * (ln + 1) for ln, m in both)
        return {"bytes": 4.0 * kv * c["Hkv"] * c["d"] + 2.0 * (rows + B * n) * c["Hq"] * c["d"] + 8.0 * B,
                "flops": 4.0 * pairs * c["Hq"] * c["d"]}
    if c["op"] == "accept":
        seen = sum(1 + min(b % (c["acc"] + 1) if B > 1 else c["acc"], _levels(n, c["branch"])) for b in range(B))
        return {"bytes": 4.0 * seen * c["V"] + 16.0 * B * n, "flops": 1.0 * seen * c["V"]}
    moved = sum(b % (c["acc"] + 1) if B > 1 else c["acc"] for b in range(B))
    return {"bytes": 8.0 * moved * c["layers"] * c["Hkv"] * c["d"] + 4.0 * (moved + 2 * B), "flops": 0.0}


def _levels(n, branch):
    """Levels below the root that every path of the complete tree reaches."""
    u, lv = 0, 0
    while (u := u * max(1, branch) + max(1, branch)) < n:
        lv += 1
    return lv


# ----------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "accept": _exact_accept, "commit": _exact_commit}[s["op"]](s)


def _slot(s, b, p):
    return int(s["table"][b, p // s["page"]]), p % s["page"]


def _ancestors(parent, i):
    got = []
    while i >= 0:
        got.append(i)
        i = parent[i]
    return got


def _exact_append(s):
    B, n, rot = s["B"], s["n"], s["rot"]
    lens, counts = _lens(s), _counts(s)
    out = {"q": s["q_out"].double(), "k": s["kp"].double(), "v": s["vp"].double()}
    table = s["table"].long().cpu()
    par = s["parent"].tolist() if s["parent"] is not None else None
    half = torch.arange(rot // 2)
    first, second = (2 * half, 2 * half + 1) if s["inter"] else (half, half + rot // 2)
    for b in range(B):
        m = counts[b]
        if m == 0:
            continue
        slots = torch.arange(lens[b], lens[b] + m)
        pg, row = table[b, slots // s["page"]], slots % s["page"]
        depth = slots if par is None else torch.tensor([lens[b] + len(_ancestors(par[b], i)) - 1 for i in range(m)])
        w = torch.outer(depth.double(), s["inv_freq"].double().cpu())
        turn = torch.polar(torch.ones_like(w), w).to(s["k"].device)
        for name, x in (("q", s["q"]), ("k", s["k"])):
            y = x[b, :m].double()
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            if name == "q":
                out["q"][b, :m] = y
            else:
                out["k"][pg, row] = y
        out["v"][pg, row] = s["v"][b, :m].double()
    return out


def _exact_attn(s):
    B, n, Hkv, d = s["B"], s["n"], s["Hkv"], s["d"]
    G, page = s["Hq"] // Hkv, s["page"]
    lens, counts, par = _lens(s), _counts(s), s["parent"].tolist()
    if sum(ln + m for ln, m in zip(lens, counts)) * n * s["Hq"] * d > 2.5e12:
        return None
    out = torch.zeros((B, n, s["Hq"], d), dtype=F64, device=s["q"].device)
    for b in range(B):
        ln, m = lens[b], counts[b]
        if m == 0:
            continue
        pages = s["table"][b, : -(-(ln + m) // page)].long()
        k, v = (x[pages].flatten(0, 1)[: ln + m].double().transpose(0, 1) for x in (s["kp"], s["vp"]))   # [Hkv, ln+m, d]
        see = torch.zeros((m, ln + m), dtype=torch.bool)
        see[:, :ln] = True
        for i in range(m):
            see[i, [ln + j for j in _ancestors(par[b], i)]] = True
        see = see.to(k.device)[:, None]
        for h in range(Hkv):
            q = s["q"][b, :m, h * G:(h + 1) * G].double()
            w = (q.reshape(m * G, d) @ k[h].T / math.sqrt(d)).view(m, G, ln + m)
            w = torch.where(see, w, -math.inf).softmax(-1)
            out[b, :m, h * G:(h + 1) * G] = (w.view(m * G, ln + m) @ v[h]).view(m, G, d)
    return out


def _exact_accept(s):
    B, n = s["B"], s["n"]
    toks, par = s["tok"].tolist(), s["parent"].tolist()
    n_acc, path, out = [], [], []
    for b in range(B):
        u, way, took = 0, [0], []
        while True:
            row = s["target"][b, u]
            t = int((row == row.max()).nonzero()[0])
            took.append(t)
            u = next((i for i in range(n) if par[b][i] == u and toks[b][i] == t), -1)
            if u < 0:
                break
            way.append(u)
        n_acc.append(len(way) - 1)
        path.append(way + [-1] * (n - len(way)))
        out.append(took + [-1] * (n - len(took)))
    return {"n_acc": torch.tensor(n_acc, dtype=I32), "path": torch.tensor(path, dtype=I32),
            "tok": torch.tensor(out, dtype=I32)}


def _exact_commit(s):
    out = {"k": s["kp"].double(), "v": s["vp"].double()}
    path, acc, lens = s["path"].tolist(), s["n_acc"].tolist(), s["len"].tolist()
    for b in range(s["B"]):
        for i in range(acc[b] + 1):
            (p0, r0), (p1, r1) = _slot(s, b, lens[b] + path[b][i]), _slot(s, b, lens[b] + i)
            for name, x in (("k", s["kp"]), ("v", s["vp"])):
                out[name][:, p1, r1] = x[:, p0, r0].double()
    return out
