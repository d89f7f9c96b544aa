"""Plain 64-bit forms of the paged-cache and tree operators, and random inputs for them.

Roundings: bf16 is off by at most half a step, 2^-8 relative (U below)."""
import math

import torch

U = 2.0 ** -8
F64 = torch.float64


def gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def make_cache(lens, n, page, H_kv, d, seed, device, spare=3, extra_slots=0, poison=False, counts=None):
    """A pool with a shuffled table holding lens[b] + n slots per sequence, and the dense K, V in
    fp64.  With `poison`, every pool row outside [0, len + count) is NaN."""
    g = gen(seed)
    B = len(lens)
    cap = max(lens) + n + extra_slots
    mp = -(-cap // page)
    n_pages = B * mp + spare
    table = torch.randperm(n_pages, generator=g)[: B * mp].view(B, mp).to(torch.int32)
    kp = torch.randn((n_pages, page, H_kv, d), generator=g).to(torch.bfloat16)
    vp = torch.randn((n_pages, page, H_kv, d), generator=g).to(torch.bfloat16)
    if poison:
        used = torch.zeros((n_pages * page,), dtype=torch.bool)
        for b in range(B):
            m = n if counts is None else counts[b]
            if m:
                used[rows_of(table, b, torch.arange(lens[b] + m), page)] = True
        kp.view(-1, H_kv, d)[~used] = float("nan")
        vp.view(-1, H_kv, d)[~used] = float("nan")
    return kp.to(device), vp.to(device), table.to(device)


def rows_of(table, b, slots, page):
    return table[b].cpu().long()[slots // page] * page + slots % page


def make_tree(B, n, kind, seed):
    """parent [B, n] int32: chain, star (all hang from node 0), forest (several roots), random."""
    i = torch.arange(n)
    if kind == "chain":
        return (i - 1).to(torch.int32).expand(B, n).contiguous()
    if kind == "star":
        return torch.where(i == 0, -1, 0).to(torch.int32).expand(B, n).contiguous()
    g = gen(seed)
    p = (torch.rand((B, n), generator=g) * i).long().clamp(max=(i - 1).clamp(min=0))
    if kind == "forest":
        p[torch.rand((B, n), generator=g) < 0.3] = -1
    p[:, 0] = -1
    return p.to(torch.int32)


def ancestors(parent_row, i):
    out = []
    while 0 <= i:
        out.append(i)
        p = int(parent_row[i]) if parent_row is not None else i - 1
        i = p if p < i else -1
    return out


def attn_ref(q, kp, vp, table, lens, parent, counts):
    """(out, bound) in fp64.  The bound on |kernel - out|, element by element: each probability
    is rounded to bf16 (U relative) and carries the error of a score and an exponential in fp32
    (2^-10 is far above both), the result is rounded once more (U)."""
    B, n, H_q, d = q.shape
    page, H_kv = kp.shape[1], kp.shape[2]
    G, cap = H_q // H_kv, table.shape[1] * page
    dev = q.device
    out = torch.zeros((B, n, H_q, d), dtype=F64, device=dev)
    tol = torch.zeros_like(out)
    for b in range(B):
        ln, m = min(max(lens[b], 0), cap), n if counts is None else min(max(counts[b], 0), n)
        total = min(cap, ln + m)
        if m == 0 or total == 0:
            continue
        rows = rows_of(table, b, torch.arange(total), page).to(dev)
        k = kp.reshape(-1, H_kv, d)[rows].to(F64)
        v = vp.reshape(-1, H_kv, d)[rows].to(F64)
        see = torch.zeros((m, total), dtype=torch.bool)
        see[:, :ln] = True
        pr = None if parent is None else parent[b].tolist()
        for i in range(m):
            for a in ancestors(pr, i):
                if ln + a < total:
                    see[i, ln + a] = True
        see = see.to(dev)[:, None, None]
        qq = q[b, :m].to(F64).view(m, H_kv, G, d)
        s = torch.einsum("mhgd,lhd->mhgl", qq, k) / math.sqrt(d)
        s = torch.where(see, s, -math.inf)
        top = s.amax(-1, keepdim=True)
        e = torch.where(top == -math.inf, 0.0, (s - torch.where(top == -math.inf, 0.0, top)).exp())
        z = e.sum(-1, keepdim=True)
        p = torch.where(z > 0, e / z.clamp(min=1e-300), 0.0)
        out[b, :m] = torch.einsum("mhgl,lhd->mhgd", p, v).reshape(m, H_q, d)
        tol[b, :m] = torch.einsum("mhgl,lhd->mhgd", p, v.abs()).reshape(m, H_q, d)
    return out, (U + 2.0 ** -10) * tol + U * out.abs() + 1e-30


def rope_ref(x, pos, inv_freq, interleaved):
    """(rotated, bound) in fp64 of x [n, H, d] at positions pos [n].  Bound: one rounding to bf16
    (U relative) and the fp32 sine, cosine and products (2^-21 of the pair's size)."""
    y = x.to(F64).clone()
    tol = torch.zeros_like(y)
    if inv_freq is None:
        return y, tol
    rot = 2 * inv_freq.numel()
    ang = pos.to(F64)[:, None] * inv_freq.to(F64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    f = torch.arange(rot // 2, device=x.device)
    i0, i1 = (2 * f, 2 * f + 1) if interleaved else (f, f + rot // 2)
    a, b = y[..., i0].clone(), y[..., i1].clone()
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    size = a.abs() + b.abs()
    tol[..., i0] = U * y[..., i0].abs() + 2.0 ** -21 * size
    tol[..., i1] = U * y[..., i1].abs() + 2.0 ** -21 * size
    return y, tol


def accept_ref(target, tok, parent, counts):
    B, n, V = target.shape
    n_acc, path, out = [], [], []
    for b in range(B):
        m = n if counts is None else min(max(counts[b], 0), n)
        way, took = [], []
        u = 0 if m else -1
        while u >= 0:
            way.append(u)
            row = target[b, u]
            t = int((row == row.max()).nonzero()[0])
            took.append(t)
            nxt = -1
            for i in range(u + 1, m):
                p = int(parent[b, i]) if parent is not None else i - 1
                if p == u and int(tok[b, i]) == t:
                    nxt = i
                    break
            u = nxt
        n_acc.append(len(way) - 1)
        path.append(way + [-1] * (n - len(way)))
        out.append(took + [-1] * (n - len(took)))
    i32 = torch.int32
    return torch.tensor(n_acc, dtype=i32), torch.tensor(path, dtype=i32), torch.tensor(out, dtype=i32)
