"""Plain 64-bit forms of the normed append, of attention behind shared prefixes, and of the
heavy-hitter draft cache.

Roundings: bf16 is off by at most half a step, 2^-8 relative (U), fp32 by 2^-24."""
import math

import torch

from tree_util import F64, U, ancestors, rows_of


def norm_rope_ref(x, w, eps, where, inv_freq, interleaved):
    """(y, bound) in fp64 of x [n, H, d]: normed by w [d] (None: not), pair f turned by where[n, f] *
    inv_freq[f].  Bound: one rounding to bf16 (U relative) and, in fp32, the sum of d squares (at most
    d 2^-24), root and products of the norm, sine, cosine and the turn's products: 2^-15 of a pair's size
    is above them all."""
    y = x.to(F64).clone()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.to(F64)
    size = y.abs()
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot:
        ang = where.to(F64) * inv_freq.to(F64)
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        f = torch.arange(rot // 2, device=x.device)
        i0, i1 = (2 * f, 2 * f + 1) if interleaved else (f, f + rot // 2)
        a, b = y[..., i0].clone(), y[..., i1].clone()
        y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
        both = a.abs() + b.abs()
        size = size.clone()
        size[..., i0], size[..., i1] = both, both
    return y, U * y.abs() + 2.0 ** -15 * size + 1e-38


def heavy_ref(q, kc, vc, weight, pos, lens, next_pos):
    """((out, bound), (weight, bound), pos) of the accumulating attention.  A probability in fp32 carries the errors of
    its score and maximum (fp32 sums of d products: with |q||k| / sqrt(d) below 100, 2^-13 absolute is above
    them), of two exponentials and of the sum; for `out` it is rounded to bf16 besides (U)."""
    B, n, H_q, d = q.shape
    H_kv, cap = kc.shape[1], kc.shape[2]
    G = H_q // H_kv
    dev = q.device
    out = torch.zeros((B, n, H_q, d), dtype=F64, device=dev)
    tol = torch.zeros_like(out)
    w, wt = weight.to(F64), torch.zeros(weight.shape, dtype=F64, device=dev)
    pos = pos.clone()
    for b in range(B):
        ln = min(max(lens[b], 0), cap)
        at = max(0, ln - n)
        if next_pos is not None:
            w[b, :, at:ln] = 0.0
            pos[b, :, at:ln] = next_pos[b] + torch.arange(at - (ln - n), n, device=dev)
        for i in range(n):
            e = ln - n + 1 + i
            if e <= 0:
                continue
            qq = q[b, i].to(F64).view(H_kv, G, d)
            p = (torch.einsum("hgd,hed->hge", qq, kc[b, :, :e].to(F64)) / math.sqrt(d)).softmax(-1)
            v = vc[b, :, :e].to(F64)
            out[b, i] = torch.einsum("hge,hed->hgd", p, v).reshape(H_q, d)
            tol[b, i] = torch.einsum("hge,hed->hgd", p, v.abs()).reshape(H_q, d)
            w[b, :, :e] += p.sum(1)
            wt[b, :, :e] += p.sum(1) * 2.0 ** -12
    # the weight is added to once, in fp32, and its terms are summed in fp32
    wt += w.abs() * 2.0 ** -23 + 1e-30
    return (out, (U + 2.0 ** -10) * tol + U * out.abs() + 1e-30), (w, wt), pos


def evict_ref(kc, vc, weight, pos, lens, total, budget, n_sink, n_recent):
    """What an eviction leaves, row by row; [layers, B, H_kv, cap, d] caches on the CPU."""
    kc, vc, weight, pos = kc.clone(), vc.clone(), weight.clone(), pos.clone()
    layers, B, H_kv, cap, _ = kc.shape
    for lay in range(layers):
        for b in range(B):
            r = min(max(lens[b], 0), cap)
            if r <= budget:
                continue
            for h in range(H_kv):
                w, p = weight[lay, b, h, :r].tolist(), pos[lay, b, h, :r].tolist()
                safe = [x < n_sink or x >= total[b] - n_recent for x in p]
                order = sorted(range(r), key=lambda j: (-(math.inf if safe[j] else w[j]), p[j], j))
                kept = set(order[:budget])
                dst = [j for j in range(budget) if j not in kept]
                src = [j for j in range(budget, r) if j in kept]
                for x in (kc, vc, weight, pos):
                    x[lay, b, h, dst] = x[lay, b, h, src]
    return kc, vc, weight, pos, [min(min(max(x, 0), cap), budget) for x in lens]


def prefix_ref(q, kp, vp, ptable, plens, first, table, lens, parent, counts):
    """(out, bound) in fp64 of attention behind shared prefixes; the bound of tree_util.attn_ref: a probability is
    rounded to bf16 once, whichever part of the softmax it is of."""
    B, n, H_q, d = q.shape
    page, H_kv = kp.shape[1], kp.shape[2]
    G, cap, pcap = H_q // H_kv, table.shape[1] * page, ptable.shape[1] * page
    dev = q.device
    out = torch.zeros((B, n, H_q, d), dtype=F64, device=dev)
    tol = torch.zeros_like(out)
    kf, vf = kp.reshape(-1, H_kv, d), vp.reshape(-1, H_kv, d)
    for b in range(B):
        g = [x for x in range(len(plens)) if first[x] <= b < first[x + 1]]
        lp = min(max(plens[g[0]], 0), pcap) if g else 0
        ln, m = min(max(lens[b], 0), cap), n if counts is None else min(max(counts[b], 0), n)
        own = min(cap, ln + m)
        if m == 0 or lp + own == 0:
            continue
        rows = rows_of(table, b, torch.arange(own), page)
        if lp:
            rows = torch.cat((rows_of(ptable, g[0], torch.arange(lp), page), rows))
        rows = rows.to(dev)
        k, v = kf[rows].to(F64), vf[rows].to(F64)
        see = torch.zeros((m, lp + own), dtype=torch.bool)
        see[:, : lp + ln] = True
        pr = None if parent is None else parent[b].tolist()
        for i in range(m):
            for a in ancestors(pr, i):
                if ln + a < own:
                    see[i, lp + ln + a] = True
        see = see.to(dev)[:, None, None]
        s = torch.einsum("mhgd,lhd->mhgl", q[b, :m].to(F64).view(m, H_kv, G, d), k) / math.sqrt(d)
        s = torch.where(see, s, -math.inf)
        top = s.amax(-1, keepdim=True)
        e = torch.where(see, (s - torch.where(top == -math.inf, 0.0, top)).exp(), 0.0)
        z = e.sum(-1, keepdim=True)
        p = torch.where(z > 0, e / z.clamp(min=1e-300), 0.0)
        out[b, :m] = torch.einsum("mhgl,lhd->mhgd", p, v).reshape(m, H_q, d)
        tol[b, :m] = torch.einsum("mhgl,lhd->mhgd", p, v.abs()).reshape(m, H_q, d)
    return out, (U + 2.0 ** -10) * tol + U * out.abs() + 1e-30
