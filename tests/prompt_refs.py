"""Plain fp64 references of attention over whole sequences, over trees of drafts, and of the cache's pages."""
import math

import torch


def spans(cu):
    return list(zip(cu[:-1], cu[1:]))


def _scores(q, k, scale, window):
    """q [n,Hq,D], k [n,Hkv,D] -> [Hq,n,n] scores, what is not seen at -inf."""
    n, Hq, _ = q.shape
    kk = k.repeat_interleave(Hq // k.shape[1], dim=1)
    s = torch.matmul(q.transpose(0, 1), kk.permute(1, 2, 0)) * scale
    i = torch.arange(n, device=q.device)
    gap = i[:, None] - i[None, :]
    see = gap >= 0
    if window:
        see &= gap < window
    return s.masked_fill(~see, -math.inf)


def attention(q, k, v, cu, scale, window=0):
    """q, k, v [tokens,H,D] of any type -> o, lse in fp64, and sum p |v| / sum p (what one rounding of each weight
    is relative to). Rows of no sequence are zero."""
    q, k, v = q.double(), k.double(), v.double()
    o, size, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q[..., 0])
    G = q.shape[1] // k.shape[1]
    for a, b in spans(cu):
        if a == b:
            continue
        s = _scores(q[a:b], k[a:b], scale, window)
        lse[a:b] = torch.logsumexp(s, -1).t()
        p = torch.softmax(s, -1)
        vv = v[a:b].repeat_interleave(G, dim=1).transpose(0, 1)
        o[a:b], size[a:b] = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
    return o, lse, size


def gradients(q, k, v, do, cu, scale, window=0):
    """dq, dk, dv in fp64, and for each the sum of its terms' sizes: of P |dO| for dv, of |dS| |k| and |dS| |q| for dq
    and dk; last, the same of P in the place of |dS|, which an error of delta is multiplied by."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    Hkv = k.shape[1]
    G = q.shape[1] // Hkv
    out = [torch.zeros_like(x) for x in (q, k, v, q, k, v, q, k)]
    top = lambda x: x.transpose(0, 1)
    shared = lambda x: x.view(Hkv, G, *x.shape[1:]).sum(1).transpose(0, 1)
    for a, b in spans(cu):
        if a == b:
            continue
        p = torch.softmax(_scores(q[a:b], k[a:b], scale, window), -1)
        qq, dd = top(q[a:b]), top(do[a:b])
        kk, vv = (top(x[a:b].repeat_interleave(G, dim=1)) for x in (k, v))
        dp = dd @ vv.transpose(1, 2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        s = abs(scale)
        out[0][a:b], out[1][a:b] = top(ds @ kk) * scale, shared(ds.transpose(1, 2) @ qq) * scale
        out[2][a:b] = shared(p.transpose(1, 2) @ dd)
        out[3][a:b], out[4][a:b] = top(ds.abs() @ kk.abs()) * s, shared(ds.abs().transpose(1, 2) @ qq.abs()) * s
        out[5][a:b] = shared(p.transpose(1, 2) @ dd.abs())
        out[6][a:b], out[7][a:b] = top(p @ kk.abs()) * s, shared(p.transpose(1, 2) @ qq.abs()) * s
    return out


def lineage(parents, i):
    """Draft i and those above it, or None where it is padding."""
    line, x = [], i
    while x >= 0:
        p = parents[x]
        line.append(x)
        if p >= x or p < -1:
            return None
        x = p
    return line


def tree(q, parents, kc, vc, table, starts, scale, window=0):
    """q [B,T,Hq,D], parents, table and starts as lists -> o, lse in fp64 on the CPU. Places on no page are masked."""
    B, T, Hq, D = q.shape
    P, page, Hkv, _ = kc.shape
    q, kc, vc = q.double().cpu(), kc.double().cpu(), vc.double().cpu()
    o, lse = torch.zeros(B, T, Hq, D, dtype=torch.float64), torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    for b in range(B):
        cap = len(table[b]) * page
        n = min(max(starts[b], 0), cap)
        for i in range(T):
            line = lineage(parents[b], i)
            if line is None:
                continue
            pos = list(range(n)) + [n + x for x in reversed(line)]
            if window:
                pos = pos[-window:]
            pos = [p for p in pos if p < cap and 0 <= table[b][p // page] < P]
            if not pos:
                continue
            rows = torch.tensor([table[b][p // page] for p in pos]), torch.tensor([p % page for p in pos])
            kk, vv = (x[rows].repeat_interleave(Hq // Hkv, dim=1).transpose(0, 1) for x in (kc, vc))
            s = (kk @ q[b, i][:, :, None]).squeeze(-1) * scale
            lse[b, i] = torch.logsumexp(s, -1)
            o[b, i] = (torch.softmax(s, -1)[:, None] @ vv).squeeze(1)
    return o, lse


def pages(lengths, counts, table, free, num_free, page, max_tokens):
    """The order of gdr2_kv_pages, request by request. Lists in, lists out: new lengths, bounds, slots, table, stack,
    free pages."""
    P, width = len(free), len(table[0]) if table else 0
    table, free = [list(r) for r in table], list(free)
    is_page = lambda p: 0 <= p < P
    top = min(max(num_free, 0), P)
    held = [min(max(n, 0), width * page) for n in lengths]
    for b, c in enumerate(counts):
        if c < 0:
            for i, p in enumerate(table[b]):
                if is_page(p):
                    if top < P:
                        free[top] = p
                    top += 1
                table[b][i] = -1
    top = min(top, P)
    new, cu, lack, taken = [], [0], 0, 0
    slots = [-1] * max_tokens
    for b, c in enumerate(counts):
        n, first = held[b], cu[-1]
        end = first + max(c, 0)
        cu.append(end)
        if c < 0:
            new.append(0)
            continue
        fits = c > 0 and n + c <= width * page and end <= max_tokens
        want = [i for i in range(n // page, -(-(n + c) // page)) if not is_page(table[b][i])] if fits else []
        lack += len(want)
        if not fits or (want and lack > top):
            new.append(n)
            continue
        for i in want:
            taken += 1
            table[b][i] = free[top - taken]
        new.append(n + c)
        for j in range(c):
            p = table[b][(n + j) // page]
            slots[first + j] = p * page + (n + j) % page if is_page(p) else -1
    return new, [min(x, max_tokens) for x in cu], slots, table, free, top - taken
