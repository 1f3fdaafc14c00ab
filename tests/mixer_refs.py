"""Plain fp64 references of the scalar-gate recurrence and of attention over a paged cache (CPU).

recurrence() is the token loop of the definition and recurrence_grads() its hand-derived
back-propagation; attention() a softmax over the visible tokens gathered page by page."""
import torch


def recurrence(q, k, v, g, beta, h0):
    """One sequence and head group: q, k [T,Hk,dk], v [T,Hv,dv], g, beta [T,Hv], h0 [Hv,dk,dv] or None, all
    fp64. Returns o, the final state and every state on the way (the start state first)."""
    T, Hv, dv = v.shape
    rep = Hv // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    S = torch.zeros(Hv, q.shape[2], dv, dtype=torch.float64) if h0 is None else h0.clone()
    states, out = [S], []
    for t in range(T):
        X = S * torch.exp(g[t])[:, None, None]
        err = v[t] - (k[t][:, :, None] * X).sum(1)
        S = X + k[t][:, :, None] * (beta[t][:, None] * err)[:, None, :]
        out.append((q[t][:, :, None] * S).sum(1))
        states.append(S)
    o = torch.stack(out) if out else torch.zeros(0, Hv, dv, dtype=torch.float64)
    return o, S, states


def recurrence_grads(q, k, v, g, beta, h0, do, dht):
    """Gradients of <o, do> + <h_T, dht>, with o and the final state."""
    T, Hv, dv = v.shape
    Hk, dk = q.shape[1:]
    rep = Hv // Hk
    o, S, states = recurrence(q, k, v, g, beta, h0)
    qe, ke = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    dS = torch.zeros_like(S) if dht is None else dht.clone()
    dq, dkk = torch.zeros_like(qe), torch.zeros_like(ke)
    dvv, dg, db = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(beta)
    for t in reversed(range(T)):
        a = torch.exp(g[t])[:, None, None]
        X = states[t] * a
        err = v[t] - (ke[t][:, :, None] * X).sum(1)
        dq[t] = (states[t + 1] * do[t][:, None, :]).sum(2)
        dS = dS + qe[t][:, :, None] * do[t][:, None, :]
        dwrite = (ke[t][:, :, None] * dS).sum(1)                 # of beta err
        dkk[t] = (dS * (beta[t][:, None] * err)[:, None, :]).sum(2)
        db[t] = (dwrite * err).sum(1)
        dvv[t] = beta[t][:, None] * dwrite
        dkk[t] -= (X * dvv[t][:, None, :]).sum(2)
        dX = dS - ke[t][:, :, None] * dvv[t][:, None, :]
        dg[t] = (dX * X).sum((1, 2))
        dS = dX * a
    group = lambda x: x.view(T, Hk, rep, dk).sum(2)
    return dict(o=o, ht=S, dq=group(dq), dk=group(dkk), dv=dvv, dg=dg, dbeta=db, dh0=dS)


def sequences(x, cu):
    """The sequences of [B,T,...] (cu None) or of packed [1,T,...] tokens, as fp64 on the CPU."""
    x = x.detach().cpu().double()
    return list(x) if cu is None else [x[0, a:b] for a, b in zip(cu[:-1], cu[1:])]


def run_recurrence(x, cu=None, grads=False):
    """x: dict of q, k, v, g, beta, h0 (None), do, dht (None). Returns the outputs as lists over sequences
    (token tensors) or stacked (states)."""
    seqs = {n: sequences(x[n], cu) for n in ("q", "k", "v", "g", "beta")}
    n = len(seqs["q"])
    h0 = [None] * n if x.get("h0") is None else list(x["h0"].cpu().double())
    outs = []
    if grads:
        do = sequences(x["do"], cu)
        dht = [None] * n if x.get("dht") is None else list(x["dht"].cpu().double())
    for i in range(n):
        a = [seqs[m][i] for m in ("q", "k", "v", "g", "beta")]
        if grads:
            outs.append(recurrence_grads(*a, h0[i], do[i], dht[i]))
        else:
            o, S, _ = recurrence(*a, h0[i])
            outs.append(dict(o=o, ht=S))
    res = {}
    for name in outs[0]:
        vals = [o[name] for o in outs]
        res[name] = torch.stack(vals) if name in ("ht", "dh0") else vals
    return res


def attention(q, k_cache, v_cache, table, lengths, scale, window):
    """q [B,Hq,D], caches [P,page,Hkv,D], table and lengths as lists of ints. Returns o, lse in fp64."""
    q, kc, vc = (x.detach().cpu().double() for x in (q, k_cache, v_cache))
    B, Hq, D = q.shape
    P, page, Hkv = kc.shape[:3]
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -float("inf"), dtype=torch.float64)
    for b in range(B):
        n = max(0, min(lengths[b], page * len(table[b])))
        first = max(0, n - window) if window else 0
        seen = [(table[b][t // page], t % page) for t in range(first, n) if 0 <= table[b][t // page] < P]
        if not seen:
            continue
        pg, off = (torch.tensor(c) for c in zip(*seen))
        keys, vals = kc[pg, off], vc[pg, off]                     # [seen, Hkv, D]
        for h in range(Hq):
            s = (keys[:, h // (Hq // Hkv)] * q[b, h]).sum(1) * scale
            lse[b, h] = torch.logsumexp(s, 0)
            o[b, h] = (torch.exp(s - lse[b, h])[:, None] * vals[:, h // (Hq // Hkv)]).sum(0)
    return o, lse


def normwise(got, ref):
    """Frobenius error over the reference's norm (the error itself where the reference is zero)."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    n = float(ref.norm())
    e = float((got - ref).norm())
    return e / n if n > 0 else e
