"""Timed cases of the operators for a decoder that mixes recurrent and attention layers.

Five operators, each with a plain form in elementary torch operations (``own`` false) and the
call a program makes of the library (``own`` true):

  train    gated delta rule with scalar gates, forward and backward in one pass
  prefill  the same forward alone, as a server runs it over a prompt
  step     its recurrent form, one or a few tokens a row on resident states
  attend   attention of one new token over a paged key-value cache
  append   new keys and values written into such a cache
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


def listed():
    return [
        # one training step of a mixer layer at the 4096-token training length of the benchmark
        {"name": "train_4k", "op": "train", "dtype": "bf16", "seqs": 2, "lo": 4096, "hi": 4096, "packed": False,
         "hk": 16, "hv": 16, "dk": 128, "dv": 128, "g_scale": 0.1, "h0": False},
        # documents of unequal length packed into one row, value heads sharing key heads, states carried in
        {"name": "train_packed", "op": "train", "dtype": "bf16", "seqs": 9, "lo": 100, "hi": 4000, "packed": True,
         "hk": 8, "hv": 16, "dk": 128, "dv": 128, "g_scale": 0.5, "h0": True},
        # a debugging or fine-tuning step in full precision, small enough that latency counts
        {"name": "train_f32_short", "op": "train", "dtype": "f32", "seqs": 1, "lo": 130, "hi": 130, "packed": False,
         "hk": 2, "hv": 4, "dk": 64, "dv": 64, "g_scale": 0.1, "h0": True},
        # one long prompt read into the state
        {"name": "prefill_16k", "op": "prefill", "dtype": "bf16", "seqs": 1, "lo": 16384, "hi": 16384,
         "packed": False, "hk": 16, "hv": 16, "dk": 128, "dv": 128, "g_scale": 0.1, "h0": True},
        # a batch of short prompts of unequal length
        {"name": "prefill_packed", "op": "prefill", "dtype": "bf16", "seqs": 24, "lo": 17, "hi": 700, "packed": True,
         "hk": 4, "hv": 8, "dk": 64, "dv": 128, "g_scale": 0.1, "h0": False},
        # a single conversation's next token
        {"name": "step_one", "op": "step", "dtype": "bf16", "batch": 1, "tokens": 1, "pool": 4, "hk": 8, "hv": 16,
         "dk": 128, "dv": 128, "g_scale": 0.1},
        # a full server's next tokens, the states in a pool larger than the Infinity Cache
        {"name": "step_512", "op": "step", "dtype": "bf16", "batch": 512, "tokens": 1, "pool": 540, "hk": 16,
         "hv": 16, "dk": 128, "dv": 128, "g_scale": 0.1},
        # a single conversation at a few hundred tokens: latency
        {"name": "attend_one", "op": "attend", "dtype": "bf16", "batch": 1, "lo": 777, "hi": 777, "window": 0,
         "hq": 16, "hkv": 2, "d": 128, "page": 64},
        # a server's batch of unequal lengths, grouped heads
        {"name": "attend_ragged", "op": "attend", "dtype": "bf16", "batch": 64, "lo": 200, "hi": 16384, "window": 0,
         "hq": 32, "hkv": 8, "d": 128, "page": 64},
        # hybrid blocks' 2048-token window in full precision, small pages
        {"name": "attend_window", "op": "attend", "dtype": "f32", "batch": 24, "lo": 1, "hi": 9000, "window": 2048,
         "hq": 16, "hkv": 16, "d": 64, "page": 16},
        # prompts of unequal length written behind what their sequences hold already
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "batch": 12, "lo": 50, "hi": 2500,
         "packed": True, "hkv": 8, "d": 128, "page": 64},
        # the next token of every sequence
        {"name": "append_tokens", "op": "append", "dtype": "bf16", "batch": 96, "lo": 1, "hi": 1, "packed": False,
         "hkv": 8, "d": 128, "page": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["train", "prefill", "step", "attend", "append"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    while True:
        if op in ("train", "prefill"):
            hk = rng.choice([1, 2, 3, 4, 8, 16])
            case = {"op": op, "dtype": dtype, "seqs": _log_int(rng, 1, 24), "packed": rng.random() < 0.5, "hk": hk,
                    "hv": hk * rng.choice([1, 1, 2, 4]), "g_scale": rng.choice([0.02, 0.1, 0.5, 2.0]),
                    "h0": rng.random() < 0.5}
            case["dk"] = 64 if dtype == "f32" else rng.choice([64, 128])
            case["dv"] = 64 if dtype == "f32" else rng.choice([64, 128])
            case["lo"] = case["hi"] = _log_int(rng, 1, 16384)
            if case["packed"]:
                case["lo"] = _log_int(rng, 1, case["hi"])
            limit = 2 * 4096 if op == "train" else 16384
            if sum(_lengths(case)) * case["hv"] > limit * 16 or case["seqs"] * case["hi"] * case["hv"] > 2 ** 20:
                continue
        elif op == "step":
            hk = rng.choice([1, 2, 4, 8, 16])
            batch = _log_int(rng, 1, 512)
            case = {"op": op, "dtype": dtype, "batch": batch, "tokens": rng.choice([1, 1, 1, 2, 5]),
                    "pool": batch + rng.randint(0, 28), "hk": hk, "hv": hk * rng.choice([1, 2, 4]),
                    "dk": 64 if dtype == "f32" else rng.choice([64, 128]),
                    "dv": 64 if dtype == "f32" else rng.choice([64, 128]), "g_scale": rng.choice([0.02, 0.1, 1.0])}
            if batch * case["hv"] * case["dk"] * case["dv"] > 512 * 16 * 128 * 128:
                continue
        elif op == "attend":
            hkv = rng.choice([1, 2, 3, 4, 8, 16])
            hi = _log_int(rng, 1, 65536)
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 128), "lo": _log_int(rng, 1, hi), "hi": hi,
                    "window": rng.choice([0, 0, 0, 1, 100, 2048]), "hq": hkv * rng.choice([1, 2, 3, 4, 8, 16]),
                    "hkv": hkv, "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 256])}
            if sum(_lengths(case)) * hkv * case["d"] * (2 if dtype == "f32" else 1) > 200000 * 8 * 128:
                continue
        else:
            hi = _log_int(rng, 1, 8192)
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 256), "lo": 1, "hi": 1, "packed": False,
                    "hkv": rng.choice([1, 2, 3, 4, 8, 16]), "d": rng.choice([64, 128]),
                    "page": rng.choice([16, 32, 64, 256])}
            if rng.random() < 0.5:
                case.update(packed=True, lo=_log_int(rng, 1, hi), hi=hi)
            if sum(_lengths(case)) * case["hkv"] * case["d"] > 16384 * 8 * 128:
                continue
        return case


def _lengths(case):
    """The case's sequence lengths: all equal, or spread between lo and hi over their logarithm."""
    n = case.get("seqs", case.get("batch"))
    if case["lo"] == case["hi"] or (case["op"] in ("train", "prefill") and not case["packed"]):
        return [case["hi"]] * n
    rng = random.Random("%d %d %d" % (n, case["lo"], case["hi"]))
    lens = [_log_int(rng, case["lo"], case["hi"]) for _ in range(n)]
    lens[rng.randrange(n)] = case["hi"]
    return lens


def _starts(case):
    """append: how many tokens each sequence holds already."""
    rng = random.Random("%d %d" % (case["batch"], case["hi"]))
    return [rng.randint(0, 3 * case["page"]) for _ in range(case["batch"])]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("train", "prefill", "step"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        rows = case["batch"] if case["op"] == "step" else case["seqs"]
        toks = rows * case["tokens"] if case["op"] == "step" else sum(_lengths(case))
        state = rows * hv * dk * dv * 4
        io = toks * es * (2 * hk * dk + 2 * hv * dv + 2 * hv)  # q, k, v, o and the two gates
        if case["op"] == "step":
            return {"bytes": io + 2 * state, "flops": 6 * toks * hv * dk * dv}
        if case["op"] == "prefill":
            return {"bytes": io + state * (2 if case["h0"] else 1), "flops": 6 * toks * hv * dk * dv}
        # do in; dq, dk, dv and the gates' gradients out; states: h_T out, and h0, dh_T in and dh0 out
        io += toks * es * (2 * hk * dk + 2 * hv * dv + 2 * hv)
        return {"bytes": io + state * (4 if case["h0"] else 1), "flops": 18 * toks * hv * dk * dv}
    if case["op"] == "attend":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
        io = case["batch"] * case["hq"] * (2 * case["d"] * es + 4)  # q, o and the log-sum of every row
        return {"bytes": seen * case["hkv"] * case["d"] * 2 * es + io,
                "flops": 4 * seen * case["hq"] * case["d"]}
    moved = sum(_lengths(case)) * case["hkv"] * case["d"] * es * 2
    return {"bytes": 2 * moved, "flops": 0}


# ------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def unit(*shape):  # keys and queries come L2-normalised
        return F.normalize(normal(*shape), dim=-1).to(dt)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    st = {"case": case}
    if case["op"] in ("train", "prefill", "step"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        if case["op"] == "step":
            rows, B, T = case["batch"], case["batch"], case["tokens"]
        else:
            lens = _lengths(case)
            rows = len(lens)
            B, T = (1, sum(lens)) if case["packed"] else (rows, lens[0])
        st["q"], st["k"] = unit(B, T, hk, dk), unit(B, T, hk, dk)
        st["v"] = normal(B, T, hv, dv).to(dt)
        st["g"] = (-F.softplus(normal(B, T, hv)) * case["g_scale"]).to(dt)
        st["beta"] = torch.sigmoid(normal(B, T, hv)).to(dt)
        if case["op"] == "step":
            st["state"] = normal(case["pool"], hv, dk, dv) * 0.1
            order = torch.randperm(case["pool"], generator=gen, device="cuda")
            st["slots"] = order[:rows].to(torch.int32)
            return st
        st["lens"] = lens
        st["cu"] = None
        if case["packed"]:
            st["cu"] = ints([0] + [sum(lens[:i + 1]) for i in range(rows)])
        st["h0"] = normal(rows, hv, dk, dv) * 0.1 if case["h0"] else None
        if case["op"] == "train":
            st["do"] = normal(B, T, hv, dv).to(dt)
            st["dht"] = normal(rows, hv, dk, dv) * 0.1 if case["h0"] else None
        return st

    hkv, d, page, batch = case["hkv"], case["d"], case["page"], case["batch"]
    lens = _lengths(case)
    starts = _starts(case) if case["op"] == "append" else [0] * batch
    need = [(s + n + page - 1) // page for s, n in zip(starts, lens)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table = [[-1] * max(need) for _ in range(batch)]
    for row, n in zip(table, need):
        for i in range(n):
            row[i] = order.pop()
    st["table"] = ints(table)
    st["lens"] = lens
    # caches are filled in the element type, in pieces, so that the largest stays small to make
    for name in ("k_cache", "v_cache"):
        cache = torch.empty(pages, page, hkv, d, dtype=dt, device="cuda")
        cache.normal_(generator=gen)
        st[name] = cache
    if case["op"] == "attend":
        st["lengths"] = ints(lens)
        st["q"] = normal(batch, case["hq"], d).to(dt)
        return st
    st["starts"] = ints(starts)
    st["cu"] = ints([0] + [sum(lens[:i + 1]) for i in range(batch)]) if case["packed"] else None
    st["k"], st["v"] = normal(sum(lens), hkv, d).to(dt), normal(sum(lens), hkv, d).to(dt)
    return st


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------------------------- the library's calls


def _own_train(s):
    import gated_delta_rule_gdr2_amd as g2
    o, ht, ws = g2.gdr2_scalar_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], cu_seqlens=s["cu"],
                                   save_for_bwd=True)
    gr = g2.gdr2_scalar_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], s["do"], s["dht"],
                            cu_seqlens=s["cu"], ws=ws, fwd_saved=True, need_dh0=s["h0"] is not None)
    out = {"o": o, "ht": ht, "dq": gr["dq"], "dk": gr["dk"], "dv": gr["dv"], "dg": gr["dg"], "dbeta": gr["dbeta"]}
    if s["h0"] is not None:
        out["dh0"] = gr["dh0"]
    return out


def _own_prefill(s):
    import gated_delta_rule_gdr2_amd as g2
    o, ht, _ = g2.gdr2_scalar_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], cu_seqlens=s["cu"])
    return {"o": o, "ht": ht}


def _own_step(s):
    import gated_delta_rule_gdr2_amd as g2
    o = g2.gdr2_scalar_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
    return {"o": o, "state": s["state"]}


def _own_attend(s):
    import gated_delta_rule_gdr2_amd as g2
    o, lse = g2.gdr2_attn_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                               window=s["case"]["window"], return_lse=True)
    return {"o": o, "lse": lse}


def _own_append(s):
    import gated_delta_rule_gdr2_amd as g2
    g2.gdr2_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["starts"], cu_seqlens=s["cu"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_OWN = {"train": _own_train, "prefill": _own_prefill, "step": _own_step, "attend": _own_attend,
        "append": _own_append}


# ------------------------------------------------------------------------------------- plain forms


class _Chunks:
    """Tokens of every sequence cut into chunks of 64, padded with zero tokens (which leave the
    recurrence unchanged). Sequences are taken longest first, so the ones that still have a chunk j
    are always the first few."""

    def __init__(self, lens, device):
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        self.order = sorted(range(len(lens)), key=lambda i: -lens[i])
        counts = [(lens[i] + CHUNK - 1) // CHUNK for i in self.order]
        first = [0]
        for c in counts:
            first.append(first[-1] + c)
        self.n = first[-1]
        self.steps = []  # per step j: the chunk ids of the sequences that reach it
        for j in range(max(counts) if counts else 0):
            ids = [first[i] + j for i in range(len(counts)) if counts[i] > j]
            self.steps.append(torch.tensor(ids, device=device))
        chunk_tok = torch.tensor([starts[s] + CHUNK * j for s, c in zip(self.order, counts) for j in range(c)],
                                 device=device)
        chunk_end = torch.tensor([starts[s] + lens[s] for s, c in zip(self.order, counts) for j in range(c)],
                                 device=device)
        tok = chunk_tok[:, None] + torch.arange(CHUNK, device=device)
        self.valid = tok < chunk_end[:, None]                      # [n, 64]
        self.tok = torch.where(self.valid, tok, torch.zeros_like(tok))
        self.flat = tok[self.valid]                                # token of every valid place

    def take(self, x):
        """[tokens, heads, ...] -> [n, heads, 64, ...] in fp32, zero in the padding."""
        y = x.float()[self.tok]
        mask = self.valid.view(*self.valid.shape, *([1] * (x.dim() - 1)))
        return torch.where(mask, y, torch.zeros_like(y)).transpose(1, 2).contiguous()

    def put(self, y, tokens):
        """The inverse of take."""
        y = y.transpose(1, 2)
        out = torch.zeros(tokens, *y.shape[2:], dtype=y.dtype, device=y.device)
        out[self.flat] = y[self.valid]
        return out


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _plain_forward(s, save):
    q, k, v, g, beta = (s[n].flatten(0, 1) for n in ("q", "k", "v", "g", "beta"))
    hk, hv = q.shape[1], v.shape[1]
    ch = _Chunks(s["lens"], q.device)
    qc = ch.take(q).repeat_interleave(hv // hk, dim=1)
    kc = ch.take(k).repeat_interleave(hv // hk, dim=1)
    vc, gc, bc = ch.take(v), ch.take(g), ch.take(beta)
    gam = gc.double().cumsum(-1)                                   # log-decay summed inside the chunk
    lower = torch.ones(CHUNK, CHUNK, device=q.device).tril()
    strict = lower.tril(-1)
    diff = (gam[..., :, None] - gam[..., None, :]).clamp(max=0.0)
    dec = diff.exp().float() * lower                               # exp(gam_r - gam_i), i <= r
    e = gam.exp().float()[..., None]
    tail = (gam[..., -1:] - gam).exp().float()[..., None]
    end = gam[..., -1].exp().float()[..., None, None]
    kt = _t(kc)
    kk = kc @ kt
    A = bc[..., None] * dec * strict * kk
    M = dec * (qc @ kt)
    T = torch.zeros_like(A)                                        # (I + A)^-1, row by row
    eye = torch.eye(CHUNK, device=q.device)
    for r in range(CHUNK):
        row = eye[r].expand(*A.shape[:2], CHUNK)
        if r:
            row = row - (A[..., r:r + 1, :r] @ T[..., :r, :]).squeeze(-2)
        T[..., r, :] = row
    U = T @ (bc[..., None] * vc)
    W = T @ (bc[..., None] * e * kc)
    kd_t = _t(tail * kc)
    n = len(s["lens"])
    dk, dv = q.shape[-1], v.shape[-1]
    state = torch.zeros(n, hv, dk, dv, device=q.device)
    if s["h0"] is not None:
        state = s["h0"][torch.tensor(ch.order, device=q.device)].clone()
    S = torch.empty(ch.n, hv, dk, dv, device=q.device)
    D = torch.empty_like(vc)
    for ids in ch.steps:
        m = ids.numel()
        cur = state[:m]
        S[ids] = cur
        delta = U[ids] - W[ids] @ cur
        D[ids] = delta
        state[:m] = end[ids] * cur + kd_t[ids] @ delta
    o = (e * qc) @ S + M @ D
    ht = torch.empty_like(state)
    ht[torch.tensor(ch.order, device=q.device)] = state
    out = {"o": ch.put(o, q.shape[0]).to(q.dtype).view(*s["v"].shape), "ht": ht}
    return out, ((ch, qc, kc, vc, bc, dec, strict, e, tail, end, A, M, T, W, S, D, kk) if save else None)


def _plain_prefill(s):
    return _plain_forward(s, False)[0]


def _plain_train(s):
    out, saved = _plain_forward(s, True)
    ch, qc, kc, vc, bc, dec, strict, e, tail, end, A, M, T, W, S, D, kk = saved
    hk, hv = s["q"].shape[2], s["v"].shape[2]
    tokens = s["q"].shape[0] * s["q"].shape[1]
    do = ch.take(s["do"].flatten(0, 1))
    dstate = torch.zeros_like(out["ht"])
    order = torch.tensor(ch.order, device=do.device)
    if s["dht"] is not None:
        dstate = s["dht"][order].clone()
    from_out = _t(M) @ do
    qg_t, w_t, kd = _t(e * qc), _t(W), tail * kc
    dS = torch.empty_like(S)                                       # gradient of every chunk's end state
    dD = torch.empty_like(D)
    for ids in reversed(ch.steps):
        m = ids.numel()
        cur = dstate[:m]
        dS[ids] = cur
        dd = from_out[ids] + kd[ids] @ cur
        dD[ids] = dd
        dstate[:m] = end[ids] * cur + qg_t[ids] @ do[ids] - w_t[ids] @ dd
    dY = _t(T) @ dD
    dM = (do @ _t(D)) * dec
    dA = -(dY @ _t(D)) * strict * dec
    P = dM
    R = dA * bc[..., None]
    s_t = _t(S)
    dq_state = e * (do @ s_t)
    dx_state = -(e * (dY @ s_t))
    dk_state = tail * (D @ _t(dS))
    dq = dq_state + P @ kc
    dk = _t(P) @ qc + R @ kc + _t(R) @ kc + bc[..., None] * dx_state + dk_state
    dv = bc[..., None] * dY
    dbeta = (dY * vc).sum(-1) + (dx_state * kc).sum(-1) + (dA * kk).sum(-1)
    qk = M * (do @ _t(D))                                          # dM * M without the second decay factor
    aa = R * kk
    both = (qk + aa).double()
    kd_dot = (dk_state * kc).sum(-1).double()
    dgam = both.sum(-1) - both.sum(-2) + (dq_state * qc).sum(-1) + bc * (dx_state * kc).sum(-1) - kd_dot
    dgam[..., -1] += kd_dot.sum(-1) + (end[..., 0, 0] * (dS * S).sum((-1, -2))).double()
    dg = dgam.flip(-1).cumsum(-1).flip(-1).float()

    def shared(x):                                                 # sum over the value heads of a key head
        return x.view(x.shape[0], hk, hv // hk, *x.shape[2:]).sum(2)

    dt = s["q"].dtype
    out["dq"] = ch.put(shared(dq), tokens).to(dt).view(s["q"].shape)
    out["dk"] = ch.put(shared(dk), tokens).to(dt).view(s["k"].shape)
    out["dv"] = ch.put(dv, tokens).to(dt).view(s["v"].shape)
    out["dg"] = ch.put(dg[..., None], tokens).to(dt).view(s["g"].shape)
    out["dbeta"] = ch.put(dbeta[..., None], tokens).to(dt).view(s["g"].shape)
    if s["h0"] is not None:
        out["dh0"] = torch.empty_like(dstate)
        out["dh0"][order] = dstate
    return out


def _plain_step(s):
    slots = s["slots"].long()
    hk, hv = s["q"].shape[2], s["v"].shape[2]
    q = s["q"].float().repeat_interleave(hv // hk, dim=2)
    k = s["k"].float().repeat_interleave(hv // hk, dim=2)
    v = s["v"].float()
    S = s["state"][slots]
    outs = []
    for t in range(q.shape[1]):
        S = S * s["g"][:, t].float().exp()[..., None, None]
        u = (S * k[:, t][..., None]).sum(-2)
        delta = s["beta"][:, t].float()[..., None] * (v[:, t] - u)
        S = S + k[:, t][..., None] * delta[..., None, :]
        outs.append((S * q[:, t][..., None]).sum(-2))
    s["state"][slots] = S
    return {"o": torch.stack(outs, dim=1).to(s["q"].dtype), "state": s["state"]}


def _plain_attend(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(case["batch"], hq, d, dtype=s["q"].dtype, device=s["q"].device)
    lse = torch.zeros(case["batch"], hq, device=s["q"].device)
    for b, n in enumerate(s["lens"]):
        lo = max(0, n - case["window"]) if case["window"] else 0
        p0 = lo // page
        ids = s["table"][b, p0:(n + page - 1) // page].long()
        ks = s["k_cache"][ids].flatten(0, 1)[lo - p0 * page:n - p0 * page].float()   # [seen, hkv, d]
        vs = s["v_cache"][ids].flatten(0, 1)[lo - p0 * page:n - p0 * page].float()
        qh = s["q"][b].float().view(hkv, hq // hkv, d)
        sc = (qh @ ks.permute(1, 2, 0).contiguous()) * d ** -0.5                     # [hkv, group, seen]
        top = sc.amax(-1, keepdim=True)
        p = (sc - top).exp()
        total = p.sum(-1, keepdim=True)
        o = (p @ vs.transpose(0, 1).contiguous()) / total
        out[b] = o.reshape(hq, d).to(out.dtype)
        lse[b] = (top + total.log()).view(hq)
    return {"o": out, "lse": lse}


def _plain_append(s):
    page = s["case"]["page"]
    total = s["k"].shape[0]
    place = torch.arange(total, device=s["k"].device)
    if s["cu"] is None:
        row, pos = place, s["starts"].long()
    else:
        cu = s["cu"].long()
        row = torch.searchsorted(cu[1:].contiguous(), place, right=True)
        pos = s["starts"].long()[row] + place - cu[row]
    ids = s["table"].long()[row, pos // page]
    s["k_cache"][ids, pos % page] = s["k"]
    s["v_cache"][ids, pos % page] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_PLAIN = {"train": _plain_train, "prefill": _plain_prefill, "step": _plain_step, "attend": _plain_attend,
          "append": _plain_append}


# ------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    if case["op"] == "append":
        return None  # copies
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "step":
        return _exact_step(s)
    lens, hv = s["lens"], case["hv"]
    if len(lens) * max(lens) * hv * case["dk"] * case["dv"] * 8 > 1e11 and case["op"] == "train":
        return None  # every state of the recurrence is kept for the way back
    if max(lens) > 40000:
        return None
    return _exact_tokens(s)


def _padded(x, lens, rep=1):
    """[B, T, H, ...] (packed or not) -> [N, longest, H * rep, ...] in fp64, zero behind each sequence."""
    flat = x.flatten(0, 1).double()
    out = torch.zeros(len(lens), max(lens), *flat.shape[1:], dtype=torch.float64, device=x.device)
    at = 0
    for i, n in enumerate(lens):
        out[i, :n] = flat[at:at + n]
        at += n
    return out.repeat_interleave(rep, dim=2) if rep > 1 else out


def _unpadded(y, lens, shape):
    return torch.cat([y[i, :n] for i, n in enumerate(lens)]).reshape(shape)


def _exact_tokens(s):
    """The recurrence, token by token; padding tokens have beta = 0 and g = 0 and change nothing."""
    case, lens = s["case"], s["lens"]
    hk, hv = case["hk"], case["hv"]
    rep = hv // hk
    q, k = _padded(s["q"], lens, rep), _padded(s["k"], lens, rep)
    v, g, beta = _padded(s["v"], lens), _padded(s["g"], lens), _padded(s["beta"], lens)
    train = case["op"] == "train"
    N, T = q.shape[:2]
    S = torch.zeros(N, hv, case["dk"], case["dv"], dtype=torch.float64, device=q.device)
    if s["h0"] is not None:
        S = s["h0"].double()
    o = torch.zeros_like(v)
    delta = torch.zeros_like(v)
    kept = [S] if train else None
    for t in range(T):
        X = S * g[:, t, :, None, None].exp()
        delta[:, t] = beta[:, t, :, None] * (v[:, t] - torch.einsum("nhk,nhkv->nhv", k[:, t], X))
        S = X + k[:, t, :, :, None] * delta[:, t, :, None, :]
        o[:, t] = torch.einsum("nhk,nhkv->nhv", q[:, t], S)
        if train:
            kept.append(S)
    out = {"o": _unpadded(o, lens, s["v"].shape), "ht": S}
    if not train:
        return out
    do = _padded(s["do"], lens)
    dS = s["dht"].double() if s["dht"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(g), torch.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        S = kept.pop()
        a = g[:, t, :, None, None].exp()
        X = kept[-1] * a
        dS = dS + q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = torch.einsum("nhkv,nhv->nhk", S, do[:, t])
        dd = torch.einsum("nhk,nhkv->nhv", k[:, t], dS)
        dk[:, t] = torch.einsum("nhkv,nhv->nhk", dS, delta[:, t])
        dv[:, t] = beta[:, t, :, None] * dd
        dbeta[:, t] = (dd * (v[:, t] - torch.einsum("nhk,nhkv->nhv", k[:, t], X))).sum(-1)
        dk[:, t] -= torch.einsum("nhkv,nhv->nhk", X, dv[:, t])
        dX = dS - k[:, t, :, :, None] * dv[:, t, :, None, :]
        dg[:, t] = (dX * X).sum((-1, -2))
        dS = dX * a

    def shared(x):
        return x.view(N, T, hk, rep, -1).sum(3)

    out["dq"] = _unpadded(shared(dq), lens, s["q"].shape)
    out["dk"] = _unpadded(shared(dk), lens, s["k"].shape)
    out["dv"] = _unpadded(dv, lens, s["v"].shape)
    out["dg"] = _unpadded(dg, lens, s["g"].shape)
    out["dbeta"] = _unpadded(dbeta, lens, s["g"].shape)
    if s["h0"] is not None:
        out["dh0"] = dS
    return out


def _exact_step(s):
    rep = s["v"].shape[2] // s["q"].shape[2]
    pool = s["state"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device=pool.device)
    slots = s["slots"].long()
    S = pool[slots]
    for t in range(o.shape[1]):
        k = s["k"][:, t].double().repeat_interleave(rep, dim=1)
        q = s["q"][:, t].double().repeat_interleave(rep, dim=1)
        S = S * s["g"][:, t].double().exp()[..., None, None]
        err = s["v"][:, t].double() - torch.einsum("bhk,bhkv->bhv", k, S)
        S = S + torch.einsum("bhk,bhv->bhkv", k, s["beta"][:, t].double()[..., None] * err)
        o[:, t] = torch.einsum("bhk,bhkv->bhv", q, S)
    pool[slots] = S
    return {"o": o, "state": pool}


def _exact_attend(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(case["batch"], hq, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"]):
        first = max(0, n - case["window"]) if case["window"] else 0
        pos = torch.arange(first, n, device=out.device)
        rows = s["table"][b].long()[pos // page]
        for h in range(hkv):
            keys = s["k_cache"][rows, pos % page, h].double()
            vals = s["v_cache"][rows, pos % page, h].double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            score = torch.mm(s["q"][b, heads].double(), keys.t()) / math.sqrt(d)
            lse[b, heads] = torch.logsumexp(score, dim=-1)
            out[b, heads] = torch.mm((score - lse[b, heads][:, None]).exp(), vals)
    return {"o": out, "lse": lse}
