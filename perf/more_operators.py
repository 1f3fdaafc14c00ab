"""Timed cases of the attention layers' prompts, gradients and drafted tokens, and of the cache's pages.

Five operators, each with a plain form in elementary torch operations (``own`` false) and the
call a program makes of the library (``own`` true):

  train    causal attention over whole sequences, forward and backward in one pass
  prompt   the same forward alone, as a server runs it over prompts
  tree     attention of a tree of drafted tokens over a paged key-value cache
  keep     the accepted drafts' keys and values moved together in the cache
  pages    pages for the tokens to come: block tables, slots and bounds from request lengths
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 2 ** 28  # scores that a plain form holds at a time


def listed():
    return [
        # one training step of an attention layer at the 4096-token training length of the benchmark
        {"name": "train_4k", "op": "train", "dtype": "bf16", "seqs": 2, "lo": 4096, "hi": 4096, "packed": False,
         "hq": 16, "hkv": 16, "d": 128, "window": 0},
        # documents of unequal length packed into one row, grouped heads, a hybrid block's 2048-token window
        {"name": "train_packed", "op": "train", "dtype": "bf16", "seqs": 9, "lo": 100, "hi": 4000, "packed": True,
         "hq": 16, "hkv": 4, "d": 64, "window": 2048},
        # a debugging or fine-tuning step in full precision, small enough that latency counts
        {"name": "train_f32_short", "op": "train", "dtype": "f32", "seqs": 1, "lo": 130, "hi": 130, "packed": False,
         "hq": 4, "hkv": 2, "d": 64, "window": 0},
        # one long prompt
        {"name": "prompt_16k", "op": "prompt", "dtype": "bf16", "seqs": 1, "lo": 16384, "hi": 16384,
         "packed": False, "hq": 16, "hkv": 2, "d": 128, "window": 0},
        # a batch of short prompts of unequal length
        {"name": "prompt_packed", "op": "prompt", "dtype": "bf16", "seqs": 24, "lo": 17, "hi": 700, "packed": True,
         "hq": 16, "hkv": 4, "d": 128, "window": 0},
        # a question of a few words: latency
        {"name": "prompt_short", "op": "prompt", "dtype": "bf16", "seqs": 1, "lo": 29, "hi": 29, "packed": False,
         "hq": 16, "hkv": 2, "d": 128, "window": 0},
        # one conversation with a few drafted tokens: latency
        {"name": "tree_one", "op": "tree", "dtype": "bf16", "batch": 1, "lo": 777, "hi": 777, "drafts": 12,
         "hq": 16, "hkv": 2, "d": 128, "page": 64, "window": 0},
        # a server's batch of unequal lengths, trees of up to 32 tokens, grouped heads
        {"name": "tree_ragged", "op": "tree", "dtype": "bf16", "batch": 32, "lo": 200, "hi": 16384, "drafts": 32,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0},
        # one accepted path of a single conversation
        {"name": "keep_one", "op": "keep", "dtype": "bf16", "batch": 1, "drafts": 12, "path": 5, "hkv": 2, "d": 128,
         "page": 64},
        # the accepted paths of a large batch with deep trees
        {"name": "keep_batch", "op": "keep", "dtype": "bf16", "batch": 256, "drafts": 64, "path": 24, "hkv": 8,
         "d": 128, "page": 16},
        # every request of a batch goes on by one token
        {"name": "pages_step", "op": "pages", "batch": 96, "lo": 1, "hi": 16384, "page": 16, "new": 0, "new_hi": 1,
         "gone": 0, "pool": 1.2},
        # a batch in which prompts come in, most requests go on, and some end
        {"name": "pages_prompts", "op": "pages", "batch": 512, "lo": 1, "hi": 16384, "page": 64, "new": 24,
         "new_hi": 2500, "gone": 16, "pool": 1.05},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["train", "train", "prompt", "prompt", "tree", "tree", "keep", "pages"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    while True:
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
        window = rng.choice([0, 0, 0, 1, 100, 2048])
        if op in ("train", "prompt"):
            case = {"op": op, "dtype": dtype, "seqs": _log_int(rng, 1, 24), "packed": rng.random() < 0.5, "hq": hq,
                    "hkv": hkv, "d": rng.choice([64, 128]), "window": window}
            case["lo"] = case["hi"] = _log_int(rng, 1, 16384)
            if case["packed"]:
                case["lo"] = _log_int(rng, 1, case["hi"])
            if op == "train" and (case["hi"] == 1 or window == 1):
                continue  # weights of one, whose gradients are zero
            if work(case)["flops"] * (8 if dtype == "f32" else 1) > 1.1e12:
                continue
            if case["seqs"] * case["hi"] ** 2 * hq > 16 * 16384 ** 2:
                continue
        elif op == "tree":
            hi = _log_int(rng, 1, 32768)
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 64), "lo": _log_int(rng, 1, hi), "hi": hi,
                    "drafts": _log_int(rng, 1, 64), "hq": hq, "hkv": hkv, "d": rng.choice([64, 128]),
                    "page": rng.choice([16, 32, 64, 256]), "window": window}
            if sum(_lengths(case)) * hkv * case["d"] * (2 if dtype == "f32" else 1) > 150000 * 8 * 128:
                continue
            if case["batch"] * hi * max(hkv * case["d"], hq * case["drafts"]) > 2 ** 30:
                continue
        elif op == "keep":
            drafts = _log_int(rng, 1, 64)
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 256), "drafts": drafts,
                    "path": rng.randint(1, drafts), "hkv": hkv, "d": rng.choice([64, 128]),
                    "page": rng.choice([16, 32, 64, 256])}
        else:
            batch = _log_int(rng, 1, 2048)
            hi = _log_int(rng, 1, 16384)
            new = rng.choice([0, 0, rng.randint(0, min(batch, 32))])
            case = {"op": op, "batch": batch, "lo": _log_int(rng, 1, hi), "hi": hi,
                    "page": rng.choice([16, 32, 64, 256]), "new": new, "new_hi": _log_int(rng, 1, 4000),
                    "gone": rng.choice([0, rng.randint(0, (batch - new) // 4 + 1)]),
                    "pool": rng.choice([1.0, 1.01, 1.2])}
            case["gone"] = min(case["gone"], batch - new)
            if batch * (hi + case["new_hi"]) // case["page"] > 2 ** 21:
                continue
        return case


def _lengths(case):
    """The case's sequence lengths: all equal, or spread between lo and hi over their logarithm."""
    n = case.get("seqs", case.get("batch"))
    if case["lo"] == case["hi"] or (case["op"] in ("train", "prompt") and not case["packed"]):
        return [case["hi"]] * n
    rng = random.Random("%d %d %d" % (n, case["lo"], case["hi"]))
    lens = [_log_int(rng, case["lo"], case["hi"]) for _ in range(n)]
    lens[rng.randrange(n)] = case["hi"]
    return lens


def _trees(case, rng):
    """Each row's drafts: the parent of each, -1 for a child of the last token held. Rows have some drafts
    fewer than the widest; the places behind them are padding, -2."""
    rows = []
    for b in range(case["batch"]):
        n = case["drafts"] if b == 0 else rng.randint((case["drafts"] + 1) // 2, case["drafts"])
        row = [rng.choice([i - 1, i - 1, rng.randint(-1, i - 1)]) for i in range(n)]
        rows.append(row + [-2] * (case["drafts"] - n))
    return rows


def _held(case):
    """keep: how many tokens each sequence holds before its drafts."""
    rng = random.Random("%d %d" % (case["batch"], case["path"]))
    return [rng.randint(0, 3 * case["page"]) for _ in range(case["batch"])]


def _seen(n, window):
    """Pairs of a causal sequence of n tokens, each seeing the last `window`."""
    w = min(window, n) if window else n
    return w * (w + 1) // 2 + (n - w) * w


def work(case):
    es = 4 if case.get("dtype") == "f32" else 2
    if case["op"] in ("train", "prompt"):
        lens = _lengths(case)
        toks, pairs = sum(lens), sum(_seen(n, case["window"]) for n in lens) * case["hq"]
        io = toks * (2 * case["hq"] + 2 * case["hkv"]) * case["d"] * es + toks * case["hq"] * 4  # q, o, k, v, lse
        if case["op"] == "prompt":
            return {"bytes": io, "flops": 4 * pairs * case["d"]}
        # do in; dq, dk and dv out; two products forward, four backward
        io += toks * (2 * case["hq"] + 2 * case["hkv"]) * case["d"] * es
        return {"bytes": io, "flops": 12 * pairs * case["d"]}
    if case["op"] == "tree":
        T, w = case["drafts"], case["window"]
        held = sum(min(n, w + T) if w else n for n in _lengths(case)) + case["batch"] * T
        rows = case["batch"] * T * case["hq"]
        return {"bytes": held * case["hkv"] * case["d"] * 2 * es + rows * (2 * case["d"] * es + 4),
                "flops": 4 * held * T * case["hq"] * case["d"]}
    if case["op"] == "keep":
        return {"bytes": 2 * case["batch"] * case["path"] * case["hkv"] * case["d"] * 2 * es, "flops": 0}
    counts, tokens = _counts(case), _max_tokens(case)
    touched = sum((c + case["page"] - 1) // case["page"] for c in counts if c > 0)
    gone = sum((n + case["page"] - 1) // case["page"] for n, c in zip(_lengths(case), counts) if c < 0)
    return {"bytes": 4 * (4 * len(counts) + 2 * touched + 3 * gone) + 8 * tokens, "flops": 0}


def _counts(case):
    """pages: the tokens that come to each request; -1 for one that ends."""
    rng = random.Random("%d %d %d" % (case["batch"], case["new"], case["gone"]))
    counts = [1] * case["batch"]
    rows = rng.sample(range(case["batch"]), case["new"] + case["gone"])
    for b in rows[:case["new"]]:
        counts[b] = _log_int(rng, 1, case["new_hi"])
    for b in rows[case["new"]:]:
        counts[b] = -1
    return counts


def _max_tokens(case):
    return sum(max(c, 0) for c in _counts(case)) + 7


# ------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    st = {"case": case}
    if case["op"] in ("train", "prompt"):
        dt = DTYPES[case["dtype"]]
        lens = _lengths(case)
        B, T = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
        st["lens"] = lens
        st["q"] = normal(B, T, case["hq"], case["d"]).to(dt)
        st["k"], st["v"] = (normal(B, T, case["hkv"], case["d"]).to(dt) for _ in range(2))
        st["cu"] = ints([0] + [sum(lens[:i + 1]) for i in range(len(lens))]) if case["packed"] else None
        if case["op"] == "train":
            st["do"] = normal(B, T, case["hq"], case["d"]).to(dt)
        return st

    if case["op"] == "pages":
        lens, counts, page = _lengths(case), _counts(case), case["page"]
        lens = [0 if b and c > 1 else n for b, (n, c) in enumerate(zip(lens, counts))]  # prompts come to empty rows
        need = [(n + page - 1) // page for n in lens]
        most = max(max(n, 0) + max(c, 0) for n, c in zip(lens, counts))
        want = sum((n + max(c, 0) + page - 1) // page for n, c in zip(lens, counts))
        pages = max(sum(need), int(want * case["pool"]))
        # 64 more pages of the pool belong to others, prompts kept for later requests
        order = torch.randperm(pages + 64, generator=gen, device="cuda").to(torch.int32)
        width = (most + page - 1) // page + 1
        need_t = ints(need).long()
        col = torch.arange(width, device="cuda")
        place = (need_t.cumsum(0) - need_t)[:, None] + col
        used = col < need_t[:, None]
        st["table"] = torch.where(used, order[place.clamp(max=pages - 1)], torch.full_like(place, -1).int())
        # the free ones first; what stands behind has no meaning
        st["free"] = torch.cat([order[sum(need):pages], order[:sum(need)], order[pages:]])
        st["num_free"] = ints([pages - sum(need)])
        st["lengths"], st["counts"] = ints(lens), ints(counts)
        st["max_tokens"] = _max_tokens(case)
        return st

    dt = DTYPES[case["dtype"]]
    hkv, d, page, batch = case["hkv"], case["d"], case["page"], case["batch"]
    lens = _lengths(case) if case["op"] == "tree" else _held(case)
    need = [(n + case["drafts"] + page - 1) // page for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table = [[-1] * max(need) for _ in range(batch)]
    for row, n in zip(table, need):
        for i in range(n):
            row[i] = order.pop()
    st["table"], st["starts"], st["lens"] = ints(table), ints(lens), lens
    for name in ("k_cache", "v_cache"):
        cache = torch.empty(pages, page, hkv, d, dtype=dt, device="cuda")
        cache.normal_(generator=gen)
        st[name] = cache
    if case["op"] == "tree":
        st["q"] = normal(batch, case["drafts"], case["hq"], d).to(dt)
        st["parents"] = ints(_trees(case, rng))
        return st
    paths = []
    for b in range(batch):  # ascending drafts, the path of some rows shorter than the longest
        n = case["path"] if b == 0 else rng.randint(0, case["path"])
        paths.append(sorted(rng.sample(range(case["drafts"]), n)) + [-1] * (case["path"] - n))
    st["path"] = ints(paths)
    return st


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------------------------- the library's calls


def _own_train(s):
    import gated_delta_rule_gdr2_amd as g2
    w = s["case"]["window"]
    o, lse, rest = g2.gdr2_attn_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], window=w, save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], rest=rest, cu_seqlens=s["cu"], window=w)
    return {"o": o, "lse": lse, "dq": gr["dq"], "dk": gr["dk"], "dv": gr["dv"]}


def _own_prompt(s):
    import gated_delta_rule_gdr2_amd as g2
    o, lse = g2.gdr2_attn_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], window=s["case"]["window"],
                              return_lse=True)
    return {"o": o, "lse": lse}


def _own_tree(s):
    import gated_delta_rule_gdr2_amd as g2
    o, lse = g2.gdr2_attn_tree(s["q"], s["parents"], s["k_cache"], s["v_cache"], s["table"], s["starts"],
                               window=s["case"]["window"], return_lse=True)
    return {"o": o, "lse": lse}


def _own_keep(s):
    import gated_delta_rule_gdr2_amd as g2
    lengths = g2.gdr2_kv_keep(s["k_cache"], s["v_cache"], s["table"], s["starts"], s["path"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": lengths}


def _own_pages(s):
    import gated_delta_rule_gdr2_amd as g2
    lengths, cu, slots = g2.gdr2_kv_pages(s["lengths"], s["counts"], s["table"], s["free"], s["num_free"],
                                          page_size=s["case"]["page"], max_tokens=s["max_tokens"])
    return {"lengths": lengths, "cu": cu, "slots": slots, "table": s["table"], "free": s["free"],
            "num_free": s["num_free"]}


_OWN = {"train": _own_train, "prompt": _own_prompt, "tree": _own_tree, "keep": _own_keep, "pages": _own_pages}


# ------------------------------------------------------------------------------------- plain forms


class _Rows:
    """Sequences as rows of one padded array, in blocks of query tokens that keep the scores small."""

    def __init__(self, s):
        case, lens = s["case"], s["lens"]
        self.n, self.longest, self.window = len(lens), max(lens), case["window"]
        self.hkv, self.group, self.d = case["hkv"], case["hq"] // case["hkv"], case["d"]
        self.shape, self.dtype = s["q"].shape, s["q"].dtype
        dev = s["q"].device
        self.pos = torch.arange(self.longest, device=dev)
        if s["cu"] is None:
            self.index = torch.arange(self.n * self.longest, device=dev).view(self.n, self.longest)
            self.real = torch.ones(self.n, self.longest, dtype=torch.bool, device=dev)
        else:
            cu = s["cu"].long()
            self.real = self.pos < (cu[1:] - cu[:-1])[:, None]
            self.index = torch.where(self.real, cu[:-1, None] + self.pos, torch.zeros_like(self.pos))
        step = max(1, min(self.longest, BLOCK // (self.n * case["hq"] * self.longest)))
        self.blocks = [(i, min(i + step, self.longest)) for i in range(0, self.longest, step)]

    def heads(self, x):
        """[B, T, H, ...] -> [n, hkv, H / hkv, longest, ...] in 32 bits."""
        y = x.flatten(0, 1).float()[self.index]
        y = y.view(self.n, self.longest, self.hkv, -1, *x.shape[3:])
        return y.permute(0, 2, 3, 1, *range(4, y.dim())).contiguous()

    def tokens(self, y, dtype):
        """The inverse of heads."""
        y = y.permute(0, 3, 1, 2, *range(4, y.dim()))
        out = y.new_zeros(self.shape[0] * self.shape[1], *y.shape[2:])
        # padded places go to a row behind the last
        place = torch.where(self.real, self.index, torch.full_like(self.index, out.shape[0]))
        out = torch.cat([out, out[:1]])
        out[place.flatten()] = y.flatten(0, 1)
        out = out[:-1].flatten(1, 2).to(dtype)
        return out.view(*self.shape[:2], *out.shape[1:])

    def scores(self, q, k, i0, i1):
        """The block's scores [n, hkv, G, i1 - i0, keys], what is not seen at -inf, and its first and last key."""
        lo = max(0, i0 - self.window + 1) if self.window else 0
        kt = k[:, :, 0, lo:i1].transpose(-1, -2).contiguous()
        sc = q[:, :, :, i0:i1].flatten(2, 3) @ kt * self.d ** -0.5
        sc = sc.view(self.n, self.hkv, self.group, i1 - i0, i1 - lo)
        far = self.pos[i0:i1, None] - self.pos[None, lo:i1]
        hide = (far < 0) | (far >= self.window) if self.window else far < 0
        return sc.masked_fill(hide, -math.inf), lo


def _plain_forward(s):
    r = _Rows(s)
    q, k, v = r.heads(s["q"]), r.heads(s["k"]), r.heads(s["v"])
    o, lse = torch.empty_like(q), torch.empty_like(q[..., 0])
    for i0, i1 in r.blocks:
        sc, lo = r.scores(q, k, i0, i1)
        top = sc.amax(-1, keepdim=True)
        p = (sc - top).exp()
        total = p.sum(-1, keepdim=True)
        o[:, :, :, i0:i1] = (p.flatten(2, 3) @ v[:, :, 0, lo:i1].contiguous()).view(o[:, :, :, i0:i1].shape) / total
        lse[:, :, :, i0:i1] = (top + total.log()).squeeze(-1)
    return r, q, k, v, o, lse


def _plain_prompt(s):
    r, _, _, _, o, lse = _plain_forward(s)
    return {"o": r.tokens(o, r.dtype), "lse": r.tokens(lse, torch.float32)}


def _plain_train(s):
    r, q, k, v, o, lse = _plain_forward(s)
    do = r.heads(s["do"]) * r.real[:, None, None, :, None]
    delta = (do * o).sum(-1, keepdim=True)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i0, i1 in r.blocks:
        sc, lo = r.scores(q, k, i0, i1)
        p = (sc - lse[:, :, :, i0:i1, None]).exp()
        dob = do[:, :, :, i0:i1].flatten(2, 3)
        dp = (dob @ v[:, :, 0, lo:i1].transpose(-1, -2).contiguous()).view(p.shape)
        ds = (p * (dp - delta[:, :, :, i0:i1]) * r.d ** -0.5).flatten(2, 3)
        dq[:, :, :, i0:i1] = (ds @ k[:, :, 0, lo:i1].contiguous()).view(dq[:, :, :, i0:i1].shape)
        dk[:, :, 0, lo:i1] += ds.transpose(-1, -2).contiguous() @ q[:, :, :, i0:i1].flatten(2, 3)
        dv[:, :, 0, lo:i1] += p.flatten(2, 3).transpose(-1, -2).contiguous() @ dob
    return {"o": r.tokens(o, r.dtype), "lse": r.tokens(lse, torch.float32), "dq": r.tokens(dq, r.dtype),
            "dk": r.tokens(dk, r.dtype), "dv": r.tokens(dv, r.dtype)}


def _plain_tree(s):
    case = s["case"]
    B, T, hq, hkv, d, page = case["batch"], case["drafts"], case["hq"], case["hkv"], case["d"], case["page"]
    dev = s["q"].device
    starts, parents = s["starts"].long(), s["parents"].long()
    draft = torch.arange(T, device=dev)
    real = (parents >= -1) & (parents < draft)
    up = torch.where(real & (parents >= 0), parents, draft)        # a root and a padding place are their own
    sees = torch.eye(T, dtype=torch.bool, device=dev).expand(B, T, T).contiguous()
    far = torch.zeros(B, T, dtype=torch.long, device=dev)          # how many drafts lie above
    far += up != draft
    real = real & torch.gather(real, 1, up)
    hop = up
    for _ in range(max(1, (T - 1).bit_length())):                  # each round doubles the way that is known
        sees = sees | torch.gather(sees, 1, hop[:, :, None].expand(B, T, T))
        far = far + torch.gather(far, 1, hop)
        real = real & torch.gather(real, 1, hop)
        hop = torch.gather(hop, 1, hop)
    pos = torch.arange(max(s["lens"]) + T, device=dev)
    ids = s["table"].long()[:, pos // page].clamp(min=0)           # [B, tokens]
    held = pos < (starts + T)[:, None]
    ks = s["k_cache"][ids, pos % page].float().permute(0, 2, 3, 1).contiguous()
    vs = s["v_cache"][ids, pos % page].float().permute(0, 2, 1, 3).contiguous()
    rel = pos - starts[:, None]                                    # the draft at this place, negative in the context
    ctx = (rel < 0)[:, None, :].expand(B, T, -1)
    hit = torch.gather(sees, 2, rel.clamp(0, T - 1)[:, None, :].expand(B, T, -1)) & (rel >= 0)[:, None, :]
    if case["window"]:
        ctx = ctx & (far[:, :, None] - rel[:, None, :] < case["window"])
        hop = torch.gather(far, 1, rel.clamp(0, T - 1))
        hit = hit & (far[:, :, None] - hop[:, None, :] < case["window"])
    see = (ctx | hit) & held[:, None, :] & real[:, :, None]
    q = s["q"].float().view(B, T, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).contiguous()
    sc = (q.flatten(2, 3) @ ks).view(B, hkv, hq // hkv, T, -1) * d ** -0.5
    sc = sc.masked_fill(~see[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = (sc - top.clamp(min=-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ vs).view(q.shape) / total.clamp(min=1e-38)
    lse = (top + total.log()).squeeze(-1)
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(B, T, hq, d).to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, T, hq)}


def _plain_keep(s):
    case, page = s["case"], s["case"]["page"]
    path, starts = s["path"].long(), s["starts"].long()
    kept = (path >= 0).long().cumprod(1)
    src = starts[:, None] + path.clamp(min=0)
    dst = starts[:, None] + torch.arange(case["path"], device=path.device)
    src = torch.where(kept > 0, src, dst)                          # the rest stays where it is
    at = [(torch.gather(s["table"].long(), 1, x // page), x % page) for x in (src, dst)]
    s["k_cache"][at[1]] = s["k_cache"][at[0]]
    s["v_cache"][at[1]] = s["v_cache"][at[0]]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": (starts + kept.sum(1)).to(torch.int32)}


def _plain_pages(s):
    page, max_tokens = s["case"]["page"], s["max_tokens"]
    table, free, counts = s["table"], s["free"], s["counts"].long()
    width, pages = table.shape[1], free.shape[0]
    held = s["lengths"].long().clamp(0, width * page)
    have = (table >= 0) & (table < pages)
    # requests that end give their pages back
    gone = counts < 0
    back = (have & gone[:, None]).flatten()
    top = s["num_free"].long().clamp(0, pages)
    place = top + back.long().cumsum(0) - 1
    stack = torch.cat([free, free[:1]])
    stack[torch.where(back & (place < pages), place, torch.full_like(place, pages))] = table.flatten()
    free.copy_(stack[:pages])
    top = (top + back.sum()).clamp(max=pages)
    table = torch.where(gone[:, None], torch.full_like(table, -1), table)
    # the others take what they lack, in order
    new = counts.clamp(min=0)
    end = new.cumsum(0)
    fits = (new > 0) & (held + new <= width * page) & (end <= max_tokens)
    col = torch.arange(width, device=table.device)
    lack = (col >= (held // page)[:, None]) & (col < ((held + new + page - 1) // page)[:, None])
    lack = lack & fits[:, None] & ~have
    n = lack.sum(1)
    upto = n.cumsum(0)
    ok = fits & ((n == 0) | (upto <= top))
    lack = lack & ok[:, None]
    nth = (upto - n)[:, None] + lack.long().cumsum(1) - 1
    table = torch.where(lack, free[(top - 1 - nth).clamp(0, pages - 1)], table)
    s["table"].copy_(table)
    s["num_free"].copy_(top - (n * ok).sum())
    cu = torch.cat([end.new_zeros(1), end]).clamp(max=max_tokens)
    tok = torch.arange(max_tokens, device=table.device)
    row = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=len(counts) - 1)
    pos = (held[row] + tok - cu[row]).clamp(0, width * page - 1)
    at = table[row, pos // page].long()
    sure = (tok < cu[-1]) & ok[row] & (at >= 0) & (at < pages)
    slots = torch.where(sure, at * page + pos % page, torch.full_like(at, -1))
    lengths = torch.where(gone, torch.zeros_like(held), held + new * ok)
    return {"lengths": lengths.to(torch.int32), "cu": cu.to(torch.int32), "slots": slots, "table": s["table"],
            "free": free, "num_free": s["num_free"]}


_PLAIN = {"train": _plain_train, "prompt": _plain_prompt, "tree": _plain_tree, "keep": _plain_keep,
          "pages": _plain_pages}


# ------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    if case["op"] in ("keep", "pages"):
        return None  # copies and whole numbers
    s = prepare(case, seed)
    return _exact_tree(s) if case["op"] == "tree" else _exact_tokens(s)


def _exact_tokens(s):
    """Head by head, rows of softmax weights over the keys of each block of queries."""
    case = s["case"]
    train, win, group = case["op"] == "train", case["window"], case["hq"] // case["hkv"]
    flat = {n: s[n].flatten(0, 1).double() for n in ("q", "k", "v", "do") if n in s}
    out = {"o": torch.zeros_like(flat["q"]), "lse": torch.zeros_like(flat["q"][..., 0])}
    if train:
        out.update({"d" + n: torch.zeros_like(flat[n]) for n in ("q", "k", "v")})
    first = 0
    for n in s["lens"]:
        at = torch.arange(first, first + n, device=s["q"].device)
        for h in range(case["hq"]):
            key, val = flat["k"][at, h // group], flat["v"][at, h // group]
            for i in range(0, n, 2048):
                rows = at[i:i + 2048]
                ask = flat["q"][rows, h]
                a, b = (max(0, i + 1 - win) if win else 0), min(n, i + 2048)
                sc = torch.mm(ask, key[a:b].t()) / math.sqrt(case["d"])
                gap = rows[:, None] - at[None, a:b]
                seen = gap >= 0
                if win:
                    seen &= gap < win
                lse = torch.logsumexp(torch.where(seen, sc, -math.inf), 1)
                wt = torch.where(seen, (sc - lse[:, None]).exp(), 0.0)
                o = torch.mm(wt, val[a:b])
                out["lse"][rows, h], out["o"][rows, h] = lse, o
                if train:
                    do = flat["do"][rows, h]
                    dsc = wt * torch.mm(do, val[a:b].t())
                    dsc = (dsc - wt * dsc.sum(1, keepdim=True)) / math.sqrt(case["d"])
                    out["dq"][rows, h] = torch.mm(dsc, key[a:b])
                    out["dk"][at[a:b], h // group] += torch.mm(dsc.t(), ask)
                    out["dv"][at[a:b], h // group] += torch.mm(wt.t(), do)
        first += n
    lead = s["q"].shape[:2]
    return {n: x.view(*lead, *x.shape[1:]) for n, x in out.items()}


def _exact_tree(s):
    """Draft by draft, over the places of the context and of the drafts above it."""
    case = s["case"]
    B, T, hq, hkv, d, page = case["batch"], case["drafts"], case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, T, hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, (n, parents) in enumerate(zip(s["lens"], s["parents"].tolist())):
        pos = torch.arange(n + T, device=out.device)
        rows = s["table"][b].long()[pos // page]
        keys = s["k_cache"][rows, pos % page].double().permute(1, 2, 0).contiguous()
        vals = s["v_cache"][rows, pos % page].double().transpose(0, 1).contiguous()
        for i in range(T):
            line, x = [], i
            while -1 < x < T and parents[x] < x and parents[x] >= -1:
                line.append(x)
                x = parents[x]
            if x != -1:
                continue  # padding
            if case["window"]:
                line, left = line[:case["window"]], max(0, case["window"] - len(line))
                ctx = list(range(max(0, n - left), n)) if left else []
            else:
                ctx = None
            seen = torch.tensor([n + y for y in line], device=out.device)
            seen = torch.cat([pos[:n] if ctx is None else torch.tensor(ctx, dtype=torch.long, device=out.device), seen])
            ask = s["q"][b, i].double().view(hkv, hq // hkv, d)
            sc = torch.matmul(ask, keys[:, :, seen]) / math.sqrt(d)
            top = torch.logsumexp(sc, -1)
            lse[b, i] = top.flatten()
            out[b, i] = torch.matmul((sc - top[..., None]).exp(), vals[:, seen]).reshape(hq, d)
    return {"o": out, "lse": lse}
