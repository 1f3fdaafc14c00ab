"""Prompt and decoding of a hybrid decoder's two mixers together (GPU): the chunked forward fills the
states and the writer the cache, then every token takes a recurrent step, whose output is the query
of the attention over the cache, all of it one captured graph.

Tolerances as in the operators' own tests: each is compared with fp64 on the inputs that it got."""
import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import mixer_refs as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_decode(dtype, captured):
    hk, hv, d, hkv, page, steps = 2, 4, 64, 2, 16, 4
    lens = [70, 0, 16, 129]
    B, total = len(lens), sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    gen = torch.Generator().manual_seed(40)
    rnd = lambda *s: torch.randn(*s, generator=gen)

    def tokens(lead, n):
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        x = dict(q=unit(rnd(lead, n, hk, d)), k=unit(rnd(lead, n, hk, d)), v=rnd(lead, n, hv, d),
                 g=-rnd(lead, n, hv).abs() * 0.2, beta=torch.sigmoid(rnd(lead, n, hv)),
                 ck=rnd(lead, n, hkv, d), cv=rnd(lead, n, hkv, d))
        return {m: t.to(dtype).cuda() for m, t in x.items()}

    names = ("q", "k", "v", "g", "beta")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    prompt, new = tokens(1, total), tokens(B, steps)
    # the cache, pages handed out in any order, and the states' pool with slots in any order
    width = 12
    order = torch.randperm(B * width, generator=gen).tolist()
    table = [order[width * b:width * (b + 1)] for b in range(B)]
    kc, vc = (torch.full((B * width, page, hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    slots, dev, held = ints([5, 2, 0, 3]), ints(table), ints(lens)
    state = torch.randn(6, hv, d, d, device="cuda")
    # ---- prompt
    o, ht, _ = g2.gdr2_scalar_fwd(*[prompt[m] for m in names], cu_seqlens=ints(cu))
    state[slots.long()] = ht
    g2.gdr2_kv_append(prompt["ck"][0], prompt["cv"][0], kc, vc, dev, torch.zeros_like(held), cu_seqlens=ints(cu))
    # ---- decoding, from one token's buffers
    buf = {m: torch.empty_like(t[:, :1]) for m, t in new.items()}
    mix, out = torch.empty(B, 1, hv, d, dtype=dtype, device="cuda"), torch.empty(B, hv, d, dtype=dtype, device="cuda")

    def step():
        g2.gdr2_scalar_step(*[buf[m] for m in names], state, slots=slots, o=mix)
        g2.gdr2_kv_append(buf["ck"][:, 0], buf["cv"][:, 0], kc, vc, dev, held)
        held.add_(1)
        g2.gdr2_attn_step(mix[:, 0], kc, vc, dev, held, o=out)

    graph = None
    if captured:
        before = state.clone()
        for m in buf:
            buf[m].copy_(new[m][:, :1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        state.copy_(before)
        held.copy_(ints(lens))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    mixes, tok, att = [o], 2.0 ** -7 if dtype == BF else 1e-5, 2.0 ** -7 if dtype == BF else 1e-5
    for t in range(steps):
        for m in buf:
            buf[m].copy_(new[m][:, t:t + 1])
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        mixes.append(mix.clone())
        want, _ = ref.attention(mix[:, 0], kc, vc, table, [n + t + 1 for n in lens], d ** -0.5, 0)
        assert held.tolist() == [n + t + 1 for n in lens]
        assert ref.normwise(out, want) <= att, t
    # what the cache holds is what was appended, and the recurrence saw prompt and tokens as one sequence
    for b, n in enumerate(lens):
        rows = [(table[b][i // page], i % page) for i in range(n + steps)]
        keys = torch.stack([kc[r] for r in rows])
        assert torch.equal(keys, torch.cat([prompt["ck"][0, cu[b]:cu[b + 1]], new["ck"][b]]))
        whole = {m: torch.cat([prompt[m][0, cu[b]:cu[b + 1]], new[m][b]])[None] for m in names}
        want = ref.run_recurrence(dict(whole, h0=None), None)
        got = torch.cat([mixes[0][0, cu[b]:cu[b + 1]], *[x[b] for x in mixes[1:]]])
        assert ref.normwise(got, want["o"][0]) <= tok, b
        assert ref.normwise(state[slots[b].long()][None], want["ht"]) <= 1e-5, b
