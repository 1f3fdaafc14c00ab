"""Causal attention over whole sequences, forward and backward, against fp64 (GPU).

Tolerances, set before the first run. fp32: 1e-5 normwise, the library's. bf16, element by element: a rounding is off
by at most 2^-8 of the value. o: its own rounding, and that of every weight, 2^-8 of sum p |v| / sum p. dv: its own and
that of every weight, 2^-8 of sum P |dO|. dq and dk: their own and that of every dS, 2^-8 of sum |dS| |k|; delta is off
by the 2^-16 of |dO| |o| that o and rest together leave out, times sum P |k|. Scores, statistics and sums are fp32: a
score is off by at most 2^-24 (D + 3) |q| |k| scale, a weight by that of it, and so are the sums; FP below covers both
at the sizes here (|q||k| scale < 30, sums of at most 2^12 terms): 2^-24 (131 * 30 + 2^12) < 2^-10.9 of the terms'
sizes. lse: 1e-5 relative and absolute, as for the step."""
import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import mixer_refs
import prompt_refs as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FP = 2.0 ** -10.9
R8 = 2.0 ** -8


def normwise(a, b):
    return mixer_refs.normwise(a, b.cpu())


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def bounds(lens, lead=0):
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def make(tokens, Hq, Hkv, D, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda h: torch.randn(1, tokens, h, D, generator=gen).to(dtype).cuda()
    return r(Hq), r(Hkv), r(Hkv), r(Hq)


def near(got, want, size, dtype, name, extra=0.0):
    got, d = got.double(), (got.double() - want).abs()
    assert torch.isfinite(got).all(), name
    if dtype == F32:
        assert normwise(got, want) <= 1e-5, name
    else:
        room = R8 * want.abs() + (1 + R8) * ((R8 + FP) * size + extra) + 1e-30
        assert (d <= room).all(), (name, (d / room).max())


def check(q, k, v, do, cu, window=0, scale=None, packed=True, alike=False):
    sc = q.shape[3] ** -0.5 if scale is None else scale
    kw = dict(cu_seqlens=ints(cu) if packed else None, scale=scale, window=window)
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, save_for_bwd=True, **kw)
    assert torch.equal(o, g2.gdr2_attn_fwd(q, k, v, **kw))
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, **kw)
    qf, kf, vf, df = (x.flatten(0, 1) for x in (q, k, v, do))
    wo, wl, size = ref.attention(qf, kf, vf, cu, sc, window)
    near(o.flatten(0, 1), wo, size, q.dtype, "o")
    assert ((lse.flatten(0, 1).double() - wl).abs() <= 1e-5 * wl.abs().clamp(min=1.0)).all()
    if rest is not None:  # o to 16 bits, but for the weights' rounding
        assert ((o.double() + rest.double()).flatten(0, 1) - wo).abs().le((R8 + FP) * size + 2.0 ** -16 * wo.abs() + 1e-30).all()
    dq, dk, dv, sq, sk, sv, pq, pk = ref.gradients(qf, kf, vf, df, cu, sc, window)
    # an error of delta of row i, and of its weights in o, times its weights
    off = (2.0 ** -16 + R8) * float((df.double().abs() * size).sum(-1).max()) if q.dtype == BF else 0.0
    near(gr["dq"].flatten(0, 1), dq, sq, q.dtype, "dq", off * pq)
    near(gr["dk"].flatten(0, 1), dk, sk, q.dtype, "dk", off * pk)
    near(gr["dv"].flatten(0, 1), dv, sv, q.dtype, "dv")
    if q.dtype == BF:  # and with roundings that are not all alike, normwise: two of them
        # (alike: keys that have most of their size in common. The dS of a row sum to zero, so of sum dS k that part
        # cancels, and of the roundings of dS, 2^-8 |dS| |k|, it does not: dq is held to the bound above alone)
        for a, b in ((o, wo), (gr["dv"], dv)) if alike else ((o, wo), (gr["dq"], dq), (gr["dk"], dk), (gr["dv"], dv)):
            if float(b.norm()):
                assert normwise(a.flatten(0, 1), b) <= 2.0 ** -7
    return o, lse, rest, gr


LENGTHS = [[2], [31, 32, 33], [64, 0, 1, 127, 128, 129], [255, 256, 257, 3], [700], [1, 2, 3, 0, 5] * 9, [1500, 40]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", range(len(LENGTHS)))
def test_lengths(dtype, D, n):
    cu = bounds(LENGTHS[n])
    check(*make(cu[-1], 4, 2, D, dtype, seed=n), cu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (24, 8), (40, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(dtype, heads, D):
    cu = bounds([70, 5, 333])
    check(*make(cu[-1], *heads, D, dtype, seed=3), cu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [2, 31, 32, 33, 64, 100, 257, 5000])
def test_window(dtype, window):
    cu = bounds([300, 1, 0, 33, 99, 100, 101, 640])
    check(*make(cu[-1], 6, 3, 64, dtype, seed=5), cu, window=window)


@pytest.mark.parametrize("lens,heads,window", [([1024] * 4, (32, 32), 0), ([1500, 1, 2047], (40, 8), 0), ([1100, 1300], (64, 2), 300),
                                               ([1, 3000, 130], (48, 48), 0), ([2200], (64, 64), 70)])
def test_long_sequences_of_many_heads(lens, heads, window):
    # enough work that waves take turns on it
    cu = bounds(lens)
    q, k, v, do = make(cu[-1], *heads, 128, BF, seed=30)
    packed = check(q, k, v, do, cu, window=window)
    again = check(q, k, v, do, cu, window=window)
    assert all(torch.equal(a, b) for a, b in zip(packed[:3], again[:3]))
    assert all(torch.equal(packed[3][n], again[3][n]) for n in packed[3])
    if len(set(lens)) == 1:
        check(*(x.view(len(lens), lens[0], -1, 128) for x in (q, k, v, do)), cu, window=window, packed=False)


@pytest.mark.parametrize("lens,heads,D", [([2], (2, 1), 64), ([2] * 12, (2, 2), 128), ([3, 1, 4, 2, 0, 64], (3, 1), 128),
                                          ([40], (2, 1), 64), ([63, 64], (16, 4), 64), ([10] * 30, (8, 8), 128)])
def test_short_sequences_carry_one_rounding(lens, heads, D):
    # Weights and their gradients enter the products in two bf16 parts, off by 2^-8 of what one part's 2^-8 left: 2^-16;
    # delta by as much of its terms from the weights in o, and again from o and rest. Then each result is rounded once.
    q, k, v, do = make(sum(lens), *heads, D, BF, seed=25)
    cu, sc = bounds(lens), D ** -0.5
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu))
    qf, kf, vf, df = (x.flatten(0, 1) for x in (q, k, v, do))
    wo, _, size = ref.attention(qf, kf, vf, cu, sc, 0)
    dq, dk, dv, sq, sk, sv, pq, pk = ref.gradients(qf, kf, vf, df, cu, sc, 0)
    off = 2.0 ** -15 * float((df.double().abs() * size).sum(-1).max())
    for got, want, terms, extra in ((o, wo, size, 0.0), (gr["dq"], dq, sq, off * pq), (gr["dk"], dk, sk, off * pk),
                                    (gr["dv"], dv, sv, 0.0)):
        room = R8 * want.abs() + (1 + R8) * ((2.0 ** -16 + FP) * terms + extra) + 1e-30
        assert ((got.flatten(0, 1).double() - want).abs() <= room).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_token_rows(dtype):
    # a token that sees itself only: o = v and lse its score, and gradients that are dO and (but for fp32's roundings
    # of dP - delta, 2^-24 (2 D) |dO| |v| |k| scale) nothing. In fp32 o = (p v) / p rounds three times, the product, the
    # reciprocal and the product with it, by 2^-24 each; in bf16 p enters the product as 1 and o rounds back to v.
    for cu, window in ((bounds([1] * 40), 0), (bounds([40]), 1)):
        q, k, v, do = make(40, 4, 2, 64, dtype, seed=6)
        o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), window=window, save_for_bwd=True)
        gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu), window=window)
        vv = v.double().repeat_interleave(2, dim=2)
        assert ((o.double() - vv).abs() <= (3.01 * 2.0 ** -24 if dtype == F32 else 0.0) * vv.abs()).all()
        s = (q.double() * k.double().repeat_interleave(2, dim=2)).sum(-1) * 0.125
        assert (lse.double() - s).abs().max() <= 1e-5 * s.abs().max()
        dv = do.double().view(1, 40, 2, 2, 64).sum(3)
        # a weight of one, off by lse's roundings on the way: three of 2^-24 of |lse| log2(e) < 8 here
        assert (gr["dv"].double() - dv).abs().max() <= (2.0 ** -8 if dtype == BF else 2e-6) * do.double().abs().max() * 2
        room = 2.0 ** -24 * 128 * float(do.double().norm(dim=-1).max() * v.double().norm(dim=-1).max()) * 0.125
        assert gr["dq"].double().abs().max() <= room * float(k.double().abs().max()) * 2
        assert gr["dk"].double().abs().max() <= room * float(q.double().abs().max()) * 4


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 64, 100, 513])
def test_sequences_of_one_length(dtype, T):
    q, k, v, do = (x.view(3, T, -1, 64) for x in make(3 * T, 4, 2, 64, dtype, seed=7))
    if T == 1:
        vv = v.double().repeat_interleave(2, dim=2)  # as in test_one_token_rows
        assert ((g2.gdr2_attn_fwd(q, k, v).double() - vv).abs() <= 3.01 * 2.0 ** -24 * vv.abs()).all()
        return
    o, lse, rest, gr = check(q, k, v, do, bounds([T] * 3), packed=False)
    flat = lambda x: x.reshape(1, 3 * T, *x.shape[2:])
    kw = dict(cu_seqlens=ints(bounds([T] * 3)))
    o2, lse2, rest2 = g2.gdr2_attn_fwd(flat(q), flat(k), flat(v), save_for_bwd=True, **kw)
    assert torch.equal(flat(o), o2) and torch.equal(flat(lse), lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_of_a_projection(dtype):
    gen = torch.Generator().manual_seed(8)
    qkv = torch.randn(2, 90, 4 + 2 + 2, 64, generator=gen).to(dtype).cuda()
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    do = torch.randn(2, 90, 4, 64, generator=gen).to(dtype).cuda()
    a = check(q, k, v, do, bounds([90, 90]), packed=False)
    b = check(q.contiguous(), k.contiguous(), v.contiguous(), do, bounds([90, 90]), packed=False)
    assert all(torch.equal(x, y) for x, y in zip(a[:2], b[:2])) and all(torch.equal(a[3][n], b[3][n]) for n in a[3])
    heads_first = torch.randn(1, 4, 130, 64, generator=gen).to(dtype).cuda()
    x = heads_first.transpose(1, 2)  # heads outside tokens in memory
    check(x, x, x, torch.randn(1, 130, 4, 64, generator=gen).to(dtype).cuda(), [0, 100, 130])
    for bad in (qkv[:, :, :4, ::2], qkv[:, ::2][:, :, :4]):
        with pytest.raises((ValueError, RuntimeError)):
            g2.gdr2_attn_fwd(bad, k, v)
    odd = torch.randn(1, 90, 4 * 64 + 1, device="cuda").to(dtype)[:, :, :256].unflatten(2, (4, 64))
    with pytest.raises(RuntimeError):
        g2.gdr2_attn_fwd(odd, odd, odd)  # rows that are no whole 16-byte pieces apart


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 0.01, 1.0])
def test_scales(dtype, scale):
    q, k, v, do = make(150, 4, 2, 64, dtype, seed=9)
    if scale:
        check(q * 0.25, k, v, do, [0, 90, 150], scale=scale, window=40)
        return
    o = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints([0, 90, 150]), scale=0.0)
    wo, _, size = ref.attention(q[0], k[0], v[0], [0, 90, 150], 0.0)
    near(o[0], wo, size, dtype, "o")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores(dtype):
    # scores of some hundreds: the weights underflow but for a few, and no exponential overflows
    q, k, v, do = make(200, 2, 2, 64, dtype, seed=10)
    o, lse = g2.gdr2_attn_fwd(q, k, v, scale=20.0, return_lse=True)
    wo, wl, _ = ref.attention(q[0], k[0], v[0], [0, 200], 20.0)
    # a score of size s is off by up to 2^-23 s, and a weight by that times itself
    tol = (2.0 ** -7 if dtype == BF else 1e-5) + 2.0 ** -22 * float(wl.abs().max())
    assert normwise(o[0], wo) <= tol and (lse[0].double() - wl).abs().max() <= 1e-5 * wl.abs().max()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_rising_maximum(dtype):
    # keys that each outdo the ones before them: the running reference moves at every tile, and by 8 at a time
    n = 400
    q, k, v, do = make(n, 2, 1, 64, dtype, seed=11)
    q[..., 0], k[..., 0] = 8.0, (torch.arange(n) / 4.0).to(dtype).cuda()[None, :, None]
    check(q * 0.25, k, v, do, [0, n], scale=0.125, alike=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_no_sequence(dtype):
    cu = [40, 75, 75, 140]
    q, k, v, do = make(333, 4, 2, 64, dtype, seed=12)
    for x in (q, k, v, do):
        x[:, :40] = float("nan")
        x[:, 140:] = float("inf")
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu))
    inner = slice(40, 140)
    part = check(*(x[:, inner].contiguous() for x in (q, k, v, do)), [0, 35, 35, 100])
    for a, b in ((o, part[0]), (lse, part[1]), *((gr[n], part[3][n]) for n in gr)):
        assert torch.equal(a[:, inner], b)
        assert (a[:, :40] == 0).all() and (a[:, 140:] == 0).all()
    # tensors of the caller's keep what they hold there
    mine = torch.full_like(o, 7.0)
    mygr = {n: torch.full_like(x, 7.0) for n, x in gr.items()}
    g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), o=mine)
    g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu), grads=mygr)
    for a, b in ((mine, o), *((mygr[n], gr[n]) for n in gr)):
        assert torch.equal(a[:, inner], b[:, inner]) and (a[:, :40] == 7).all() and (a[:, 140:] == 7).all()


def test_no_tokens_and_no_sequences():
    e = torch.empty(1, 0, 4, 64, dtype=BF, device="cuda")
    assert g2.gdr2_attn_fwd(e, e, e).numel() == 0
    assert g2.gdr2_attn_fwd(e, e, e, cu_seqlens=ints([0, 0, 0])).numel() == 0
    x = torch.randn(1, 9, 4, 64, device="cuda")
    o, lse, rest = g2.gdr2_attn_fwd(x, x, x, cu_seqlens=ints([0]), save_for_bwd=True)
    assert rest is None and not o.any() and not lse.any()
    gr = g2.gdr2_attn_bwd(x, x, x, o, lse, x, cu_seqlens=ints([0]))
    assert not any(t.any() for t in gr.values())
    o = g2.gdr2_attn_fwd(x, x, x, cu_seqlens=ints([3, 3]))
    assert not o.any()


def test_other_sequences_keep_clear_of_nan():
    cu = [0, 50, 120, 200]
    q, k, v, do = make(200, 4, 2, 64, BF, seed=13)
    want = check(q, k, v, do, cu)
    for x in (q, k, v, do):
        x[:, 50:120] = float("nan")
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu))
    for a, b in ((o, want[0]), (lse, want[1]), *((gr[n], want[3][n]) for n in gr)):
        assert torch.equal(a[:, :50], b[:, :50]) and torch.equal(a[:, 120:], b[:, 120:])


def test_bounds_out_of_order_stay_inside():
    q, k, v, do = make(300, 4, 2, 64, BF, seed=14)
    for cu in ([5, 90, 40, 300], [-7, 2 ** 31 - 1, 12], [300, 300, 0], [290, 1000, 1000, 2000]):
        o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), save_for_bwd=True)
        gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu))
        assert o.shape == q.shape and gr["dk"].shape == k.shape
    torch.cuda.synchronize()


def test_repeats_streams_and_calls_at_once():
    cu = bounds([300, 17, 513])
    args = make(cu[-1], 8, 2, 128, BF, seed=15)
    want = check(*args, cu)
    q, k, v, do = args
    s = [torch.cuda.Stream() for _ in range(2)]
    c = ints(cu)
    torch.cuda.synchronize()
    outs = []
    for x in s * 2:
        o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=c, save_for_bwd=True, stream=x)
        outs.append((o, lse, rest, g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=c, stream=x)))
        torch.empty(1 << 20, device="cuda").fill_(float("nan"))  # freed memory is used again on the current stream
    torch.cuda.synchronize()
    for o, lse, rest, gr in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(rest, want[2])
        assert all(torch.equal(gr[n], want[3][n]) for n in gr)


def test_a_captured_step_is_replayed():
    cu = bounds([200, 64, 1, 100])
    args = make(cu[-1], 4, 1, 64, BF, seed=16)
    q, k, v, do = args
    c = ints(cu)
    want = check(*args, cu)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    gr = {n: torch.empty_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    ws = torch.empty(g2.gdr2_attn_bwd_workspace_bytes(4, cu[-1], 4, 1, 64, True), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=c, o=o, lse=lse, save_for_bwd=True)
        g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=c, grads=gr, ws=ws)
    for _ in range(3):
        for x in (o, lse, rest, ws, *gr.values()):
            x.fill_(77)
        check(*args, cu)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert all(torch.equal(gr[n], want[3][n]) for n in gr)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd(dtype):
    cu = [0, 61, 130]
    q, k, v, do = make(130, 4, 2, 64, dtype, seed=17)
    want = check(q, k, v, do, cu, window=50)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = g2.GDR2AttnFunction.apply(*leaves, ints(cu), None, 50)
    o.backward(do)
    assert torch.equal(o, want[0])
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(x.grad, want[3][n])
    with torch.no_grad():
        assert torch.equal(g2.GDR2AttnFunction.apply(*leaves, ints(cu), None, 50), want[0])
    with torch.inference_mode():
        assert torch.equal(g2.GDR2AttnFunction.apply(*leaves, ints(cu), None, 50), want[0])
    # one key head for all, broadcast: its gradient is the sum over the heads
    one = torch.randn(1, 130, 1, 64, device="cuda", dtype=F32).to(dtype).requires_grad_()
    g2.GDR2AttnFunction.apply(q, one.expand(1, 130, 4, 64), v.repeat_interleave(2, dim=2), ints(cu)).backward(do)
    wide = one.detach().expand(1, 130, 4, 64).contiguous().requires_grad_()
    g2.GDR2AttnFunction.apply(q, wide, v.repeat_interleave(2, dim=2), ints(cu)).backward(do)
    s = wide.grad.double().sum(2, keepdim=True)
    # torch adds the four heads in its type: three sums
    tol = 3 * (2.0 ** -8 if dtype == BF else 2.0 ** -24)
    assert (one.grad.double() - s).abs().max() <= tol * wide.grad.double().abs().sum(2).max()


def test_gradients_against_differences():
    # fp32, along random directions u: <grad, u> against central differences of L(x) = <o(x), do> with steps h and
    # h / 2, extrapolated. The differences' own error: o's, 1e-6 of |o| |do| (the fp32 roundings), 2 / h of it, times 3
    # for the extrapolation, and the fifth derivative's h^4 / 480, of scores that a step changes by less than one:
    # together less than 1e-3 of |do| |o| at h = 1/32.
    q, k, v, do = make(70, 4, 2, 64, F32, seed=18)
    c = ints([0, 33, 70])
    f = lambda a, b, d: (g2.gdr2_attn_fwd(a, b, d, cu_seqlens=c, window=20).double() * do.double()).sum()
    o, lse, _ = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=c, window=20, save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, cu_seqlens=c, window=20)
    room = 1e-3 * float(o.double().norm() * do.double().norm())
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, n in enumerate(("dq", "dk", "dv")):
        for _ in range(4):
            x = [q, k, v]
            u = torch.randn(x[i].shape, generator=gen, device="cuda") * 0.1

            def slope(h):
                hi, lo = list(x), list(x)
                hi[i], lo[i] = x[i] + h * u, x[i] - h * u
                return (f(*hi) - f(*lo)) / (2 * h)

            d = (4 * slope(1 / 64) - slope(1 / 32)) / 3
            assert abs(float(d - (gr[n].double() * u.double()).sum())) <= room, n


def test_a_captured_backward_of_leaves_in_another_graph_is_refused():
    leaves = [x.requires_grad_() for x in make(40, 2, 2, 64, BF, seed=19)[:3]]
    do = torch.ones(1, 40, 2, 64, dtype=BF, device="cuda")
    alive = g2.GDR2AttnFunction.apply(*leaves)
    pool = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="cannot capture"):
        with torch.cuda.graph(graph, stream=pool):
            o = g2.GDR2AttnFunction.apply(*leaves)
            torch.autograd.grad(o, leaves, do)
    del alive


def test_offsets_past_32_bits():
    T, H, D = 1_050_400, 16, 128  # 2.2e9 elements of q, o, dq
    lens = [200, 0, 130]
    cu = bounds(lens, T - 400)
    n = cu[-1] - cu[0]
    small = make(n, H, H // 8, D, BF, seed=20)
    want = check(*small, bounds(lens))
    big = []
    for x in small:
        y = torch.zeros(1, T, *x.shape[2:], dtype=BF, device="cuda")
        y[:, cu[0]:cu[-1]] = x
        big.append(y)
    q, k, v, do = big
    c = ints(cu)
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=c, save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=c)
    # (how waves share the work goes by the call's sizes, and with it the order of sums: two results within 2^-7 each)
    for a, b in ((o, want[0]), (lse, want[1]), *((gr[x], want[3][x]) for x in gr)):
        assert normwise(a[:, cu[0]:cu[-1]].double(), b.double()) <= 2.0 ** -6
        assert not a[:, :cu[0]].any() and not a[:, cu[-1]:].any()


def test_token_strides_past_32_bits():
    T, far = 70, 5 << 26  # 640 MiB from token to token: of 8 rows, 7 strides pass 32 bits
    q, k, v, do = make(T, 4, 2, 64, BF, seed=22)
    want = check(q, k, v, do, [0, T])
    room = torch.empty(T * far, dtype=BF, device="cuda").view(1, T, far)[:, :, :4 * 64].unflatten(2, (4, 64))
    room[:, :, :2] = k
    room[:, :, 2:] = v
    got = check(q, room[:, :, :2], room[:, :, 2:], do, [0, T])
    assert all(torch.equal(x, y) for x, y in zip(want[:3], got[:3])) and all(torch.equal(want[3][n], got[3][n]) for n in want[3])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_token_of_each_sequence(dtype):
    q, k, v, do = (x.view(3, 50, -1, 64) for x in make(150, 4, 2, 64, dtype, seed=23))
    one = [x[:, 7:8] for x in (q, k, v)]
    assert torch.equal(g2.gdr2_attn_fwd(*one), g2.gdr2_attn_fwd(*(x.contiguous() for x in one)))


def test_refusals():
    q, k, v, do = make(20, 4, 2, 64, BF, seed=21)
    f = g2.gdr2_attn_fwd
    o, lse, rest = f(q, k, v, save_for_bwd=True)
    for bad in ((q, k.float(), v), (q, k, v[:, :10]), (q, k[:, :, :1], v), (q.half(), k.half(), v.half()), (q[0], k, v),
                (q.cpu(), k.cpu(), v.cpu()), (q, k.cpu(), v)):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(RuntimeError):
        f(q[:, :, :3].contiguous(), k, v)  # heads that do not divide
    with pytest.raises(RuntimeError):
        f(*(x[..., :32].contiguous() for x in (q, k, v)))
    for kw in (dict(window=-1), dict(window=-2 ** 32 + 5), dict(scale=float("inf")), dict(scale=float("nan"))):
        with pytest.raises(RuntimeError):
            f(q, k, v, **kw)
    with pytest.raises(ValueError):
        f(q.view(2, 10, 4, 64), k.view(2, 10, 2, 64), v.view(2, 10, 2, 64), cu_seqlens=ints([0, 10]))
    with pytest.raises(ValueError):
        f(q, k, v, cu_seqlens=torch.tensor([0, 20]).cuda())
    b = g2.gdr2_attn_bwd
    with pytest.raises(ValueError):
        b(q, k, v, o, lse.half(), do)
    with pytest.raises(ValueError):
        b(q, k, v, o, lse, do.transpose(1, 2))
    with pytest.raises(ValueError):
        b(q, k, v, o, lse, do, grads={"dq": q})
    with pytest.raises(RuntimeError):
        b(q, k, v, o, lse, do, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert torch.equal(f(q, k, v, window=2 ** 32 + 5), o)


MANY = [(1, (1, 1), 64, 127), (1, (4, 2), 64, 128), (1, (4, 2), 128, 126), (1, (4, 2), 128, 256), (1, (2, 1), 128, 65),
        (1, (2, 1), 64, 512), (1, (8, 8), 128, 320), (1, (2, 1), 128, 4096), (8, (4, 4), 64, 190), (40, (2, 2), 128, 127)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("longer,heads,D,N", MANY)
def test_more_sequences_than_lanes(dtype, longer, heads, D, N):
    # A slot's sequence is searched by 64 probes at a time, the last of which is a sequence where N > 63 ceil(N / 64).
    # Outputs of the caller's, so that rows that nothing is written to show.
    lens = [longer * ((5 * i) % 23 + (60 if i % 17 == 3 else 0)) for i in range(N - 1)] + [9]
    cu = bounds(lens)
    args = make(cu[-1], *heads, D, dtype, seed=40)
    q, k, v, do = args
    c = ints(cu)
    full = lambda x: torch.full_like(x, float("nan"))
    o, lse, gr = full(q), full(q[..., 0].float()), {n: full(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    ws = torch.full((g2.gdr2_attn_bwd_workspace_bytes(N, cu[-1], *heads, D, True, g2._DT[dtype]),), 255, dtype=torch.uint8, device="cuda")
    _, _, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=c, o=o, lse=lse, save_for_bwd=True)
    g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=c, grads=gr, ws=ws)
    want = check(*args, cu)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert all(torch.equal(gr[n], want[3][n]) for n in gr)


def test_long_sequences_more_than_lanes():
    # 256 queries a workgroup
    lens = [1030 + i % 5 for i in range(127)] + [300]
    cu = bounds(lens)
    check(*make(cu[-1], 2, 1, 128, BF, seed=41), cu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,heads,D", [(33, (3, 1), 64), (45, (5, 1), 128), (7, (9, 3), 64)])
def test_odd_numbers_of_rows(dtype, T, heads, D):
    # parts of dK and dV behind an odd number of rows of the workspace, and nothing behind its end
    args = make(T, *heads, D, dtype, seed=44)
    q, k, v, do = args
    o, lse, rest, gr = check(*args, [0, T])
    n = g2.gdr2_attn_bwd_workspace_bytes(1, T, *heads, D, True, g2._DT[dtype])
    room = torch.full((n + 256,), 93, dtype=torch.uint8, device="cuda")
    again = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints([0, T]), ws=room[:n])
    assert all(torch.equal(again[x], gr[x]) for x in gr) and (room[n:] == 93).all()


@pytest.mark.parametrize("cu", [[0], [3, 3], [9, 9, 9]])
def test_rows_of_no_sequence_in_an_lse_of_the_callers(cu):
    x = torch.randn(1, 9, 4, 64, device="cuda")
    for own in (True, False):  # zero where o is allocated here, else left as they are
        o, lse = torch.full_like(x, 7.0), torch.full((1, 9, 4), 7.0, device="cuda")
        got = g2.gdr2_attn_fwd(x, x, x, cu_seqlens=ints(cu), o=None if own else o, lse=lse)
        assert got[1] is lse and all((t == (0 if own else 7)).all() for t in got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,scale", [(60, 2.0 ** -123), (60, -2.0 ** -123), (61, 2.0 ** -125), (50, 2.0 ** -103)])
def test_small_scales_of_large_scores(dtype, n, scale):
    # powers of two that come out again: bit for bit what scores of the usual size give
    cu = [0, 80, 90]
    q, k, v, do = make(90, 4, 2, 64, dtype, seed=41)
    kw = dict(cu_seqlens=ints(cu))
    f = 2.0 ** n
    want = g2.gdr2_attn_fwd(q, k, v, scale=scale * f * f, save_for_bwd=True, **kw)
    got = g2.gdr2_attn_fwd(q * f, k * f, v, scale=scale, save_for_bwd=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
    a = g2.gdr2_attn_bwd(q, k, v, want[0], want[1], do, rest=want[2], scale=scale * f * f, **kw)
    b = g2.gdr2_attn_bwd(q * f, k * f, v, want[0], want[1], do, rest=want[2], scale=scale, **kw)
    assert torch.equal(a["dv"], b["dv"]) and all(torch.equal(a[x], b[x] * f) for x in ("dq", "dk"))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, 1e-45, -1e-41])
def test_scales_of_nothing(dtype, scale):
    cu = [0, 150, 260]
    q, k, v, do = make(260, 4, 2, 64, dtype, seed=42)
    kw = dict(cu_seqlens=ints(cu), scale=scale, window=100)
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, save_for_bwd=True, **kw)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, **kw)
    wo, wl, size = ref.attention(q[0], k[0], v[0], cu, scale, 100)
    near(o[0], wo, size, dtype, "o")
    assert ((lse[0].double() - wl).abs() <= 1e-5 * wl.abs().clamp(min=1.0)).all()
    _, _, dv, _, _, sv, _, _ = ref.gradients(q[0], k[0], v[0], do[0], cu, scale, 100)
    near(gr["dv"][0], dv, sv, dtype, "dv")
    # the others are the scale times sums of at most 110 terms below 2^16: denormal numbers, which keep few or no bits
    for x in ("dq", "dk"):
        assert (gr[x].double().abs() <= abs(scale) * 2.0 ** 23 + 2.0 ** -133).all()


FEW = [([300] * 3, (4, 4), 64, 0), ([700, 200, 1000], (16, 4), 128, 0), ([1100] * 4, (32, 32), 128, 0), ([400] * 40, (8, 8), 128, 0),
       ([500] * 5, (12, 3), 64, 40), ([1024] * 4, (32, 32), 128, 64), ([4096], (1, 1), 128, 0), ([90] * 100, (16, 2), 64, 0)]


@pytest.mark.parametrize("lens,heads,D,window", FEW)
def test_first_tokens_carry_one_rounding_in_any_batch(lens, heads, D, window):
    # o as in test_short_sequences_carry_one_rounding: of the first 64 tokens, or with a window of at most 64 of all
    q, k, v, do = make(sum(lens), *heads, D, BF, seed=43)
    cu = bounds(lens)
    o, _, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), window=window, save_for_bwd=True)
    for a, n in zip(cu[:6], lens):
        at = slice(a, a + (n if window else min(n, 64)))
        wo, _, size = ref.attention(q[0, at], k[0, at], v[0, at], [0, at.stop - a], D ** -0.5, window)
        two = (2.0 ** -16 + FP) * size
        assert ((o[0, at].double() - wo).abs() <= R8 * wo.abs() + (1 + R8) * two + 1e-30).all()
        both = o[0, at].double() + rest[0, at].double()
        assert ((both - wo).abs() <= 2.0 ** -16 * wo.abs() + two + 1e-30).all()


@pytest.mark.parametrize("heads,D,lens,window", [((4, 2), 64, [33, 37], 20), ((3, 1), 128, [150], 0), ((4, 4), 64, [40, 90, 5], 0)])
def test_gradients_against_differences_along_themselves(heads, D, lens, window):
    # fp32: <grad, u> against central differences of L(x) = <o(x), do> with steps h and h / 2, extrapolated, where u is the
    # gradient (in fp64) on random pieces of it, 8 tokens of a head each, so that <grad, u> is as large as it can be.
    # Room: o off by 1e-5 normwise, the library's, moves L by 1e-5 |o| |do|, a quotient of step s by that over s and the
    # extrapolation, (4 (2 / h) + 1 / h) / 3, by three times as much; what the extrapolation leaves is the same
    # differences' own in fp64. That is less than a fiftieth of <grad, u>: a gradient that is zero, doubled, of the other
    # sign or lacks one of its pieces' factors is not near it.
    n = sum(lens)
    q, k, v, do = make(n, *heads, D, F32, seed=45)
    cu, sc, c = bounds(lens), D ** -0.5, ints(bounds(lens))
    f = lambda x: (g2.gdr2_attn_fwd(*x, cu_seqlens=c, window=window).double() * do.double()).sum()
    f64 = lambda x: (ref.attention(*(t[0] for t in x), cu, sc, window)[0] * do[0].double()).sum()
    o, lse, _ = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=c, window=window, save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, cu_seqlens=c, window=window)
    exact = ref.gradients(q[0], k[0], v[0], do[0], cu, sc, window)[:3]
    size = float(o.double().norm() * do.double().norm())
    gen = torch.Generator().manual_seed(2)
    for i, name in enumerate(("dq", "dk", "dv")):
        for part in range(6):
            g = exact[i][None]
            on = torch.rand((n + 7) // 8, g.shape[2], generator=gen) < (1.0, 0.5, 0.5, 0.25, 0.25, 0.25)[part]
            u = g * on.repeat_interleave(8, 0)[:n, :, None].to(g.device)
            u = u * (0.02 * g.numel() ** 0.5 / float(u.norm()))  # 0.02 an element, were they alike

            def slope(fun, h, wide):
                x = [[t.double() for t in (q, k, v)] for _ in range(2)]
                x[0][i], x[1][i] = x[0][i] + h * u, x[1][i] - h * u
                if not wide:
                    x = [[t.float() for t in y] for y in x]
                return float(fun(x[0]) - fun(x[1])) / (2 * h)

            diff = lambda fun, wide: (4 * slope(fun, 0.5, wide) - slope(fun, 1.0, wide)) / 3
            want, got = float((g * u).sum()), float((gr[name].double() * u).sum())
            # (the rounding of x + h u to fp32, 2^-24 of 4 h an element at most, moves L by that times |grad|: within 1e-5 too)
            room = 3 * 1e-5 * size + abs(diff(f64, True) - want)
            assert want > 50 * room, (name, want, room)
            assert abs(got - diff(f, False)) <= room, (name, part, got, want, room)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_no_sequence_around_many(dtype):
    # as test_rows_of_no_sequence, of more sequences than lanes; and bounds out of order among as many stay inside
    lens = [(3 * i) % 19 for i in range(190)] + [7]
    cu, n = bounds(lens, 130), sum(lens)
    args = make(n, 4, 2, 128, dtype, seed=46)
    want = check(*args, bounds(lens))
    pad = lambda x: torch.cat([x.new_full((1, 130, *x.shape[2:]), float("nan")), x, x.new_full((1, 77, *x.shape[2:]), float("inf"))], 1)
    q, k, v, do = (pad(x) for x in args)
    o, lse, rest = g2.gdr2_attn_fwd(q, k, v, cu_seqlens=ints(cu), save_for_bwd=True)
    gr = g2.gdr2_attn_bwd(q, k, v, o, lse, do, rest=rest, cu_seqlens=ints(cu))
    inner = slice(130, 130 + n)
    for a, b in ((o, want[0]), (lse, want[1]), *((gr[x], want[3][x]) for x in gr)):
        # (the sizes of the call choose how waves share the work, and with it the order of sums: as test_offsets_past_32_bits)
        assert normwise(a[:, inner].double(), b.double()) <= (2.0 ** -6 if dtype == BF else 2e-5)
        assert (a[:, :130] == 0).all() and (a[:, 130 + n:] == 0).all()
    for bad in ([5, 90, 40] * 30 + [n], [0] * 70 + [2 ** 31 - 1] * 70, list(range(n, 0, -1))[:200], [-9] * 66):
        o, lse, rest = g2.gdr2_attn_fwd(*args[:3], cu_seqlens=ints(bad), save_for_bwd=True)
        gr = g2.gdr2_attn_bwd(*args[:3], o, lse, args[3], rest=rest, cu_seqlens=ints(bad))
        assert o.shape == args[0].shape and gr["dk"].shape == args[1].shape
    torch.cuda.synchronize()


def test_autograd_twice_broadcast_and_of_a_projection():
    cu = [0, 50, 140]
    q, k, v, do = make(140, 4, 2, 64, BF, seed=47)
    c = ints(cu)
    want = check(q, k, v, do, cu)[3]
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = g2.GDR2AttnFunction.apply(*leaves, c)
    for _ in range(2):
        got = torch.autograd.grad(o, leaves, do, retain_graph=True)
        assert all(torch.equal(a, want[n]) for a, n in zip(got, ("dq", "dk", "dv")))
    # an output's gradient that is one number, broadcast
    ones = check(q, k, v, torch.ones_like(do), cu)[3]
    assert all(torch.equal(a, ones[n]) for a, n in zip(torch.autograd.grad(o.sum(), leaves), ("dq", "dk", "dv")))
    # parts of one projection's output, and a gradient for keys alone
    qkv = torch.cat([q, k, v], 2).requires_grad_()
    a, b, d = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    g2.GDR2AttnFunction.apply(a, b, d, c).backward(do)
    assert torch.equal(qkv.grad, torch.cat([want["dq"], want["dk"], want["dv"]], 2))
    key = k.clone().requires_grad_()
    g2.GDR2AttnFunction.apply(q, key, v, c).backward(do)
    assert torch.equal(key.grad, want["dk"])
    with pytest.raises(RuntimeError):  # no second derivatives
        g = torch.autograd.grad(g2.GDR2AttnFunction.apply(*leaves, c), leaves, do, create_graph=True)
        torch.autograd.grad(g[0].sum(), leaves)


@pytest.mark.parametrize("dtype,T,heads,D", [(BF, 200, (4, 1), 64), (BF, 1100, (16, 16), 128), (F32, 90, (4, 4), 128)])
def test_autograd_in_a_graph(dtype, T, heads, D):
    args = make(T, *heads, D, dtype, seed=48)
    q, k, v, do = args
    want = check(*args, [0, T], packed=False)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]

    def step():
        o = g2.GDR2AttnFunction.apply(*leaves)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(3)
        check(*args, [0, T], packed=False)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (want[0], want[3]["dq"], want[3]["dk"], want[3]["dv"])))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_padded_batch(dtype):
    # sequences of one length, the last tokens of some of them padding with gradients of zero: what comes before does not
    # depend on it, and neither does it get or give a gradient through it
    T, lens = 90, [90, 33, 64, 1]
    q, k, v, do = (x.view(4, T, -1, 64) for x in make(4 * T, 4, 2, 64, dtype, seed=49))
    keep = torch.arange(T, device="cuda")[None, :] < ints(lens)[:, None]
    do = do * keep[:, :, None, None]
    run = lambda *x: (lambda o, lse, rest: (o, g2.gdr2_attn_bwd(*x, o, lse, do, rest=rest)))(*g2.gdr2_attn_fwd(*x, save_for_bwd=True))
    o, gr = run(q, k, v)
    other = [torch.where(keep[:, :, None, None], x, 3.0 * x.roll(1, 1)) for x in (q, k, v)]
    o2, gr2 = run(*other)
    assert torch.equal(o[keep], o2[keep])
    for n in gr:
        assert torch.equal(gr[n][keep], gr2[n][keep]) and not gr[n][~keep].any() and not gr2[n][~keep].any()
