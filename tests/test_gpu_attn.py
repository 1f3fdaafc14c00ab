"""Attention over a paged key-value cache, and the cache's writer, against fp64 (GPU).

Tolerances, normwise, set before the first run. fp32: 1e-5, the library's. bf16 outputs: each weight
is rounded to bf16 once (its sum is not) and the output once, two roundings of at most 2^-8 of the
value: 2^-7. lse is fp32 throughout in both types: absolute errors of a score are at most
2^-24 (D + 3) |q||k| scale, below 1e-5 of an lse of order one; 1e-5 relative and absolute."""
import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import mixer_refs as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-5, BF: 2.0 ** -7}


def make(lengths, Hq, Hkv, D, page, dtype, seed=0, order="NHD", spare=3, width=0):
    """Caches with random pages; everything that no sequence holds is NaN or infinite."""
    gen = torch.Generator().manual_seed(seed)
    B = len(lengths)
    need = [(n + page - 1) // page for n in lengths]
    P = sum(need) + spare
    free = torch.randperm(P, generator=gen).tolist()
    table = [[free.pop() for _ in range(n)] for n in need]
    wide = max(max(need), width)
    kc = torch.full((P, page, Hkv, D), float("nan"))
    vc = torch.full((P, page, Hkv, D), float("inf"))
    for b, n in enumerate(lengths):
        for t in range(n):
            kc[table[b][t // page], t % page] = torch.randn(Hkv, D, generator=gen)
            vc[table[b][t // page], t % page] = torch.randn(Hkv, D, generator=gen)
    q = torch.randn(B, Hq, D, generator=gen).to(dtype).cuda()
    kc, vc = kc.to(dtype), vc.to(dtype)
    if order == "HND":      # heads outside tokens in memory
        kc, vc = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (kc, vc))
    elif order == "KV":     # keys and values in one tensor, two more rows of heads between tokens
        both = torch.full((P, 2, page, Hkv + 2, D), float("nan"), dtype=dtype)
        both[:, 0, :, :Hkv], both[:, 1, :, :Hkv] = kc, vc
        both = both.cuda()
        kc, vc = both[:, 0, :, :Hkv], both[:, 1, :, :Hkv]
    else:
        kc, vc = kc.cuda(), vc.cuda()
    full = [row + [-1] * (wide - len(row)) for row in table]
    dev = torch.tensor(full, dtype=torch.int32).reshape(B, wide).cuda()
    return q, kc, vc, full, dev, torch.tensor(lengths, dtype=torch.int32).cuda()


def check(q, kc, vc, table, dev, lengths, window=0, scale=None, lens=None, **kw):
    D = q.shape[2]
    o, lse = g2.gdr2_attn_step(q, kc, vc, dev, lengths, window=window, scale=scale, return_lse=True, **kw)
    wo, wl = ref.attention(q, kc, vc, table, lengths.tolist() if lens is None else lens,
                           D ** -0.5 if scale is None else scale, window)
    assert torch.isfinite(o.float()).all()
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse.cpu()), empty) and (lse.cpu()[empty] < 0).all()
    assert (o.cpu()[empty] == 0).all()
    if (~empty).any():
        assert (lse.cpu().double() - wl)[~empty].abs().max() <= 1e-5 * max(1.0, wl[~empty].abs().max())
        for b in range(q.shape[0]):
            assert ref.normwise(o[b], wo[b]) <= TOL[q.dtype], b
    return o, lse


LENGTHS = [[1], [16], [17], [31, 32, 33], [64, 0, 1, 127, 128, 129], [1000, 3], [0, 0], [5000]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", range(len(LENGTHS)))
def test_lengths(dtype, n):
    check(*make(LENGTHS[n], 8, 2, 128, 64, dtype, seed=n))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (40, 2), (64, 2), (32, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(dtype, heads, D):
    check(*make([70, 5, 333], *heads, D, 32, dtype, seed=3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("order", ["NHD", "HND", "KV"])
def test_pages_and_strides(dtype, page, order):
    check(*make([200, 16, 1, 47], 4, 2, 64, page, dtype, seed=4, order=order))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 15, 16, 33, 100, 1000])
def test_window(dtype, window):
    check(*make([300, 1, 0, 33, 99, 100, 101], 6, 3, 64, 16, dtype, seed=5), window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_and_scale(dtype):
    gen = torch.Generator().manual_seed(6)
    lengths = torch.randint(0, 90, (700,), generator=gen).tolist()  # more sequences than a workgroup's threads
    check(*make(lengths, 2, 1, 64, 16, dtype, seed=6), scale=0.3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores(dtype):
    # scores of some hundreds: the weights underflow but for a few, and no exponential overflows
    q, kc, vc, table, dev, lengths = make([257, 40], 4, 4, 64, 32, dtype, seed=7)
    o, lse = g2.gdr2_attn_step(q, kc, vc, dev, lengths, scale=20.0, return_lse=True)
    wo, wl = ref.attention(q, kc, vc, table, lengths.tolist(), 20.0, 0)
    # a score of size s is off by up to 2^-23 s, and a weight by that times itself
    tol = TOL[dtype] + 2.0 ** -22 * float(wl.abs().max())
    assert ref.normwise(o, wo) <= tol and (lse.cpu().double() - wl).abs().max() <= 1e-5 * wl.abs().max()


@pytest.mark.parametrize("lens", [[2], [3], [40, 7], [777], [4000]])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_keep_their_digits(lens, D):
    # bf16: every element of o is off by its own rounding, 2^-8 of it, and by what the weights are off by:
    # a score by up to 2^-24 (D + 3) |q||k| scale, in the weight and in the sum of the weights, and a weight
    # held in two bf16 parts by 2^-17 and less of it, with 2^-20 for the sums; that of sum p |v| / sum p
    q, kc, vc, table, dev, lengths = make(lens, 4, 2, D, 64, BF, seed=50)
    o = g2.gdr2_attn_step(q, kc, vc, dev, lengths)
    wo, _ = ref.attention(q, kc, vc, table, lens, D ** -0.5, 0)
    size, _ = ref.attention(q, kc, vc.abs(), table, lens, D ** -0.5, 0)
    kn = torch.where(torch.isnan(kc), torch.zeros_like(kc), kc).double().norm(dim=-1).max()
    score = 2.0 ** -24 * (D + 3) * float(q.double().norm(dim=-1).max() * kn) * D ** -0.5
    room = 2.0 ** -8 * wo.abs() + (2 * score + 2.0 ** -17 + 2.0 ** -20) * size * (1 + 2.0 ** -8)
    assert ((o.cpu().double() - wo).abs() <= room).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_that_are_none(dtype):
    # holes in the table, ids past the pool, lengths past the table and below zero
    q, kc, vc, table, dev, _ = make([100, 100, 100, 64, 48], 4, 2, 64, 16, dtype, seed=8)
    P = kc.shape[0]
    for row, col, bad in ((0, 1, -1), (0, 6, P), (1, 0, 2 ** 31 - 1), (1, 3, -2 ** 31)):
        table[row][col] = bad
    for c in range(len(table[2])):
        table[2][c] = -7
    dev = torch.tensor(table, dtype=torch.int32).cuda()
    lens = [100, 100, 100, 64, 48]
    check(q, kc, vc, table, dev, torch.tensor(lens, dtype=torch.int32).cuda())
    width = 16 * len(table[0])
    some = torch.tensor([100, 100, -5, 64, 0], dtype=torch.int32).cuda()
    check(q, kc, vc, table, dev, some, lens=[100, 100, 0, 64, 0])
    q2, kc2, vc2, table2, dev2, _ = make([width], 4, 2, 64, 16, dtype, seed=9)
    check(q2, kc2, vc2, table2, dev2, torch.tensor([2 ** 31 - 1], dtype=torch.int32).cuda(), lens=[width])


def test_no_pages_and_no_rows():
    q = torch.randn(2, 4, 64, device="cuda")
    z = torch.empty(0, 16, 2, 64, device="cuda")
    t = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    o, lse = g2.gdr2_attn_step(q, z, z, t(2, 3), t(2) + 20, return_lse=True)
    assert (o == 0).all() and (lse == -float("inf")).all()
    c = torch.randn(4, 16, 2, 64, device="cuda")
    o = g2.gdr2_attn_step(q, c, c, t(2, 0), t(2) + 20)
    assert (o == 0).all()
    assert g2.gdr2_attn_step(q[:0], c, c, t(0, 3), t(0)).numel() == 0


def test_shared_pages_and_repeats():
    q, kc, vc, table, dev, lengths = make([96, 96, 96], 8, 2, 128, 32, BF, seed=10)
    for row in table[1:]:
        row[:2] = table[0][:2]  # a common prefix
    dev = torch.tensor(table, dtype=torch.int32).cuda()
    o, lse = check(q, kc, vc, table, dev, lengths)
    for _ in range(3):
        o2, lse2 = g2.gdr2_attn_step(q, kc, vc, dev, lengths, return_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_graph_and_streams():
    a = make([700, 30, 0, 255], 8, 2, 128, 64, BF, seed=11)
    q, kc, vc, table, dev, lengths = a
    want, wl = check(*a)
    ws = [torch.empty(g2.gdr2_attn_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    o, lse = torch.empty_like(q), torch.empty(4, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.gdr2_attn_step(q, kc, vc, dev, lengths, o=o, lse=lse, ws=ws[0])
    for _ in range(3):
        o.fill_(1)
        lse.fill_(1)
        ws[0].fill_(255)
        check(*a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)
    # two calls at once, a workspace each
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [g2.gdr2_attn_step(q, kc, vc, dev, lengths, ws=ws[i], stream=s[i]) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 2500])
def test_ragged_rows_on_shared_workgroups(dtype, window):
    # tables wide enough for long rows: rows of any length share the line of workgroups
    lens = [0, 4000, 1, 17, 0, 900, 31, 2600, 64] + [5] * 20
    check(*make(lens, 4, 2, 64, 16, dtype, seed=15, width=600), window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_rows_than_lanes_on_shared_workgroups(dtype):
    gen = torch.Generator().manual_seed(16)
    lens = [n if n > 20 else 0 for n in torch.randint(0, 150, (150,), generator=gen).tolist()]
    check(*make(lens, 3, 3, 64, 16, dtype, seed=16, width=700))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_thousands_of_rows_on_shared_workgroups(dtype):
    gen = torch.Generator().manual_seed(19)
    lens = torch.randint(0, 5, (2500,), generator=gen).tolist()
    lens[1234] = 3000
    check(*make(lens, 2, 1, 64, 16, dtype, seed=19, width=300))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_heads_of_a_long_row(dtype):
    check(*make([2100, 700], 34, 2, 128, 32, dtype, seed=17, width=200))


def test_offsets_past_32_bits():
    P, page, H, D = 2100, 1024, 8, 128  # 2.2e9 elements a cache
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.empty(P, page, H, D, dtype=BF, device="cuda") for _ in range(2))
    ids = [2099, 7, 2060]
    for c in (kc, vc):
        for p in ids:
            c[p] = torch.randn(page, H, D, generator=gen, device="cuda")
    small_k, small_v = kc[ids], vc[ids]
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 16, D, generator=gen, device="cuda").to(BF)
    far, near = ints([2099, 7], [2060, -1]), ints([0, 1], [2, -1])
    held = ints(1500, 700)
    k, v = (torch.randn(2, H, D, generator=gen, device="cuda").to(BF) for _ in range(2))
    g2.gdr2_kv_append(k, v, kc, vc, far, held)
    g2.gdr2_kv_append(k, v, small_k, small_v, near, held)
    assert torch.equal(kc[ids], small_k) and torch.equal(vc[ids], small_v)
    for a, b in zip(g2.gdr2_attn_step(q, kc, vc, far, held + 1, return_lse=True),
                    g2.gdr2_attn_step(q, small_k, small_v, near, held + 1, return_lse=True)):
        assert torch.equal(a, b)


def test_more_rows_than_a_launch_takes_workgroups():
    # 2^23 rows and some: short rows, but one launch of a workgroup each would pass 2^32 threads
    B, H, D = 2 ** 19 + 3, 16, 64
    lens = {0: 5, 77: 16, B // 2: 31, B - 1: 1}
    q, kc, vc, table, _, _ = make(list(lens.values()), H, H, D, 16, BF, seed=20, width=2)
    wide = torch.zeros(B, H, D, dtype=BF, device="cuda")
    dev = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = torch.tensor(list(lens), device="cuda")
    wide[rows], dev[rows] = q, torch.tensor(table, dtype=torch.int32).cuda()
    lengths[rows] = torch.tensor(list(lens.values()), dtype=torch.int32).cuda()
    o, lse = g2.gdr2_attn_step(wide, kc, vc, dev, lengths, return_lse=True)
    wo, wl = ref.attention(q, kc, vc, table, list(lens.values()), D ** -0.5, 0)
    assert ref.normwise(o[rows], wo) <= TOL[BF] and (lse[rows].cpu().double() - wl).abs().max() <= 1e-5 * wl.abs().max()
    empty = torch.ones(B, dtype=torch.bool, device="cuda")
    empty[rows] = False
    assert not o[empty].any() and (lse[empty] == -float("inf")).all()


def test_windows_past_32_bits():
    q, kc, vc, table, dev, lengths = make([40], 2, 2, 64, 16, BF, seed=18)
    assert torch.equal(g2.gdr2_attn_step(q, kc, vc, dev, lengths, window=2 ** 32 + 5),
                       g2.gdr2_attn_step(q, kc, vc, dev, lengths))
    with pytest.raises(RuntimeError):
        g2.gdr2_attn_step(q, kc, vc, dev, lengths, window=-2 ** 32 + 5)


# ---------------------------------------------------------------- the cache's writer


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", ["NHD", "HND", "KV"])
@pytest.mark.parametrize("packed", [False, True])
def test_append(dtype, order, packed):
    page, H, D = 16, 3, 64
    held = [0, 15, 16, 40]
    new = [5, 0, 33, 1] if packed else [1] * 4
    total = [a + b for a, b in zip(held, new)]
    _, kc, vc, table, dev, _ = make(total, H, H, D, page, dtype, seed=12, order=order)
    want_k, want_v = kc.clone(), vc.clone()
    gen = torch.Generator().manual_seed(2)
    pad = 3 if packed else 0  # rows behind the last sequence are not written
    k, v = (torch.randn(sum(new) + pad, H, D, generator=gen).to(dtype).cuda() for _ in range(2))
    i = 0
    for s, n in enumerate(new):
        for t in range(n):
            pos = held[s] + t
            want_k[table[s][pos // page], pos % page] = k[i]
            want_v[table[s][pos // page], pos % page] = v[i]
            i += 1
    cu = None
    if packed:
        cu = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32).cuda()
    g2.gdr2_kv_append(k, v, kc, vc, dev, torch.tensor(held, dtype=torch.int32).cuda(), cu_seqlens=cu)
    same = lambda a, b: torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))
    assert same(kc, want_k) and same(vc, want_v)


def test_append_drops_tokens_without_a_place():
    kc, vc = torch.zeros(3, 16, 1, 64, device="cuda"), torch.zeros(3, 16, 1, 64, device="cuda")
    k = torch.ones(6, 1, 64, device="cuda")
    dev = torch.tensor([[0, -1], [3, 1], [2, 2], [2, 2], [-9, 2 ** 31 - 1], [1, 1]], dtype=torch.int32).cuda()
    starts = torch.tensor([16, 0, -1, 32, 3, 2 ** 31 - 1], dtype=torch.int32).cuda()
    g2.gdr2_kv_append(k, k, kc, vc, dev, starts)
    assert (kc == 0).all() and (vc == 0).all()
    cu = torch.tensor([2, 4, 3, 9], dtype=torch.int32).cuda()  # out of order and past the end
    g2.gdr2_kv_append(k, k, kc, vc, dev[:3], torch.zeros(3, dtype=torch.int32).cuda(), cu_seqlens=cu)
    assert torch.isfinite(kc).all()


def test_append_then_attend():
    # a prompt in two pieces, then token by token
    page, Hq, Hkv, D = 16, 4, 2, 64
    lens = [35, 18]
    q, kc, vc, table, dev, _ = make([n + 3 for n in lens], Hq, Hkv, D, page, BF, seed=13)
    full_k, full_v = kc.clone(), vc.clone()
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    rows = lambda c, s, a, b: torch.stack([c[table[s][t // page], t % page] for t in range(a, b)])
    ints = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    for a, b in ((0, 17), (17, None)):
        parts = [(a, n if b is None else b) for n in lens]
        k, v = (torch.cat([rows(c, s, *p) for s, p in enumerate(parts)]) for c in (full_k, full_v))
        n0, n1 = (p[1] - p[0] for p in parts)
        g2.gdr2_kv_append(k, v, kc, vc, dev, ints(a, a), cu_seqlens=ints(0, n0, n0 + n1))
    for step in range(3):
        at = [n + step for n in lens]
        k, v = (torch.cat([rows(c, s, t, t + 1) for s, t in enumerate(at)]) for c in (full_k, full_v))
        g2.gdr2_kv_append(k, v, kc, vc, dev, ints(*at))
        check(q, kc, vc, table, dev, ints(*[t + 1 for t in at]))


def test_refusals():
    q, kc, vc, _, dev, lengths = make([20, 30], 4, 2, 64, 16, BF, seed=14)
    f = g2.gdr2_attn_step
    with pytest.raises(ValueError):
        f(q.float(), kc, vc, dev, lengths)
    with pytest.raises(ValueError):
        f(q, kc, vc[:, :, :1], dev, lengths)
    with pytest.raises(ValueError):
        f(q, kc, vc, dev.long(), lengths)
    with pytest.raises(ValueError):
        f(q, kc, vc, dev, lengths[:1])
    with pytest.raises(ValueError):
        f(q, kc.transpose(1, 3), vc.transpose(1, 3), dev, lengths)
    with pytest.raises(RuntimeError):
        f(q[:, :3].contiguous(), kc, vc, dev, lengths)
    with pytest.raises(RuntimeError):
        f(q, kc[:, :8], vc[:, :8], dev, lengths)  # pages of 8 tokens
    with pytest.raises(RuntimeError):
        f(q, kc, vc, dev, lengths, window=-1)
    with pytest.raises(RuntimeError):
        f(q, kc, vc, dev, lengths, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        g2.gdr2_kv_append(q, q, kc, vc, dev, lengths)
    k = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        g2.gdr2_kv_append(k, k, kc, vc, dev, lengths)
