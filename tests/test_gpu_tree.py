"""Attention of trees of drafted tokens over a paged cache, and the move that keeps an accepted path, against fp64 and
copies (GPU). Tolerances as tests/test_gpu_attn.py: fp32 1e-5 normwise, bf16 the output's own rounding and no more than
that again, 2^-7; lse 1e-5 relative and absolute."""
import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import mixer_refs
import prompt_refs as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-5, BF: 2.0 ** -7}


def normwise(a, b):
    return mixer_refs.normwise(a, b.cpu())


def ints(x, *shape):
    t = torch.tensor(x, dtype=torch.int32)
    return (t.reshape(*shape) if shape else t).cuda()


def grow(T, n, gen, kind="any"):
    """Parents of n drafts and T - n places of padding."""
    r = lambda hi: int(torch.randint(0, hi, (1,), generator=gen))
    if kind == "chain":
        row = list(range(-1, n - 1))
    elif kind == "flat":
        row = [-1] * n
    else:
        row = [r(i + 1) - 1 for i in range(n)]
    return row + [-2] * (T - n)


def make(starts, T, Hq, Hkv, D, page, dtype, seed=0, order="NHD", width=0, kind="any", drafts=None, spare=3):
    """Caches with random pages; everything that no draft sees is NaN or infinite."""
    gen = torch.Generator().manual_seed(seed)
    B = len(starts)
    drafts = [T] * B if drafts is None else drafts
    parents = [grow(T, n, gen, kind) for n in drafts]
    need = [(n + T + page - 1) // page for n in starts]
    P = sum(need) + spare
    free = torch.randperm(P, generator=gen).tolist()
    table = [[free.pop() for _ in range(n)] for n in need]
    kc, vc = torch.full((P, page, Hkv, D), float("nan")), torch.full((P, page, Hkv, D), float("inf"))
    for b, n in enumerate(starts):
        t = torch.arange(n + drafts[b])
        rows = torch.tensor(table[b] + [0], dtype=torch.long)[t // page], t % page
        kc[rows], vc[rows] = (torch.randn(len(t), Hkv, D, generator=gen) for _ in range(2))
    q = torch.randn(B, T, Hq, D, generator=gen).to(dtype).cuda()
    kc, vc = kc.to(dtype), vc.to(dtype)
    if order == "HND":
        kc, vc = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (kc, vc))
    elif order == "KV":
        both = torch.full((P, 2, page, Hkv + 2, D), float("nan"), dtype=dtype)
        both[:, 0, :, :Hkv], both[:, 1, :, :Hkv] = kc, vc
        both = both.cuda()
        kc, vc = both[:, 0, :, :Hkv], both[:, 1, :, :Hkv]
    else:
        kc, vc = kc.cuda(), vc.cuda()
    wide = max(max(need), width)
    full = [row + [-1] * (wide - len(row)) for row in table]
    return q, parents, kc, vc, full, starts


def check(q, parents, kc, vc, table, starts, window=0, scale=None, **kw):
    B, T, Hq, D = q.shape
    o, lse = g2.gdr2_attn_tree(q, ints(parents, B, T), kc, vc, ints(table, B, -1 if table[0] else 0), ints(starts),
                               window=window, scale=scale, return_lse=True, **kw)
    wo, wl = ref.tree(q, parents, kc, vc, table, starts, D ** -0.5 if scale is None else scale, window)
    assert torch.isfinite(o.float()).all()
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse.cpu()), empty) and (lse.cpu()[empty] < 0).all()
    assert (o.cpu()[empty] == 0).all()
    if (~empty).any():
        assert (lse.cpu().double() - wl)[~empty].abs().max() <= 1e-5 * max(1.0, float(wl[~empty].abs().max()))
        for b in range(B):
            if float(wo[b].norm()):
                assert normwise(o[b], wo[b]) <= TOL[q.dtype], b
    return o, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 7, 16, 33, 64])
@pytest.mark.parametrize("kind", ["any", "chain", "flat"])
def test_shapes_of_trees(dtype, T, kind):
    check(*make([0, 1, 17, 64, 200], T, 4, 2, 64, 16, dtype, seed=T, kind=kind))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (40, 2), (32, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(dtype, heads, D):
    check(*make([70, 5, 333], 11, *heads, D, 32, dtype, seed=3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("order", ["NHD", "HND", "KV"])
def test_pages_and_strides(dtype, page, order):
    check(*make([200, 16, 0, 47], 9, 4, 2, 64, page, dtype, seed=4, order=order))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 5, 11, 12, 13, 33, 100, 1000])
def test_window(dtype, window):
    check(*make([300, 1, 0, 33, 99, 100, 101], 12, 6, 3, 64, 16, dtype, seed=5), window=window)
    check(*make([300, 1, 0, 20], 12, 2, 1, 64, 16, dtype, seed=6, kind="chain", drafts=[12, 12, 5, 3]), window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding(dtype):
    check(*make([40, 0, 129, 15], 20, 4, 2, 64, 16, dtype, seed=7, drafts=[20, 3, 0, 1]))
    # parents that are none, and drafts that continue them
    q, parents, kc, vc, table, starts = make([40, 40], 8, 4, 2, 64, 16, dtype, seed=8, kind="flat")
    parents[0] = [-1, 1, 0, 7, 2, -5, 4, 2 ** 31 - 1]
    parents[1] = [0, 0, 1, -1, 3, 4, -2 ** 31, 6]
    o, lse = check(q, parents, kc, vc, table, starts)
    assert torch.isinf(lse[0]).all(-1).tolist() == [False, True, False, True, False, True, False, True]
    assert torch.isinf(lse[1]).all(-1).tolist() == [True, True, True, False, False, False, True, True]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_on_shared_workgroups(dtype):
    # tables wide enough for long rows: rows of any length share the line of workgroups
    starts = [0, 1500, 1, 17, 0, 900, 31, 2600, 64] + [5] * 12
    check(*make(starts, 6, 4, 2, 64, 16, dtype, seed=15, width=600))
    check(*make(starts[:9], 6, 4, 2, 64, 16, dtype, seed=15, width=600), window=700)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [3, 24, 64])
def test_a_long_row_on_many_workgroups(dtype, T):
    # more (draft, head) pairs than waves side by side take, and parts of a row in many workgroups
    check(*make([5000], T, 16, 2, 128, 64, dtype, seed=16))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_rows_than_lanes(dtype):
    gen = torch.Generator().manual_seed(17)
    starts = [n if n > 20 else 0 for n in torch.randint(0, 120, (150,), generator=gen).tolist()]
    check(*make(starts, 3, 3, 3, 64, 16, dtype, seed=17, width=700))
    check(*make(starts, 3, 3, 3, 64, 16, dtype, seed=17))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_that_are_none(dtype):
    q, parents, kc, vc, table, starts = make([100, 100, 100, 64, 42], 6, 4, 2, 64, 16, dtype, seed=9)
    P = kc.shape[0]
    for row, col, bad in ((0, 1, -1), (0, 6, P), (1, 0, 2 ** 31 - 1), (1, 3, -2 ** 31), (4, 2, -1)):
        table[row][col] = bad
    table[2] = [-7] * len(table[2])
    check(q, parents, kc, vc, table, starts)
    # lengths past the table and below zero; drafts that the table has no room for
    check(q, parents, kc, vc, [r[:6] for r in table], [96, 94, 5000, 64, 2 ** 31 - 1])
    fresh = make([112], 6, 4, 2, 64, 16, dtype, seed=10)
    check(*fresh[:4], [fresh[4][0][:7]], [109])
    q, parents, kc, vc, table, _ = make([0, 0], 6, 4, 2, 64, 16, dtype, seed=10)
    check(q, parents, kc, vc, table, [-3, -2 ** 31])


def test_no_pages_and_no_rows():
    q = torch.randn(2, 3, 4, 64, device="cuda")
    z = torch.empty(0, 16, 2, 64, device="cuda")
    t = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    o, lse = g2.gdr2_attn_tree(q, t(2, 3) - 1, z, z, t(2, 3), t(2) + 20, return_lse=True)
    assert (o == 0).all() and (lse == -float("inf")).all()
    c = torch.randn(4, 16, 2, 64, device="cuda")
    assert (g2.gdr2_attn_tree(q, t(2, 3) - 1, c, c, t(2, 0), t(2) + 20) == 0).all()
    assert g2.gdr2_attn_tree(q[:0], t(0, 3), c, c, t(0, 3), t(0)).numel() == 0
    assert g2.gdr2_attn_tree(q[:, :0].contiguous(), t(2, 0), c, c, t(2, 3), t(2)).numel() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_draft_is_a_step(dtype):
    q, parents, kc, vc, table, starts = make([0, 31, 700], 1, 8, 2, 128, 32, dtype, seed=11)
    for window in (0, 1, 100):
        o, lse = check(q, parents, kc, vc, table, starts, window=window)
        so, sl = g2.gdr2_attn_step(q[:, 0], kc, vc, ints(table), ints(starts) + 1, window=window, return_lse=True)
        assert normwise(o[:, 0], so.double().cpu()) <= TOL[dtype] and (lse[:, 0] - sl).abs().max() <= 2e-5 * max(1.0, float(sl.abs().max()))


def test_large_scores_and_scales():
    for scale, hkv in ((20.0, 4), (-0.2, 4), (0.0, 4), (20.0, 1), (-0.2, 1), (0.0, 1)):
        q, parents, kc, vc, table, starts = make([257, 40], 9, 4, hkv, 64, 32, BF, seed=12)
        o, lse = g2.gdr2_attn_tree(q, ints(parents), kc, vc, ints(table), ints(starts), scale=scale, return_lse=True)
        wo, wl = ref.tree(q, parents, kc, vc, table, starts, scale)
        tol = TOL[BF] + 2.0 ** -22 * float(wl.abs().max())
        assert normwise(o, wo) <= tol and (lse.cpu().double() - wl).abs().max() <= 1e-5 * wl.abs().max()


def test_graph_streams_and_repeats():
    a = make([1700, 30, 0, 255], 12, 8, 2, 128, 64, BF, seed=13)
    q, parents, kc, vc, table, starts = a
    want, wl = check(*a)
    p, t, st = ints(parents), ints(table), ints(starts)
    n = g2.gdr2_attn_tree_workspace_bytes(4, 12, 8, 2, 128)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    o, lse = torch.empty_like(q), torch.empty(4, 12, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.gdr2_attn_tree(q, p, kc, vc, t, st, o=o, lse=lse, ws=ws[0])
    for _ in range(3):
        o.fill_(1)
        lse.fill_(1)
        ws[0].fill_(255)
        check(*a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [g2.gdr2_attn_tree(q, p, kc, vc, t, st, ws=ws[i], stream=s[i]) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


def test_offsets_past_32_bits():
    P, page, H, D = 2100, 1024, 8, 128  # 2.2e9 elements a cache
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.empty(P, page, H, D, dtype=BF, device="cuda") for _ in range(2))
    ids = [2099, 7, 2060]
    for c in (kc, vc):
        for p in ids:
            c[p] = torch.randn(page, H, D, generator=gen, device="cuda")
    small_k, small_v = kc[ids], vc[ids]
    q = torch.randn(2, 5, 16, D, generator=gen, device="cuda").to(BF)
    far, near = ints([[2099, 7], [2060, -1]]), ints([[0, 1], [2, -1]])
    held, parents = ints([1500, 700]), ints([[-1, 0, 1, 0, -1]] * 2)
    path = ints([[4, 2, -1], [1, 1, 3]])
    for a, b in zip(g2.gdr2_attn_tree(q, parents, kc, vc, far, held, return_lse=True),
                    g2.gdr2_attn_tree(q, parents, small_k, small_v, near, held, return_lse=True)):
        assert torch.equal(a, b)
    assert torch.equal(g2.gdr2_kv_keep(kc, vc, far, held, path), g2.gdr2_kv_keep(small_k, small_v, near, held, path))
    assert torch.equal(kc[ids], small_k) and torch.equal(vc[ids], small_v)


def test_tree_refusals():
    q, parents, kc, vc, table, starts = make([20, 30], 4, 4, 2, 64, 16, BF, seed=14)
    p, t, st = ints(parents), ints(table), ints(starts)
    f = g2.gdr2_attn_tree
    for bad in ((q.float(), p, kc, vc, t, st), (q, p.long(), kc, vc, t, st), (q, p[:, :3].contiguous(), kc, vc, t, st),
                (q, p, kc, vc[:, :, :1], t, st), (q, p, kc, vc, t.long(), st), (q, p, kc, vc, t, st[:1]),
                (q[0], p, kc, vc, t, st), (q.transpose(1, 2), p, kc, vc, t, st), (q, p.cpu(), kc, vc, t, st)):
        with pytest.raises(ValueError):
            f(*bad)
    wide = torch.zeros(2, 65, 4, 64, dtype=BF, device="cuda")
    with pytest.raises(RuntimeError):
        f(wide, torch.zeros(2, 65, dtype=torch.int32, device="cuda"), kc, vc, t, st)
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(RuntimeError):
            f(q, p, kc, vc, t, st, **kw)
    with pytest.raises(RuntimeError):
        f(q[:, :, :3].contiguous(), p, kc, vc, t, st)


@pytest.mark.parametrize("hkv", [4, 1])
def test_small_scales_of_large_scores(hkv):
    # powers of two that come out again; up to 32 rows a key head, and more
    q, parents, kc, vc, table, starts = make([257, 40], 9, 4, hkv, 64, 32, BF, seed=24)
    f = 2.0 ** 60
    run = lambda s, scale: g2.gdr2_attn_tree(q * s, ints(parents), kc * s, vc, ints(table), ints(starts), scale=scale, return_lse=True)
    for scale in (0.125, -0.25):
        assert all(torch.equal(a, b) for a, b in zip(run(1.0, scale), run(f, scale / f / f)))
    for scale in (0.0, 1e-45):
        check(q, parents, kc, vc, table, starts, scale=scale)


# ---------------------------------------------------------------- keeping an accepted path


def kept(kc, vc, table, starts, path):
    """The move in plain form, on the CPU."""
    P, page = kc.shape[:2]
    out = [kc.cpu().clone(), vc.cpu().clone()]
    src = [x.clone() for x in out]
    lengths = []

    def place(b, pos):
        if pos < 0 or pos // page >= len(table[b]) or not 0 <= table[b][pos // page] < P:
            return None
        return table[b][pos // page], pos % page

    for b, row in enumerate(path):
        n = next((j for j, x in enumerate(row) if x < 0), len(row))
        lengths.append(starts[b] + n)
        for j in range(n):
            s, d = place(b, starts[b] + row[j]), place(b, starts[b] + j)
            if s and d:
                for x, y in zip(out, src):
                    x[d] = y[s]
    return out[0], out[1], lengths


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", ["NHD", "HND", "KV"])
@pytest.mark.parametrize("heads", [(1, 64), (3, 64), (8, 128)])
def test_keep(dtype, order, heads):
    H, D = heads
    starts = [0, 15, 16, 40, 7, 3]
    _, _, kc, vc, table, _ = make(starts, 64, H, H, D, 16, dtype, seed=20, order=order)
    path = [[0, 1, 2, 3, 4, 5], [1, 3, 4, 9, 30, 63], [5, -1, 7, 8, 9, 10], [5, 4, 3, 2, 1, 0], [2, 2, 2, 0, 0, 63],
            [-9, 3, 3, 3, 3, 3]]
    wk, wv, wl = kept(kc, vc, table, starts, path)
    lengths = g2.gdr2_kv_keep(kc, vc, ints(table), ints(starts), ints(path))
    same = lambda a, b: torch.equal(a.cpu().contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert same(kc, wk) and same(vc, wv) and lengths.tolist() == wl


def test_keep_long_paths_and_places_that_are_none():
    gen = torch.Generator().manual_seed(21)
    starts = [0, 100, 37, 5, -3, 2 ** 31 - 70]
    _, _, kc, vc, table, _ = make([0, 100, 37, 5, 0, 0], 64, 2, 2, 64, 32, BF, seed=21)
    table[1][4] = -1
    table[2][1] = 10 ** 6
    path = [torch.randperm(64, generator=gen).tolist(), sorted(torch.randperm(64, generator=gen).tolist()),
            torch.randint(0, 64, (64,), generator=gen).tolist(), [200] * 64, list(range(1, 64)) + [0], [1] * 64]
    wk, wv, wl = kept(kc, vc, table, starts, path)
    mine = torch.empty(6, dtype=torch.int32, device="cuda")
    assert g2.gdr2_kv_keep(kc, vc, ints(table), ints(starts), ints(path), lengths=mine) is mine
    same = lambda a, b: torch.equal(a.cpu().contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert same(kc, wk) and same(vc, wv) and mine.tolist() == wl
    none = g2.gdr2_kv_keep(kc, vc, ints(table), ints(starts), torch.empty(6, 0, dtype=torch.int32, device="cuda"))
    assert none.tolist() == starts and same(kc, wk)
    with pytest.raises(RuntimeError):
        g2.gdr2_kv_keep(kc, vc, ints(table), ints(starts), torch.zeros(6, 65, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        g2.gdr2_kv_keep(kc, vc, ints(table), ints(starts), ints(path).long())
    with pytest.raises(ValueError):
        g2.gdr2_kv_keep(kc, vc[:1], ints(table), ints(starts), ints(path))
