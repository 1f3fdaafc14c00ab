"""Trees of drafts with more than 32 (draft, head) rows a key head, which take the cache through tiles in LDS: windows,
holes in tables, places past a table's end, in each layout of the tiles, for rows that one workgroup takes and for rows
that several share (GPU). References and tolerances are those of tests/test_gpu_tree.py."""
import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
from test_gpu_tree import check, ints, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# rows a key head and channels: 33 to 64, 65 to 128 and more; the last is more than one block of 256
ROWS = [(40, (2, 2), 64), (33, (3, 3), 128), (40, (4, 2), 64), (12, (16, 2), 128), (50, (5, 1), 64), (64, (16, 2), 128)]
# pages of 16 tokens of a table: of up to 512 tokens, which a workgroup takes whole; and of so many that rows are split, as
# tiles of 128 tokens and (one sequence, at 65 to 128 rows) of 64
SHORT, LONG = [200, 1, 0, 129, 64], [300, 1, 0, 129, 64, 1500]


@pytest.mark.parametrize("T,heads,D", ROWS)
@pytest.mark.parametrize("starts,width", [(SHORT, 0), (LONG, 120), (LONG, 1200)])
@pytest.mark.parametrize("window", [1, 5, 11, 12, 13, 63, 64, 65, 130, 700])
def test_window(T, heads, D, starts, width, window):
    drafts = [T, T, 3, T // 2, T, T][:len(starts)]
    check(*make(starts, T, *heads, D, 16, BF, seed=46, width=width, drafts=drafts), window=window)
    check(*make([starts[-1]], T, *heads, D, 16, BF, seed=47, width=width, kind="chain"), window=window)


@pytest.mark.parametrize("T,heads,D", ROWS)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("width", [0, 300])
def test_pages_that_are_none(T, heads, D, page, width):
    n = 18 * page
    q, parents, kc, vc, table, starts = make([n, n, n, 64, 42, 7], T, *heads, D, page, BF, seed=48, width=width)
    P = kc.shape[0]
    for row, col, bad in ((0, 1, -1), (0, 18, P), (1, 0, 2 ** 31 - 1), (1, 3, -2 ** 31), (1, 17, -1), (3, 0, -1), (4, 2, -1), (5, 0, P)):
        table[row][col] = bad
    table[2] = [-7] * len(table[2])
    for window in (0, 5, 90):
        check(q, parents, kc, vc, table, starts, window=window)


@pytest.mark.parametrize("T,heads,D", ROWS)
def test_places_past_the_table(T, heads, D):
    # lengths past the table and below zero; drafts that the table has no room for
    q, parents, kc, vc, table, _ = make([100, 100, 700], T, *heads, D, 16, BF, seed=49)
    for window in (0, 7, 50):
        for starts in ([96, 94, 2 ** 31 - 1], [95, 5000, 90], [96, 96, 96]):
            check(q, parents, kc, vc, [r[:6] for r in table], starts, window=window)
        long = [r + [-1] * 400 for r in table]
        check(q, parents, kc, vc, [r[:6] + [-1] * 400 for r in table], [96, 94, 95], window=window)
        check(q, parents, kc, vc, long, [100, 100, 700], window=window)
    q, parents, kc, vc, table, _ = make([0, 0], T, *heads, D, 16, BF, seed=50)
    check(q, parents, kc, vc, table, [-3, -2 ** 31])


@pytest.mark.parametrize("T,heads,D", ROWS)
def test_all_padding_and_strides(T, heads, D):
    for order in ("HND", "KV"):
        q, parents, kc, vc, table, starts = make([70, 0, 500], T, *heads, D, 32, BF, seed=51, order=order, width=80)
        parents[0] = [-2] * T
        parents[2] = [0] * T  # a draft that continues itself, and all that continue it
        o, lse = check(q, parents, kc, vc, table, starts)
        assert torch.isinf(lse[0]).all() and torch.isinf(lse[2]).all()


@pytest.mark.parametrize("T,heads,D", ROWS)
def test_graph_and_streams(T, heads, D):
    a = make([1700, 30, 0, 255], T, *heads, D, 64, BF, seed=52)
    q, parents, kc, vc, table, starts = a
    want, wl = check(*a, window=600)
    p, t, st = ints(parents), ints(table), ints(starts)
    n = g2.gdr2_attn_tree_workspace_bytes(4, T, *heads, D)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    o, lse = torch.empty_like(q), torch.empty_like(wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.gdr2_attn_tree(q, p, kc, vc, t, st, window=600, o=o, lse=lse, ws=ws[0])
    for _ in range(3):
        for x in (o, lse):
            x.fill_(1)
        ws[0].fill_(255)
        check(*a, window=600)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [g2.gdr2_attn_tree(q, p, kc, vc, t, st, window=600, ws=ws[i], stream=s[i]) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)
