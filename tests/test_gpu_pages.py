"""Block tables, slots and bounds built on the GPU against the same order of events in Python, and the cache's operators
together: pages, prompts, trees of drafts, accepted paths (GPU). Whole numbers are equal; attention's tolerances are
those of tests/test_gpu_attn.py."""
import random

import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import mixer_refs
import prompt_refs as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normwise(a, b):
    return mixer_refs.normwise(a, b.cpu())


def ints(x, *shape):
    t = torch.tensor(x, dtype=torch.int32)
    return (t.reshape(*shape) if shape else t).cuda()


def run(lengths, counts, table, free, num_free, page, max_tokens, **kw):
    B = len(lengths)
    dev = [ints(lengths, B), ints(counts, B), ints(table, B, len(table[0]) if B else 3), ints(free, len(free)), ints([num_free])]
    new, cu, slots = g2.gdr2_kv_pages(*dev, page_size=page, max_tokens=max_tokens, **kw)
    return dev, (new.tolist(), cu.tolist(), slots.tolist(), dev[2].tolist(), dev[3].tolist(), int(dev[4]))


def check(*args, again=True):
    dev, got = run(*args)
    want = ref.pages(*args)
    for a, b, n in zip(got, want, ("lengths", "bounds", "slots", "table", "stack", "free pages")):
        assert a == b, n
    if not again:
        return want
    # the same call again changes nothing
    again = g2.gdr2_kv_pages(*dev, page_size=args[5], max_tokens=args[6])
    assert [x.tolist() for x in again] == list(want[:3])
    assert (dev[2].tolist(), dev[3].tolist(), int(dev[4])) == tuple(want[3:])
    return want


def pool(rng, B, width, page, high, spare, new=0.0, gone=0.0, new_hi=1, holes=0.0):
    lengths = [rng.randint(0, high) for _ in range(B)]
    counts = [rng.choice([0, 1, 1, 1]) for _ in range(B)]
    for b in range(B):
        x = rng.random()
        if x < new:
            counts[b] = rng.randint(1, new_hi)
        elif x < new + gone:
            counts[b] = -rng.randint(1, 5)
    need = [-(-n // page) for n in lengths]
    P = sum(need) + spare
    ids = list(range(P))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(n)] + [-1] * (width - n) for n in need]
    for row in table:
        for i in range(width):
            if rng.random() < holes:
                row[i] = rng.choice([-1, -5, P, 2 ** 31 - 1])
    free = ids + [rng.randrange(P) for _ in range(P - len(ids))]
    return lengths, counts, table, free, len(ids)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = random.Random(seed)
    page = rng.choice([16, 32, 256])
    B = rng.choice([1, 5, 63, 64, 65, 300])
    width = rng.choice([4, 70, 200])
    high = page * width // 2
    a = pool(rng, B, width, page, high, rng.choice([0, 3, B, 50 * B]), new=0.2, gone=0.2 * (seed % 3), new_hi=page * 40,
             holes=0.05 * (seed % 2))
    check(*a, page, sum(max(c, 0) for c in a[1]) + rng.choice([0, 5]))


def test_more_requests_than_threads_and_many_tokens():
    rng = random.Random(100)
    a = pool(rng, 3000, 12, 16, 150, 1500, new=0.1, gone=0.1, new_hi=40)
    check(*a, 16, 9000)  # slots by the second kernel
    a = pool(rng, 2100, 5, 16, 60, 4000, new=0.0)
    check(*a, 16, 2100)


def test_too_few_pages():
    # the third request lacks more than is left; the fourth lacks one page and waits behind it, the fifth lacks none
    table = [[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, -1, -1], [4, -1, -1]]
    want = check([16, 16, 16, 16, 3], [1, 16, 20, 1, 2], table, [5, 6, 7, 0, 0, 0, 0, 0], 3, 16, 40)
    assert want[0] == [17, 32, 16, 16, 5] and want[5] == 1
    # pages that are given back are taken in the same call, also by requests before theirs
    want = check([16, 16, 33], [5, 5, -1], [[0, -1, -1], [1, -1, -1], [2, 3, 4]], [9, 9, 9, 9, 9], 0, 16, 10)
    assert want[3] == [[0, 4, -1], [1, 3, -1], [-1, -1, -1]] and want[5] == 1


def test_bounds_and_odd_numbers():
    t = [[0, 1], [2, -1], [3, -1]]
    f = [4, 5, 6, 7, 0, 0, 0, 0]
    check([32, 10, 5], [1, 3, 2 ** 31 - 1], t, f, 4, 16, 4)           # no room in the table; past max_tokens
    check([-7, 2 ** 31 - 1, 40], [3, 1, 1], t, f, 4, 16, 8)           # lengths that are none
    check([20, 10, 5], [3, 1, 1], t, f, -3, 16, 8)                    # a count of free pages that is none
    check([20, 10, 5], [13, 30, -2], t, f, 100, 16, 60)
    check([20, 10, 5], [-1, -1, -1], t, [0] * 8, 7, 16, 0)            # more given back than the stack holds
    check([0, 0], [0, 0], [[-1], [-1]], [0], 1, 16, 3)
    check([0, 20], [3, 3], [[-1, -1], [5, 5]], [9, -4, 2, 2, 2, 2], 2, 16, 6, again=False)  # a stack that holds no pages:
    # what is taken is still none, and a second call takes again


def test_no_requests_and_no_pages():
    _, got = run([], [], [], [3, 1], 2, 16, 4)
    assert got[0] == [] and got[1] == [0] and got[2] == [-1] * 4 and got[5] == 2
    check([5], [3], [[-1, -1]], [], 0, 16, 3)
    dev = [ints([5]), ints([3]), torch.empty(1, 0, dtype=torch.int32, device="cuda"), ints([1, 0]), ints([2])]
    new, cu, slots = g2.gdr2_kv_pages(*dev, page_size=16, max_tokens=3)
    assert new.tolist() == [0] and cu.tolist() == [0, 3] and slots.tolist() == [-1] * 3


def test_tensors_of_the_callers_graph_and_streams():
    rng = random.Random(7)
    a = pool(rng, 130, 40, 16, 300, 200, new=0.2, gone=0.2, new_hi=200)
    tokens = sum(max(c, 0) for c in a[1]) + 3
    want = ref.pages(*a, 16, tokens)
    first = [ints(a[0]), ints(a[1]), ints(a[2]), ints(a[3]), ints([a[4]])]
    dev = [x.clone() for x in first]
    out = dict(new_lengths=ints([0] * 130), cu_seqlens=ints([0] * 131), slots=torch.zeros(tokens, dtype=torch.int64, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.gdr2_kv_pages(*dev, page_size=16, max_tokens=tokens, **out)
    for _ in range(3):
        for x, y in zip(dev, first):
            x.copy_(y)
        for x in out.values():
            x.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [out[n].tolist() for n in out] + [dev[2].tolist(), dev[3].tolist(), int(dev[4])]
        assert got == list(want)
    s = torch.cuda.Stream()
    for x, y in zip(dev, first):
        x.copy_(y)
    torch.cuda.synchronize()
    got = g2.gdr2_kv_pages(*dev, page_size=16, max_tokens=tokens, stream=s)
    torch.empty(1 << 16, device="cuda").fill_(float("nan"))
    torch.cuda.synchronize()
    assert [x.tolist() for x in got] == list(want[:3])


def test_refusals():
    a = [ints([5, 5]), ints([1, 1]), ints([[0, -1], [1, -1]]), ints([2, 3, 0, 0]), ints([2])]
    kw = dict(page_size=16, max_tokens=4)
    for i, bad in ((0, a[0].long()), (1, a[1][:1]), (2, a[2].t()), (2, a[0]), (3, a[3].float()), (4, ints([1, 1])), (1, a[1].cpu())):
        with pytest.raises(ValueError):
            g2.gdr2_kv_pages(*a[:i], bad, *a[i + 1:], **kw)
    with pytest.raises(ValueError):
        g2.gdr2_kv_pages(*a, page_size=16, max_tokens=-1)
    for page in (0, 8, 24, 1 << 21, 2 ** 32 + 16):
        with pytest.raises(RuntimeError):
            g2.gdr2_kv_pages(*a, page_size=page, max_tokens=4)
    with pytest.raises(ValueError):
        g2.gdr2_kv_pages(*a, **kw, slots=torch.zeros(5, dtype=torch.int64, device="cuda"))
    assert [x.tolist() for x in a] == [[5, 5], [1, 1], [[0, -1], [1, -1]], [2, 3, 0, 0], [2]]


def test_a_server_from_prompt_to_accepted_drafts():
    """Prompts come in, are read by whole-sequence attention, drafts are checked and their best path kept, a plain step
    follows, a request ends and another takes its pages: every output against fp64 over the tokens that were accepted."""
    Hq, Hkv, D, page, B, width, T = 4, 2, 64, 16, 3, 12, 7
    gen = torch.Generator().manual_seed(31)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(BF).cuda()
    kc, vc = (torch.full((24, page, Hkv, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    table, free, num_free = ints([[-1] * width] * B), ints(list(range(23, -1, -1))), ints([24])
    lengths = ints([0] * B)
    held = [[torch.empty(0, Hkv, D, dtype=BF, device="cuda")] * 2 for _ in range(B)]
    spot = lambda x: ints(x)

    def grow(counts):
        nonlocal lengths
        total = sum(max(c, 0) for c in counts)
        starts = lengths
        lengths, cu, slots = g2.gdr2_kv_pages(lengths, spot(counts), table, free, num_free, page_size=page, max_tokens=total)
        k, v = rnd(total, Hkv, D), rnd(total, Hkv, D)
        g2.gdr2_kv_append(k, v, kc, vc, table, starts, cu_seqlens=cu)
        # the slots say where the tokens went
        assert torch.equal(kc.flatten(0, 1)[slots], k) and torch.equal(vc.flatten(0, 1)[slots], v)
        return starts, cu, k, v

    def prompt(counts):
        _, cu, k, v = grow(counts)
        q = rnd(1, k.shape[0], Hq, D)
        o = g2.gdr2_attn_fwd(q, k[None], v[None], cu_seqlens=cu)
        wo, _, size = ref.attention(q[0], k, v, cu.tolist(), D ** -0.5)
        assert ((o[0].double() - wo).abs() <= 2.0 ** -7 * size + 2.0 ** -8 * wo.abs()).all()
        for b, (i, j) in enumerate(ref.spans(cu.tolist())):
            held[b] = [torch.cat([x, y[i:j]]) for x, y in zip(held[b], (k, v))]

    def attend(q, k, v):
        wo, _ = ref.tree(q[None], [[-1]], k[None], v[None], [[0]], [k.shape[0] - 1], D ** -0.5)
        return wo[0, 0]

    def speculate(paths):
        starts, cu, k, v = grow([T] * B)
        parents = [[-1, 0, 0, 1, 3, 2, -1]] * B
        q = rnd(B, T, Hq, D)
        o = g2.gdr2_attn_tree(q, spot(parents), kc, vc, table, starts)
        for b in range(B):
            for i in range(T):
                line = sorted(ref.lineage(parents[b], i))
                at = torch.tensor([b * T + x for x in line], device="cuda")
                wo = attend(q[b, i:i + 1], *(torch.cat([x, y[at]]) for x, y in zip(held[b], (k, v))))
                assert normwise(o[b, i], wo) <= 2.0 ** -7
        nonlocal lengths
        lengths = g2.gdr2_kv_keep(kc, vc, table, starts, spot([p + [-1] * (T - len(p)) for p in paths]))
        for b, p in enumerate(paths):
            at = torch.tensor([b * T + x for x in p], dtype=torch.long, device="cuda")
            held[b] = [torch.cat([x, y[at]]) for x, y in zip(held[b], (k, v))]

    def step():
        _, _, k, v = grow([1] * B)
        q = rnd(B, Hq, D)
        o = g2.gdr2_attn_step(q, kc, vc, table, lengths)
        for b in range(B):
            held[b] = [torch.cat([x, y[b:b + 1]]) for x, y in zip(held[b], (k, v))]
            assert normwise(o[b], attend(q[b:b + 1], *held[b])) <= 2.0 ** -7

    prompt([37, 5, 80])
    speculate([[0, 1, 3, 4], [6], []])
    step()
    speculate([[0, 2, 5], [0, 1, 3, 4], [0]])
    step()
    assert lengths.tolist() == [x[0].shape[0] for x in held]
    before = int(num_free)
    lengths, _, _ = g2.gdr2_kv_pages(lengths, spot([0, 0, -1]), table, free, num_free, page_size=page, max_tokens=0)
    held[2] = [x[:0] for x in held[2]]
    assert int(num_free) > before and lengths[2] == 0
    prompt([0, 0, 60])
    step()
    assert lengths.tolist() == [x[0].shape[0] for x in held]


@pytest.mark.parametrize("tokens", [2040, 2041, 2042, 4088, 4089, 4090])
def test_tokens_around_the_second_kernel(tokens):
    # slots by the workgroup that hands out the pages, and by a kernel of their own; max_tokens is 7 more
    lengths, counts = [5, 0, 31, 7], [1, tokens - 12, 10, 1]
    table = [[3, -1], [-1] * 2, [1, 2], [0, -1]]
    table = [r + [-1] * 300 for r in table]
    free = [4 + i for i in range(296)] + [0] * 4
    check(lengths, counts, table, free, 296, 16, tokens + 7)
