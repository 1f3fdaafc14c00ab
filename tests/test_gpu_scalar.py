"""The gated delta rule with scalar gates against its token loop in fp64 (GPU).

Tolerances, as normwise (Frobenius) errors, set before the first run:
  fp32         1e-5, the bound of the library's fp32 path.
  bf16 tokens  2^-7. One rounding to bf16 is off by at most 2^-8 of the value, 2^-8 / sqrt(3) in the
               mean square over a uniform rounding error; no token output passes through more than
               eight independent ones (states, Delta and dY, P and R, beta K, the output), and
               sqrt(8) 2^-8 / sqrt(3) = 6.4e-3 < 2^-7 = 7.8e-3.
  bf16 states  1e-5: what reaches the carried states is held in two bf16 parts. A pair's error is at
               most 2^-16 of the value, 2^-16 / sqrt(3) = 8.8e-6 for one at its worst mean, and the
               mean over a binade of the two roundings' product is 3e-6; four of them in quadrature
               give 6e-6.
"""
import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import mixer_refs as ref

pytestmark = pytest.mark.gpu

TOK = ("o", "dq", "dk", "dv", "dg", "dbeta")
TOL = {torch.float32: dict(tok=1e-5, state=1e-5), torch.bfloat16: dict(tok=2.0 ** -7, state=1e-5)}


def inputs(lens, packed, hk, hv, dk, dv, dtype, g_scale=0.1, h0=True, seed=0, beta_scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    x = dict(q=unit(rnd(B, T, hk, dk)), k=unit(rnd(B, T, hk, dk)), v=rnd(B, T, hv, dv),
             g=-torch.nn.functional.softplus(rnd(B, T, hv)) * g_scale, beta=beta_scale * torch.sigmoid(rnd(B, T, hv)),
             do=rnd(B, T, hv, dv))
    x = {n: t.to(dtype).cuda() for n, t in x.items()}
    n = len(lens)
    x["h0"] = (rnd(n, hv, dk, dv) * 0.1).float().cuda() if h0 else None
    x["dht"] = (rnd(n, hv, dk, dv) * 0.1).float().cuda() if h0 else None
    cu = None
    if packed:
        cu = [0]
        for m in lens:
            cu.append(cu[-1] + m)
    return x, cu


def device_cu(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def train(x, cu, **kw):
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    o, ht, ws = g2.gdr2_scalar_fwd(*args, cu_seqlens=device_cu(cu), save_for_bwd=True)
    gr = g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], cu_seqlens=device_cu(cu), ws=ws, fwd_saved=True, **kw)
    torch.cuda.synchronize()
    return dict(o=o, ht=ht, **gr)


def check(got, x, cu, dtype, scale=1.0):
    want = ref.run_recurrence(x, cu, grads="dq" in got)
    bad = []
    for n in want:
        if got.get(n) is None:
            continue
        if n in TOK:
            w = torch.cat([t.reshape(-1, *t.shape[1:]) for t in want[n]]) if cu is not None else torch.stack(want[n])
            w = w.reshape(got[n].shape) if w.numel() == got[n].numel() else w
            err = ref.normwise(got[n][:, :cu[-1]].reshape(w.shape) if cu is not None else got[n], w)
            tol = TOL[dtype]["tok"]
        else:
            err, tol = ref.normwise(got[n], want[n]), TOL[dtype]["state"]
        if not err <= tol * scale:
            bad.append((n, err, tol * scale))
    assert not bad, bad


BF, F32 = torch.bfloat16, torch.float32
SHAPES = [
    # lens, packed, hk, hv, dk, dv, dtype
    ([1], False, 1, 1, 64, 64, F32),
    ([63, 63], False, 1, 2, 64, 64, F32),
    ([130], False, 2, 2, 64, 64, F32),
    ([1, 64, 0, 65, 200, 3], True, 2, 4, 64, 64, F32),
    ([1], False, 1, 1, 128, 128, BF),
    ([2], False, 1, 3, 64, 64, BF),
    ([64], False, 2, 2, 128, 128, BF),
    ([65, 65], False, 1, 1, 128, 64, BF),
    ([257], False, 2, 2, 64, 128, BF),
    ([200, 200, 200], False, 3, 6, 128, 128, BF),
    ([300], False, 1, 4, 128, 128, BF),
    ([64, 1, 63, 128, 0, 0, 77], True, 1, 2, 128, 128, BF),
    ([5, 190, 31], True, 2, 2, 64, 64, BF),
    ([0, 100], True, 4, 4, 128, 64, BF),
    ([99, 0], True, 1, 1, 64, 128, BF),
]


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_forward_and_gradients(case, h0):
    lens, packed, hk, hv, dk, dv, dtype = SHAPES[case]
    x, cu = inputs(lens, packed, hk, hv, dk, dv, dtype, h0=h0, seed=case)
    check(train(x, cu), x, cu, dtype)


@pytest.mark.parametrize("g", [0.0, -0.5, -8.0, -20.0, -50.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_any_decay(dtype, g):
    x, cu = inputs([150], False, 1, 2, 64, 64, dtype, seed=5)
    x["g"].fill_(g)
    check(train(x, cu), x, cu, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weak_decay_after_a_strong_one(dtype):
    # the running log-decay stands at some thousands when the weak decays come
    x, cu = inputs([128], False, 1, 1, 64, 64, dtype, seed=6)
    x["g"][:, 3:40] = -60.0
    check(train(x, cu), x, cu, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", [[5], [3, 40], [0, 1, 63, 64], list(range(20, 90))])
@pytest.mark.parametrize("g", [-1000.0, -1e18, None])
def test_decays_that_reset_the_state(dtype, at, g):
    # a log-decay of any finite size, the type's lowest value among them (a usual mark of a new document):
    # nothing of the state is left, and the weak decays behind it count as they would without it
    x, cu = inputs([150], False, 1, 2, 64, 64, dtype, seed=41)
    x["g"][:, at] = torch.finfo(dtype).min if g is None else g
    got = train(x, cu)
    check(got, x, cu, dtype)
    # the recurrent step says the same: each is within its own bound of the exact result
    state = x["h0"].clone()
    o = g2.gdr2_scalar_step(*[x[n] for n in ("q", "k", "v", "g", "beta")], state)
    tok, step = (2.0 ** -7, 2.0 ** -8) if dtype == BF else (1e-5, 1e-5)
    assert ref.normwise(got["o"], o.cpu().double()) <= tok + step
    assert ref.normwise(got["ht"], state.cpu().double()) <= 2e-5


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeated_keys_and_full_writes(dtype):
    # one key throughout and beta = 1: the powers of A grow like binomials, its inverse does not.
    # The corrections Delta_i = v_i - e^g v_(i-1) are sqrt(2) as large as a write and telescope to the
    # last one, while their rounding errors add up in quadrature over the 64 rows of a chunk: the
    # tolerances, of the result's norm, grow by sqrt(64) sqrt(2).
    x, cu = inputs([192], False, 1, 1, 64, 64, dtype, seed=7)
    x["k"][:] = x["k"][:, :1]
    x["k"][:] = torch.where(torch.arange(64, device="cuda") < 4, 0.5, 0.0).to(dtype)
    x["beta"].fill_(1.0)
    x["g"].fill_(-0.01)
    check(train(x, cu), x, cu, dtype, scale=128 ** 0.5)


def test_write_strength_two_and_zero():
    x, cu = inputs([130], False, 1, 2, 64, 64, F32, seed=8, beta_scale=2.0)
    x["beta"][:, ::7] = 0.0
    check(train(x, cu), x, cu, F32)


@pytest.mark.parametrize("noise", [0.1, 0.03])
@pytest.mark.parametrize("case", [(130, 1, 2, 64, 64, F32), (130, 1, 2, 64, 64, BF), (200, 2, 2, 128, 128, BF),
                                  (130, 1, 4, 128, 64, BF)])
def test_gradients_where_the_state_predicts_the_values(case, noise):
    # v = what the state holds for k, and a little noise: dbeta = dY.(v - k^T X) is small against dY.v
    T, hk, hv, dk, dv, dtype = case
    x, _ = inputs([T], False, hk, hv, dk, dv, dtype, g_scale=0.01, seed=42)
    gen = torch.Generator().manual_seed(42)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    S = rnd(hv, dk, dv).float().double()
    x["h0"] = S[None].float().cuda()
    k, g, beta = (ref.sequences(x[n], None)[0] for n in ("k", "g", "beta"))
    k = k.repeat_interleave(hv // hk, 1)
    v = torch.empty(T, hv, dv, dtype=torch.float64)
    for t in range(T):
        X = S * torch.exp(g[t])[:, None, None]
        seen = (k[t][:, :, None] * X).sum(1)
        v[t] = (seen + noise * rnd(hv, dv)).to(dtype).double()
        S = X + k[t][:, :, None] * (beta[t][:, None] * (v[t] - seen))[:, None, :]
    x["v"] = v[None].to(dtype).cuda()
    check(train(x, None), x, None, dtype)


@pytest.mark.parametrize("beta", [0.0, 1e-30, 1e-12, 1e-8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_write_strengths_next_to_nothing(dtype, beta):
    x, cu = inputs([130], False, 1, 2, 64, 64, dtype, seed=43)
    x["beta"][:, ::3] = beta
    x["beta"][:, 1::5] = -0.25
    check(train(x, cu), x, cu, dtype)


@pytest.mark.parametrize("case", [([64] * 8, False, 4, 4, 128, 128), ([200, 57, 130], True, 2, 4, 64, 128),
                                  ([300, 300], False, 2, 2, 128, 64)])
@pytest.mark.parametrize("g_scale", [0.02, 0.5])
def test_output_is_off_by_two_roundings(case, g_scale):
    # bf16: a term of O is rounded once (S's in one operand, M Delta's in the other), and O itself. A rounding is
    # uniform over a step, 2^-8 / sqrt(3) of the step's lower end in the mean square, and over the numbers of a
    # binade, evenly spread in their logarithm, sqrt(3 / (8 ln 2)) of that: 1.66e-3. Two are sqrt(2) of it (three
    # sqrt(3)); a tenth more for what spread the numbers really have.
    lens, packed, hk, hv, dk, dv = case
    x, cu = inputs(lens, packed, hk, hv, dk, dv, BF, g_scale=g_scale, seed=44)
    want = ref.run_recurrence(x, cu)
    w = torch.cat([t.reshape(-1, hv, dv) for t in want["o"]])
    once = 2.0 ** -8 / 3 ** 0.5 * (3 / 8 / 0.6931471805599453) ** 0.5
    for o in (train(x, cu)["o"], g2.gdr2_scalar_fwd(*[x[n] for n in ("q", "k", "v", "g", "beta", "h0")],
                                                    cu_seqlens=device_cu(cu))[0]):
        assert ref.normwise(o.reshape(w.shape), w) <= 1.1 * 2 ** 0.5 * once


@pytest.mark.parametrize("case", [([130] * 4, False, 2, 4, 128, 128), ([200, 57, 130], True, 4, 4, 64, 128),
                                  ([300, 300], False, 2, 2, 128, 64)])
def test_query_gradient_is_off_by_two_roundings(case):
    # bf16: as the output. dq's terms are rounded once each, in S and in Delta (P is held in two parts), then dq
    lens, packed, hk, hv, dk, dv = case
    x, cu = inputs(lens, packed, hk, hv, dk, dv, BF, g_scale=0.5, seed=45)
    want = ref.run_recurrence(x, cu, grads=True)
    w = torch.cat([t.reshape(-1, hk, dk) for t in want["dq"]])
    once = 2.0 ** -8 / 3 ** 0.5 * (3 / 8 / 0.6931471805599453) ** 0.5
    assert ref.normwise(train(x, cu)["dq"].reshape(w.shape), w) <= 1.1 * 2 ** 0.5 * once


@pytest.mark.parametrize("dtype", [BF, F32])
def test_inference_forward_recompute_and_repeats(dtype):
    x, cu = inputs([100, 64, 7], True, 2, 4, 64, 64, dtype, seed=9)
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    a, b = train(x, cu), train(x, cu)
    o, ht, _ = g2.gdr2_scalar_fwd(*args, cu_seqlens=device_cu(cu))
    c = g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], cu_seqlens=device_cu(cu))  # recomputes the forward
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert torch.equal(o, a["o"]) and torch.equal(ht, a["ht"])
    for n in c:
        assert torch.equal(c[n], a[n]), n


def test_no_state_in_or_out():
    x, cu = inputs([70], False, 1, 1, 64, 64, BF, h0=False, seed=10)
    o, ht, _ = g2.gdr2_scalar_fwd(*[x[n] for n in ("q", "k", "v", "g", "beta")], output_final_state=False)
    assert ht is None
    check(dict(o=o), x, cu, BF)


def test_packed_equals_separate_calls():
    lens = [65, 1, 128]
    x, cu = inputs(lens, True, 1, 2, 128, 128, BF, seed=11)
    whole = train(x, cu)
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        part = {n: x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta", "do")}
        part.update(h0=x["h0"][i:i + 1], dht=x["dht"][i:i + 1])
        alone = train(part, None)
        for n in TOK:
            assert torch.equal(alone[n], whole[n][:, a:b]), n
        assert torch.equal(alone["ht"][0], whole["ht"][i]) and torch.equal(alone["dh0"][0], whole["dh0"][i])


@pytest.mark.parametrize("first", [0, 5])
def test_rows_of_no_sequence(first):
    # padding before the first and behind the last sequence holds NaN: it is not read, and is not
    # written in the caller's own outputs, zero in new ones
    lens, pad = [40, 90], 70
    x, cu = inputs(lens, True, 1, 2, 64, 64, BF, seed=12)
    want = train(x, cu)
    wide = dict(x)
    for n in ("q", "k", "v", "g", "beta", "do"):
        t = torch.full((1, first + sum(lens) + pad, *x[n].shape[2:]), float("nan"), dtype=BF, device="cuda")
        t[:, first:first + sum(lens)] = x[n]
        wide[n] = t
    cw = [c + first for c in cu]
    got = train(wide, cw)
    args = [wide[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    mark = {n: torch.full_like(got[n], 7.0) for n in TOK}
    o, _, ws = g2.gdr2_scalar_fwd(*args, cu_seqlens=device_cu(cw), save_for_bwd=True, o=mark["o"])
    g2.gdr2_scalar_bwd(*args, wide["do"], wide["dht"], cu_seqlens=device_cu(cw), ws=ws, fwd_saved=True,
                       grads={n: mark[n] for n in TOK[1:]})
    inside = slice(first, first + sum(lens))
    for n in TOK:
        assert torch.equal(got[n][:, inside], want[n]), n
        assert torch.equal(mark[n][:, inside], want[n]), n
        for s in (slice(0, first), slice(first + sum(lens), None)):
            assert (got[n][:, s] == 0).all() and (mark[n][:, s] == 7.0).all(), n
    for n in ("ht", "dh0"):
        assert torch.equal(got[n], want[n])


@pytest.mark.parametrize("cu", [[0, 200, 100, 130], [-5, 60, 2000, 130], [130, 0, 130, 130]])
def test_bad_bounds_stay_inside(cu):
    # entries out of order or range: wrong results for those sequences, no access outside the tensors
    # (the maps are checked on the CPU in test_mixers_host.py); a call after it is as it was
    x, good = inputs([60, 70], True, 1, 1, 64, 64, BF, seed=13)
    want = train(x, good)
    bad = train(dict(x, h0=None, dht=None), cu)
    assert bad["ht"].shape[0] == len(cu) - 1
    again = train(x, good)
    for n in want:
        assert torch.equal(again[n], want[n]), n


def test_no_tokens():
    h0 = torch.randn(2, 3, 64, 64, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")
    o, ht, ws = g2.gdr2_scalar_fwd(e(2, 0, 1, 64), e(2, 0, 1, 64), e(2, 0, 3, 64), e(2, 0, 3), e(2, 0, 3), h0)
    assert torch.equal(ht, h0) and o.numel() == 0 and ws.numel() == 0
    gr = g2.gdr2_scalar_bwd(e(2, 0, 1, 64), e(2, 0, 1, 64), e(2, 0, 3, 64), e(2, 0, 3), e(2, 0, 3), h0,
                            e(2, 0, 3, 64), h0)
    assert torch.equal(gr["dh0"], h0)
    # packed, no sequences: nothing but rows of no sequence
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, _ = inputs([10], True, 1, 3, 64, 64, BF, h0=False)
    o, ht, _ = g2.gdr2_scalar_fwd(*[x[n] for n in ("q", "k", "v", "g", "beta")], cu_seqlens=cu)
    assert (o == 0).all() and ht.shape[0] == 0


def test_no_sequences_on_another_stream():
    # the zeros are written on the stream that was asked for, not on one that is busy with other work
    x, _ = inputs([4000], True, 1, 3, 64, 64, BF, h0=False)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    busy, s = torch.randn(8192, 8192, device="cuda"), torch.cuda.Stream()
    marks = [torch.full_like(x[n], 7.0) for n in ("q", "k", "v", "v", "g", "beta")]
    torch.cuda.synchronize()
    del marks  # their memory is what the outputs are likely to get
    for _ in range(4):
        busy @ busy
    o, _, _ = g2.gdr2_scalar_fwd(*a, cu_seqlens=cu, stream=s)
    gr = g2.gdr2_scalar_bwd(*a, None, x["do"], cu_seqlens=cu, stream=s)
    with torch.cuda.stream(s):
        got = [t.cpu() for t in (o, *(gr[n] for n in TOK[1:]))]
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in got)


def test_gradients_against_differences():
    x, cu = inputs([70], False, 1, 2, 64, 64, F32, seed=14)
    got = train(x, cu)
    gen = torch.Generator().manual_seed(3)

    def loss(y):
        r = ref.run_recurrence(y, None)
        return float((r["o"][0] * y["do"].cpu().double()[0]).sum() + (r["ht"] * y["dht"].cpu().double()).sum())

    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("h0", "dh0")):
        d = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, dn = ({**x, n: x[n].cpu().double() + s * h * d} for s in (1, -1))
        num = (loss(up) - loss(dn)) / (2 * h)
        ana = float((got[gn].cpu().double() * d).sum())
        # fp32 gradients: 1e-5 of the product of norms; the difference itself is good to 1e-8
        assert abs(num - ana) <= 2e-5 * float(got[gn].cpu().double().norm() * d.norm()), (n, num, ana)


def test_autograd():
    x, cu = inputs([50, 90], True, 1, 2, 64, 64, F32, seed=15)
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta", "h0")]
    o, ht = g2.GDR2ScalarFunction.apply(*leaves, device_cu(cu))
    ((o * x["do"]).sum() + (ht * x["dht"]).sum()).backward()
    want = train(x, cu)
    for leaf, n in zip(leaves, ("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        assert torch.equal(leaf.grad, want[n]), n
    # only the output used, no initial state
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    o, _ = g2.GDR2ScalarFunction.apply(*leaves, None, device_cu(cu))
    (o * x["do"]).sum().backward()
    want = train(dict(x, h0=None, dht=None), cu)
    for leaf, n in zip(leaves, ("dq", "dk", "dv", "dg", "dbeta")):
        assert torch.equal(leaf.grad, want[n]), n


def test_equals_the_channelwise_operator():
    # b = w = beta and one decay for all channels: gdr2_fwd's recurrence. Each side is within its own
    # bound of the exact result, 1e-5 normwise in fp32.
    x, _ = inputs([150], False, 2, 2, 64, 64, F32, seed=16)
    wide = lambda t: t[..., None].expand(*t.shape, 64).contiguous()
    o, ht, _ = g2.gdr2_fwd(x["q"], x["k"], x["v"], wide(x["g"]), wide(x["beta"]), wide(x["beta"]), x["h0"])
    o2, ht2, _ = g2.gdr2_scalar_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["h0"])
    assert ref.normwise(o2, o.cpu().double()) <= 2e-5 and ref.normwise(ht2, ht.cpu().double()) <= 2e-5


@pytest.mark.parametrize("packed", [False, True])
def test_graph_replays(packed):
    x, cu = inputs([64, 64], packed, 1, 2, 128, 128, BF, seed=17)
    dcu = device_cu(cu)
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    want = train(x, cu)
    o = torch.empty_like(want["o"])
    grads = {n: torch.empty_like(want[n]) for n in TOK[1:]}
    ws = torch.empty(g2.gdr2_scalar_workspace_bytes(2, 128 if packed else 64, 1, 2, 128, 128, packed, g2.DTYPE_BF16, True),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g2.gdr2_scalar_fwd(*args, cu_seqlens=dcu, save_for_bwd=True, ws=ws, o=o)
        g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], cu_seqlens=dcu, ws=ws, fwd_saved=True, grads=grads)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, ht, _ = g2.gdr2_scalar_fwd(*args, cu_seqlens=dcu, save_for_bwd=True, ws=ws, o=o)
        r = g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], cu_seqlens=dcu, ws=ws, fwd_saved=True, grads=grads)
    for _ in range(3):
        for t in (o, ht, ws, *grads.values(), r["dh0"]):
            t.fill_(3)
        train(x, cu)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want["o"]) and torch.equal(ht, want["ht"]) and torch.equal(r["dh0"], want["dh0"])
        for n in grads:
            assert torch.equal(grads[n], want[n]), n


def test_another_stream():
    x, cu = inputs([200], False, 2, 2, 128, 128, BF, seed=18)
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    want = train(x, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, ht, ws = g2.gdr2_scalar_fwd(*args, save_for_bwd=True, stream=s)
    gr = g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], ws=ws, fwd_saved=True, stream=s)
    del ws
    junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(o, want["o"]) and torch.equal(ht, want["ht"]) and len(junk) == 8
    for n in TOK[1:]:
        assert torch.equal(gr[n], want[n]), n


def many(lo, hi, n, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (n,), generator=gen).tolist()


@pytest.mark.parametrize("case", [
    # chains enough for two column tiles a workgroup, at equal and at ragged lengths; more sequences
    # than a wave has lanes, with and without that
    ([70] * 4, False, 8, 16, 128, 128, BF), ([129] * 8, False, 4, 16, 64, 64, F32),
    ([66] * 9, False, 2, 8, 64, 128, BF), (many(0, 90, 70, 1), True, 5, 5, 64, 64, BF),
    (many(0, 70, 80, 2), True, 1, 4, 64, 64, F32), (many(0, 20, 100, 3), True, 1, 1, 128, 64, BF),
    (many(1, 3, 300, 4), True, 1, 2, 64, 64, F32)])
def test_many_chains(case):
    lens, packed, hk, hv, dk, dv, dtype = case
    x, cu = inputs(lens, packed, hk, hv, dk, dv, dtype, seed=30)
    check(train(x, cu), x, cu, dtype)


@pytest.mark.parametrize("case", [
    # few chains and long: whole, and cut in three to eight segments, the last ones ragged
    ([2100], 1, 1, 64, 64, F32), ([4133], 1, 2, 64, 64, F32), ([2050, 2050], 2, 2, 128, 128, BF),
    ([3300, 3300], 2, 2, 128, 128, BF),
    ([4200], 1, 2, 128, 64, BF), ([5500], 1, 1, 64, 128, BF), ([8300], 1, 1, 64, 64, BF), ([4096], 4, 4, 128, 128, BF),
    ([4160], 2, 8, 64, 128, BF), ([3300], 16, 16, 64, 64, F32)])
@pytest.mark.parametrize("h0", [True, False])
def test_long_sequences(case, h0):
    # weak decays and writes, so that what one segment leaves still counts in the next ones
    lens, hk, hv, dk, dv, dtype = case
    x, cu = inputs(lens, False, hk, hv, dk, dv, dtype, g_scale=0.0005, beta_scale=0.05, h0=h0, seed=35)
    check(train(x, cu), x, cu, dtype)


@pytest.mark.parametrize("hv", [4, 16])
def test_long_sequences_repeat_and_recompute(hv):
    x, _ = inputs([3300], False, 2, hv, 128, 64, BF, g_scale=0.001, beta_scale=0.1, seed=36)
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    a, b = train(x, None), train(x, None)
    o, ht, _ = g2.gdr2_scalar_fwd(*args)
    c = g2.gdr2_scalar_bwd(*args, x["do"], x["dht"])
    assert torch.equal(o, a["o"]) and torch.equal(ht, a["ht"])
    for n in a:
        assert torch.equal(a[n], b[n]), n
    for n in c:
        assert torch.equal(a[n], c[n]), n


@pytest.mark.parametrize("hv", [2, 16])
def test_long_sequences_in_a_graph(hv):
    # segments, found and joined in the workspace: nothing of it may count between calls
    x, _ = inputs([3300], False, 2, hv, 64, 64, BF, g_scale=0.001, beta_scale=0.1, seed=37)
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")]
    want = train(x, None)
    ws = torch.empty(g2.gdr2_scalar_workspace_bytes(1, 3300, 2, hv, 64, 64, save_for_bwd=True), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, ht, _ = g2.gdr2_scalar_fwd(*args, save_for_bwd=True, ws=ws)
        gr = g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], ws=ws, fwd_saved=True)
    for _ in range(3):
        for t in (o, ht, ws, *gr.values()):
            t.fill_(3)
        train(x, None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in dict(gr, o=o, ht=ht).items():
            assert torch.equal(t, want[n]), n


def test_many_value_heads_of_a_key_head():
    x, cu = inputs([130], False, 2, 14, 64, 64, BF, seed=31)
    check(train(x, cu), x, cu, BF)


def test_backward_twice():
    x, cu = inputs([50, 90], True, 1, 2, 64, 64, BF, seed=32)
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta", "h0")]
    o, ht = g2.GDR2ScalarFunction.apply(*leaves, device_cu(cu))
    run = lambda: torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]], retain_graph=True)
    a, b = run(), run()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    # an output's gradient that is one number, broadcast
    c = torch.autograd.grad(o.sum(), leaves[:5])
    want = train(dict(x, do=torch.ones_like(x["do"]), dht=torch.zeros_like(x["dht"])), cu)
    for t, n in zip(c, ("dq", "dk", "dv", "dg", "dbeta")):
        assert torch.equal(t, want[n]), n


def test_autograd_in_a_graph():
    x, cu = inputs([64, 40], True, 1, 2, 128, 128, BF, seed=33)
    dcu = device_cu(cu)
    want = train(x, cu)
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta", "h0")]

    def step():
        o, ht = g2.GDR2ScalarFunction.apply(*leaves, dcu)
        return (o.detach(), ht.detach(), *torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]]))

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
        train(x, cu)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, n in zip(got, ("o", "ht", "dq", "dk", "dv", "dg", "dbeta", "dh0")):
            assert torch.equal(t, want[n]), n


def test_two_calls_at_once():
    x, cu = inputs([300, 200], True, 2, 4, 128, 128, BF, seed=34)
    want = train(x, cu)
    args, dcu = [x[n] for n in ("q", "k", "v", "g", "beta", "h0")], device_cu(cu)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    res = []
    for s in streams:
        o, ht, ws = g2.gdr2_scalar_fwd(*args, cu_seqlens=dcu, save_for_bwd=True, stream=s)
        res.append(dict(o=o, ht=ht, **g2.gdr2_scalar_bwd(*args, x["do"], x["dht"], cu_seqlens=dcu, ws=ws, fwd_saved=True,
                                                         stream=s)))
    torch.cuda.synchronize()
    for r in res:
        for n in want:
            assert torch.equal(r[n], want[n]), n


def test_packed_without_tokens():
    h0 = torch.randn(2, 3, 64, 64, device="cuda")
    e = lambda *s: torch.empty(1, 0, *s, dtype=BF, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    a = (e(1, 64), e(1, 64), e(3, 64), e(3), e(3), h0)
    o, ht, ws = g2.gdr2_scalar_fwd(*a, cu_seqlens=cu, save_for_bwd=True)
    gr = g2.gdr2_scalar_bwd(*a, e(3, 64), h0 * 2, cu_seqlens=cu, ws=ws, fwd_saved=True)
    assert torch.equal(ht, h0) and torch.equal(gr["dh0"], h0 * 2)


def test_offsets_past_32_bits():
    # 2.2e9 elements of v; the last sequence against a call of its own
    n, T, hv, d = 520, 256, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF)
    x = dict(q=rnd(n, T, 1, d) * d ** -0.5, k=rnd(n, T, 1, d) * d ** -0.5, v=rnd(n, T, hv, d),
             g=-rnd(n, T, hv).abs() * 0.1, beta=torch.sigmoid(rnd(n, T, hv)), do=rnd(n, T, hv, d), h0=None, dht=None)
    got = train(x, None)
    want = train({m: t if t is None else t[-1:].contiguous() for m, t in x.items()}, None)
    for m in want:
        assert torch.equal(got[m][-1], want[m][0]), m


# ---------------------------------------------------------------- the recurrent step


@pytest.mark.parametrize("case", [
    # B, T, hk, hv, dk, dv, dtype, pool (None: one state a row, no slots)
    (1, 1, 1, 1, 64, 64, F32, None), (3, 4, 2, 4, 64, 64, F32, 7), (1, 1, 8, 16, 128, 128, BF, 4),
    (5, 1, 1, 3, 128, 64, BF, 5), (2, 3, 2, 2, 64, 128, BF, None), (300, 1, 1, 2, 64, 64, BF, 301)])
def test_step(case):
    B, T, hk, hv, dk, dv, dtype, pool = case
    x, _ = inputs([T] * B, False, hk, hv, dk, dv, dtype, seed=20)
    gen = torch.Generator().manual_seed(1)
    n = pool or B
    state = (torch.randn(n, hv, dk, dv, generator=gen) * 0.1).cuda()
    slots = torch.randperm(n, generator=gen)[:B].to(torch.int32).cuda() if pool else None
    rows = slots.long() if pool else torch.arange(B, device="cuda")
    x["h0"] = state[rows]
    before = state.clone()
    o = g2.gdr2_scalar_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state, slots=slots)
    want = ref.run_recurrence(x, None)
    # fp32 arithmetic throughout: bf16 outputs are off by their one rounding, at most 2^-8
    assert ref.normwise(o, torch.stack(want["o"])) <= (1e-5 if dtype == F32 else 2.0 ** -8)
    assert ref.normwise(state[rows], want["ht"]) <= 1e-5
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(state[rest], before[rest])


def test_step_padding_rows_and_shared_slots():
    B, hv, d = 6, 2, 64
    x, _ = inputs([2] * B, False, 1, hv, d, d, F32, seed=21)
    state = torch.randn(3, hv, d, d, device="cuda") * 0.1
    before = state.clone()
    slots = torch.tensor([2, -1, 0, 2, 3, 2], dtype=torch.int32, device="cuda")
    o = g2.gdr2_scalar_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state, slots=slots,
                            o=torch.full((B, 2, hv, d), 5.0, device="cuda"))
    assert (o[1] == 0).all() and (o[4] == 0).all() and torch.equal(state[1], before[1])
    for slot, rows in ((2, [0, 3, 5]), (0, [2])):
        y = {n: x[n][rows].reshape(1, -1, *x[n].shape[2:]) for n in ("q", "k", "v", "g", "beta")}
        want = ref.run_recurrence(dict(y, h0=before[slot:slot + 1]))
        assert ref.normwise(o[rows].reshape(1, -1, hv, d), torch.stack(want["o"])) <= 1e-5
        assert ref.normwise(state[slot:slot + 1], want["ht"]) <= 1e-5


def test_step_continues_a_prompt():
    x, _ = inputs([70], False, 1, 2, 128, 128, BF, h0=False, seed=22)
    n = 66
    head = {m: x[m][:, :n].contiguous() for m in ("q", "k", "v", "g", "beta")}
    tail = {m: x[m][:, n:].contiguous() for m in ("q", "k", "v", "g", "beta")}
    o1, ht, _ = g2.gdr2_scalar_fwd(*head.values())
    o2 = g2.gdr2_scalar_step(*tail.values(), ht)
    check(dict(o=torch.cat([o1, o2], 1), ht=ht), x, None, BF)


def test_step_graph_replays():
    x, _ = inputs([1] * 4, False, 1, 2, 64, 64, BF, seed=23)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    start = torch.randn(4, 2, 64, 64, device="cuda") * 0.1
    state = start.clone()
    slots = torch.tensor([3, 1, 0, 2], dtype=torch.int32, device="cuda")
    o = torch.empty(4, 1, 2, 64, dtype=BF, device="cuda")
    g2.gdr2_scalar_step(*args, state, slots=slots, o=o)
    want_o, want_s = o.clone(), state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.gdr2_scalar_step(*args, state, slots=slots, o=o)
    for _ in range(3):
        state.copy_(start)
        o.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(state, want_s)


def test_step_offsets_past_32_bits():
    hv, d, S = 16, 128, 8300  # 2.2e9 elements of state
    x, _ = inputs([1] * 3, False, 8, hv, d, d, BF, seed=24)
    state = torch.zeros(S, hv, d, d, device="cuda")
    slots = torch.tensor([8299, 0, 4100], dtype=torch.int32, device="cuda")
    state[slots.long()] = x["h0"]
    o = g2.gdr2_scalar_step(*[x[n] for n in ("q", "k", "v", "g", "beta")], state, slots=slots)
    want = ref.run_recurrence(x, None)
    assert ref.normwise(o, torch.stack(want["o"])) <= 2.0 ** -8
    assert ref.normwise(state[slots.long()], want["ht"]) <= 1e-5
    assert int(torch.count_nonzero(state.view(S, -1).any(1))) == 3


# ---------------------------------------------------------------- refusals (before any launch)


def test_refusals():
    x, cu = inputs([10, 20], True, 1, 2, 64, 64, BF)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    f = g2.gdr2_scalar_fwd
    with pytest.raises(ValueError):
        f(a[0], a[1], a[2], a[3].float(), a[4])
    with pytest.raises(ValueError):
        f(a[0], a[1], a[2][:, :, :, :32].contiguous(), a[3][:, :5], a[4])
    with pytest.raises(ValueError):
        f(*a, cu_seqlens=torch.tensor([0, 30], device="cuda"))  # int64
    with pytest.raises(ValueError):
        f(*a, x["h0"][:1], cu_seqlens=device_cu(cu))
    with pytest.raises(ValueError):
        f(a[0].half(), a[1].half(), a[2].half(), a[3].half(), a[4].half())
    with pytest.raises(ValueError):  # three value heads over two key heads
        two = torch.cat([a[0], a[0]], 2)
        f(two, two, torch.cat([a[2], a[2][:, :, :1]], 2), torch.cat([a[3], a[3][:, :, :1]], 2),
          torch.cat([a[4], a[4][:, :, :1]], 2))
    with pytest.raises(RuntimeError):
        f(*a, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        g2.gdr2_scalar_bwd(*a, None, x["do"], fwd_saved=True)
    with pytest.raises(ValueError):
        g2.gdr2_scalar_step(*a, x["h0"][:0])
    with pytest.raises(ValueError):
        g2.gdr2_scalar_step(*a, x["h0"], slots=torch.zeros(2, dtype=torch.int32, device="cuda"))
