"""Host-only checks (no GPU) of the scalar-gate and paged-attention entry points: sizes, refusals
before any launch, and the maps from tokens to chunk slots for any cu_seqlens."""
import ctypes
import gc
import os
import random

import pytest

import gated_delta_rule_gdr2_amd as g2

OK, NULL, SHAPE, UNSUP, ALIGN, WS, HIP, VALUE = 0, -1, -2, -3, -4, -5, -6, -7
BF, F32 = g2.DTYPE_BF16, g2.DTYPE_F32
FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation, or has nothing to do
I64x6 = ctypes.c_longlong * 6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(g2.library_path()):
        from gated_delta_rule_gdr2_amd import build
        build.build()
    return g2.load_library()


def scalar(lib, bwd=False, ptrs=None, cu=None, N=1, T=64, Hk=1, Hv=1, dk=64, dv=64, dtype=BF, ws=FAKE,
           ws_bytes=1 << 40):
    n = 14 if bwd else 8
    p = list([FAKE] * n if ptrs is None else ptrs)
    p.insert(8 if bwd else 6, cu)
    f = lib.gdr2_scalar_bwd if bwd else lib.gdr2_scalar_fwd
    return f(*p, N, T, Hk, Hv, dk, dv, dtype, 0, 1, ws, ws_bytes, None)


def step(lib, ptrs=None, slots=FAKE, B=1, T=1, Hk=1, Hv=1, dk=64, dv=64, states=1, dtype=BF):
    p = list([FAKE] * 7 if ptrs is None else ptrs)
    p.insert(6, slots)
    return lib.gdr2_scalar_step(*p, B, T, Hk, Hv, dk, dv, states, dtype, None)


def attn(lib, q=FAKE, k=FAKE, v=FAKE, strides=(8192, 128, 64) * 2, table=FAKE, lengths=FAKE, o=FAKE, B=1, Hq=2, Hkv=1,
         D=64, pages=4, page=64, max_pages=4, scale=0.1, window=0, dtype=BF, ws=FAKE, ws_bytes=1 << 40):
    st = None if strides is None else I64x6(*strides)
    return lib.gdr2_attn_step(q, k, v, st, table, lengths, o, None, B, Hq, Hkv, D, pages, page, max_pages, scale, window,
                              dtype, ws, ws_bytes, None)


def append(lib, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, strides=(8192, 128, 64) * 2, table=FAKE, starts=FAKE, cu=None, B=1,
           tokens=1, Hkv=1, D=64, pages=4, page=64, max_pages=4, dtype=BF):
    st = None if strides is None else I64x6(*strides)
    return lib.gdr2_kv_append(k, v, kc, vc, st, table, starts, cu, B, tokens, Hkv, D, pages, page, max_pages, dtype, None)


def test_scalar_workspace_sizes(lib):
    f = g2.gdr2_scalar_workspace_bytes
    a, b = f(2, 4096, 16, 16, 128, 128), f(2, 4096, 16, 16, 128, 128, save_for_bwd=True)
    assert 0 < a < b
    assert f(1, 65, 1, 1, 64, 64) == f(1, 128, 1, 1, 64, 64)
    assert f(3, 8192, 16, 16, 128, 128, packed=True) > a  # spare chunks
    assert f(1, 8192, 16, 16, 128, 128) > a  # as many chunks, and segments of few long walks
    assert f(1, 64, 2, 3, 64, 64) == 0 and f(1, 64, 1, 1, 96, 64) == 0 and f(-1, 64, 1, 1, 64, 64) == 0
    assert f(1, 64, 1, 1, 128, 128, dtype=F32) == 0
    assert f(0, 64, 1, 1, 64, 64) == 0 and f(1, 0, 1, 1, 64, 64) == 0
    assert f(1 << 20, 1 << 20, 1, 1, 64, 64) == 0  # too many tokens


@pytest.mark.parametrize("bwd", [False, True])
def test_scalar_refusals(lib, bwd):
    n = 14 if bwd else 8
    optional = (5, 7, 13) if bwd else (5, 7)  # h0, dht, dh0 / h0, ht
    for i in range(n):
        p = [FAKE] * n
        p[i] = 0
        assert scalar(lib, bwd, p, ws=0) == (WS if i in optional else NULL), i
        gate = i in ((3, 4, 11, 12) if bwd else (3, 4))  # read element by element
        p[i] = FAKE + 2
        assert scalar(lib, bwd, p, ws=0) == (WS if gate else ALIGN), i
        p[i] = FAKE + 1
        assert scalar(lib, bwd, p) == ALIGN, i
    assert scalar(lib, bwd, N=-1) == SHAPE and scalar(lib, bwd, T=-1) == SHAPE
    assert scalar(lib, bwd, Hk=2, Hv=3) == SHAPE and scalar(lib, bwd, Hk=0, Hv=3) == SHAPE
    assert scalar(lib, bwd, dk=96) == UNSUP and scalar(lib, bwd, dtype=F32, dk=128) == UNSUP
    assert scalar(lib, bwd, dtype=7) == UNSUP
    assert scalar(lib, bwd, N=1 << 20, T=1 << 20) == SHAPE
    need = g2.gdr2_scalar_workspace_bytes(1, 64, 1, 1, 64, 64, save_for_bwd=True)
    assert scalar(lib, bwd, ws_bytes=need - 1) == WS and scalar(lib, bwd, ws=FAKE + 8) == ALIGN
    packed = g2.gdr2_scalar_workspace_bytes(3, 64, 1, 1, 64, 64, packed=True, save_for_bwd=True)
    assert scalar(lib, bwd, cu=FAKE, N=3, ws_bytes=packed - 1) == WS
    # nothing to do
    none = [0] * n
    assert scalar(lib, bwd, none, N=0, ws=0) == OK and scalar(lib, bwd, none, Hk=0, Hv=0, ws=0) == OK


def test_step_refusals(lib):
    for i in range(7):
        p = [FAKE] * 7
        p[i] = 0
        assert step(lib, p) == NULL, i
        p[i] = FAKE + (1 if i in (3, 4) else 4)
        assert step(lib, p) == ALIGN, i
    assert step(lib, slots=0, B=2, states=1) == SHAPE and step(lib, states=-1) == SHAPE
    assert step(lib, Hk=2, Hv=3) == SHAPE and step(lib, dk=32) == UNSUP and step(lib, dtype=5) == UNSUP
    assert step(lib, [0] * 7, B=0) == OK and step(lib, [0] * 7, T=0) == OK


def test_attention_refusals(lib):
    need = g2.gdr2_attn_workspace_bytes(1, 2, 1, 64)
    assert need > 0 and g2.gdr2_attn_workspace_bytes(0, 2, 1, 64) == 0 and g2.gdr2_attn_workspace_bytes(1, 3, 2, 64) == 0
    assert g2.gdr2_attn_workspace_bytes(9, 64, 1, 128) == g2.gdr2_attn_workspace_bytes(1, 16, 1, 128)
    for name in ("q", "k", "v", "table", "lengths", "o", "strides"):
        assert attn(lib, **{name: None if name == "strides" else 0}) == NULL, name
    for name in ("q", "k", "v", "o", "ws"):
        assert attn(lib, **{name: FAKE + 8}) == ALIGN, name
    assert attn(lib, strides=(8192, 128, 60, 8192, 128, 64)) == ALIGN and attn(lib, strides=(-8, 8, 8, 8, 8, 8)) == ALIGN
    assert attn(lib, Hq=3, Hkv=2) == SHAPE and attn(lib, B=-1) == SHAPE and attn(lib, pages=-1) == SHAPE
    assert attn(lib, D=96) == UNSUP and attn(lib, dtype=9) == UNSUP
    for page in (0, 8, 24, -16, 1 << 21):
        assert attn(lib, page=page) == VALUE, page
    assert attn(lib, window=-1) == VALUE
    for s in (float("inf"), float("nan")):
        assert attn(lib, scale=s) == VALUE
    assert attn(lib, ws=0) == WS and attn(lib, ws_bytes=need - 1) == WS
    assert attn(lib, B=0, q=0, ws=0) == OK


def test_append_refusals(lib):
    for name in ("k", "v", "kc", "vc", "table", "starts", "strides"):
        assert append(lib, **{name: None if name == "strides" else 0}) == NULL, name
    for name in ("k", "v", "kc", "vc"):
        assert append(lib, **{name: FAKE + 8}) == ALIGN, name
    assert append(lib, tokens=2) == SHAPE and append(lib, tokens=-1, cu=FAKE) == SHAPE and append(lib, B=-1) == SHAPE
    assert append(lib, page=20) == VALUE and append(lib, D=32) == UNSUP
    assert append(lib, strides=(8192, 128, 64, 8192, 128, 4)) == ALIGN
    assert append(lib, tokens=0, cu=FAKE) == OK and append(lib, B=0, tokens=0) == OK


def seq_map(cu, T, s):
    """The library's map of a packed sequence: first row, rows, first chunk slot."""
    clamp = lambda x, lo, hi: max(lo, min(hi, x))
    b = clamp(cu[s], 0, T)
    e = clamp(cu[s + 1], b, T)
    return b, e - b, b // 64 + s


def test_packed_maps_stay_inside():
    rng = random.Random(0)
    for n in range(3000):
        T, N = rng.randint(1, 400), rng.randint(1, 9)
        if n % 2:  # as documented
            cu = sorted(rng.choice([0, T, rng.randint(0, T)]) for _ in range(N + 1))
        else:      # anything
            cu = [rng.randint(-300, 700) for _ in range(N + 1)]
        slots = T // 64 + N
        used = {}
        for s in range(N):
            row0, rows, slot0 = seq_map(cu, T, s)
            chunks = (rows + 63) // 64
            assert 0 <= row0 and row0 + rows <= T
            assert 0 <= slot0 and slot0 + chunks <= slots
            for c in range(chunks):
                if n % 2:
                    assert slot0 + c not in used
                used[slot0 + c] = (s, c)
        if n % 2:  # the way back: the last sequence whose first slot is not behind the slot
            for slot in range(slots):
                s = max([i for i in range(N) if cu[i] // 64 + i <= slot], default=0)
                row0, rows, slot0 = seq_map(cu, T, s)
                c = slot - slot0
                found = (s, c) if 0 <= c < (rows + 63) // 64 else None
                assert found == used.get(slot), (cu, slot)


def test_key_heads_without_value_heads_are_refused(lib):
    # their gradients would have no kernel to write them
    assert scalar(lib, Hk=2, Hv=0) == SHAPE and scalar(lib, True, Hk=2, Hv=0) == SHAPE and step(lib, Hk=2, Hv=0) == SHAPE


def test_token_numbers_fit_in_32_bits(lib):
    assert attn(lib, page=1 << 20, max_pages=2047, ws_bytes=0) == WS  # past the check of sizes
    assert attn(lib, page=1 << 20, max_pages=2048) == SHAPE


def test_long_tables_of_many_rows(lib):
    # as many places as the line of rows can number, and one row more
    past = lambda **kw: attn(lib, page=1024, strides=(1 << 20, 128, 64) * 2, ws_bytes=0, **kw)
    assert past(B=512, Hq=64, Hkv=8, max_pages=1024) == WS   # 4096 rows of 2^20 tokens
    assert past(B=2048, Hq=64, Hkv=8, max_pages=256) == WS
    rows = (2 ** 31 - 1) // (2 ** 15 + 6)
    assert past(B=rows, Hq=16, Hkv=1, max_pages=1024) == WS
    assert past(B=rows + 1, Hq=16, Hkv=1, max_pages=1024) == SHAPE
    assert past(B=rows // 2 + 1, Hq=17, Hkv=1, max_pages=1024) == SHAPE  # two groups of heads
    assert past(B=rows, Hq=1, Hkv=1, max_pages=1024, dtype=F32) == SHAPE  # units of 16 tokens
    assert past(B=rows + 1, Hq=1, Hkv=1, max_pages=1024, window=5000) == WS  # what the window leaves of them
    assert past(B=2 ** 31 // 7, Hq=1, Hkv=1, max_pages=0) == WS and past(B=2 ** 31 // 7 + 1, Hq=1, max_pages=0) == SHAPE


def test_launches_fit_in_32_bits_of_threads(lib):
    # past that a launch fails, after earlier ones of the same call perhaps: such sizes are refused before any
    odd = FAKE + 8  # not aligned: the next refusal, so that no call here gets as far as a launch
    pieces = lambda n, **kw: append(lib, k=odd, cu=FAKE, tokens=n, Hkv=8, D=128, **kw)
    assert pieces(2 ** 25 - 1) == ALIGN and pieces(2 ** 25) == SHAPE           # 128 pieces of 16 bytes a token
    assert pieces(2 ** 24 - 1, dtype=F32) == ALIGN and pieces(2 ** 24, dtype=F32) == SHAPE
    assert append(lib, cu=FAKE, tokens=2 ** 31 - 1, Hkv=2 ** 31 - 1, D=128) == SHAPE
    rows = lambda b: step(lib, [odd] + [FAKE] * 6, B=b, dk=128, dv=128, states=1)
    assert rows(2 ** 24 - 1) == ALIGN and rows(2 ** 24) == SHAPE               # two workgroups of 128 threads a row
    for bwd in (False, True):
        chains = lambda n, **kw: scalar(lib, bwd, N=n, T=1, dk=128, dv=128, ws=0, **kw)
        most = 2 ** 32 // 640 // 4                                             # four workgroups of 640 threads
        assert chains(most - 1) == WS and chains(most + 1) == SHAPE
    assert g2.gdr2_scalar_workspace_bytes(2 ** 32 // 640 // 4 + 1, 1, 1, 1, 128, 128) == 0


def test_marks_of_leaves_live_as_long_as_their_graphs():
    import torch
    a, b = torch.randn(3, requires_grad=True), torch.randn(3)
    marks = lambda: g2._accumulation_streams((a, b, None, a * 2))
    assert len(marks()) == 1  # leaves that want a gradient
    y = a * 3
    marks()[0].setdefault("gdr2_stream", 7)
    assert marks()[0]["gdr2_stream"] == 7
    y.sum().backward()
    assert marks()[0]["gdr2_stream"] == 7
    del y
    assert "gdr2_stream" not in marks()[0]
    with torch.inference_mode():
        assert marks() == []


def test_calls_without_tokens_have_no_launch_to_fit(lib):
    for bwd in (False, True):
        n = 14 if bwd else 8
        assert scalar(lib, bwd, [0] * n, N=1 << 22, T=0, dk=128, dv=128, ws=0) == OK
    assert step(lib, [0] * 7, B=1 << 25, T=0, states=1) == OK


def test_nothing_is_saved_where_no_gradient_is_wanted(monkeypatch):
    import types

    import torch
    saved = []

    def forward(q, *a, save_for_bwd=False, **kw):
        saved.append(save_for_bwd)
        return q * 1, torch.zeros(1), torch.zeros(1)

    monkeypatch.setattr(g2, "gdr2_scalar_fwd", forward)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=1))
    plain, wants = torch.randn(2), torch.randn(2, requires_grad=True)
    f = g2.GDR2ScalarFunction.apply
    assert not f(*[plain] * 5)[0].requires_grad and not f(*[plain] * 6, None)[0].requires_grad
    with torch.no_grad():
        assert not f(*[wants] * 5)[0].requires_grad
    with torch.inference_mode():
        f(*[wants] * 5)
    assert saved == [False] * 4
    assert f(wants, *[plain] * 4)[0].requires_grad and f(*[plain] * 5, wants)[0].requires_grad
    assert saved[4:] == [True] * 2


def test_a_captured_backward_with_a_foreign_graph_is_refused(monkeypatch):
    # the check alone, on the CPU: the GPU calls are stand-ins, the stream a number
    import types

    import torch
    now = types.SimpleNamespace(cuda_stream=1)
    capturing = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))
    names = ("dq", "dk", "dv", "dg", "dbeta")
    monkeypatch.setattr(g2, "gdr2_scalar_fwd", lambda q, *a, **kw: (q * 1, torch.zeros(1), torch.zeros(1)))
    monkeypatch.setattr(g2, "gdr2_scalar_bwd",
                        lambda *a, **kw: dict({n: torch.ones(2) for n in names}, dh0=None))
    leaves = [torch.randn(2, requires_grad=True) for _ in range(5)]
    eager, _ = g2.GDR2ScalarFunction.apply(*leaves)
    now.cuda_stream = 2
    capturing.append(True)
    o, _ = g2.GDR2ScalarFunction.apply(*leaves)
    with pytest.raises(RuntimeError, match="cannot capture"):
        o.sum().backward()
    del eager, o, _
    gc.collect()  # the error's traceback held the refused graph
    o, _ = g2.GDR2ScalarFunction.apply(*leaves)
    o.sum().backward()
    assert all(torch.equal(t.grad, torch.ones(2)) for t in leaves)
    # and no second derivative, rather than one without this operator's part
    capturing.clear()
    o, _ = g2.GDR2ScalarFunction.apply(*leaves)
    gr, = torch.autograd.grad(o.sum(), leaves[:1], create_graph=True)
    with pytest.raises(RuntimeError):
        gr.sum().backward()
