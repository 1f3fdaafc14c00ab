"""Host-only checks (no GPU) of whole-sequence attention, trees of drafts and the cache's pages: sizes, refusals before
any launch, and the plain references that the GPU tests compare with."""
import ctypes
import math
import os
import random

import pytest
import torch

import gated_delta_rule_gdr2_amd as g2
import prompt_refs as ref

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


def fwd(lib, q=FAKE, k=FAKE, v=FAKE, strides=None, cu=None, o=FAKE, lse=FAKE, rest=FAKE, N=1, T=64, Hq=2, Hkv=1, D=64,
        scale=0.1, window=0, dtype=BF):
    st = None if strides is None else I64x6(*strides)
    return lib.gdr2_attn_fwd(q, k, v, st, cu, o, lse, rest, N, T, Hq, Hkv, D, scale, window, dtype, 0, None)


def bwd(lib, q=FAKE, k=FAKE, v=FAKE, strides=None, o=FAKE, lse=FAKE, rest=FAKE, dout=FAKE, cu=None, dq=FAKE, dk=FAKE,
        dv=FAKE, N=1, T=64, Hq=2, Hkv=1, D=64, scale=0.1, window=0, dtype=BF, ws=FAKE, ws_bytes=1 << 40):
    st = None if strides is None else I64x6(*strides)
    return lib.gdr2_attn_bwd(q, k, v, st, o, lse, rest, dout, cu, dq, dk, dv, N, T, Hq, Hkv, D, scale, window, dtype, 0,
                             ws, ws_bytes, None)


def tree(lib, q=FAKE, parents=FAKE, k=FAKE, v=FAKE, strides=(8192, 128, 64) * 2, table=FAKE, starts=FAKE, o=FAKE, lse=FAKE,
         B=1, T=3, Hq=2, Hkv=1, D=64, pages=4, page=64, max_pages=4, scale=0.1, window=0, dtype=BF, ws=FAKE,
         ws_bytes=1 << 40):
    st = None if strides is None else I64x6(*strides)
    return lib.gdr2_attn_tree(q, parents, k, v, st, table, starts, o, lse, B, T, Hq, Hkv, D, pages, page, max_pages, scale,
                              window, dtype, ws, ws_bytes, None)


def keep(lib, k=FAKE, v=FAKE, strides=(8192, 128, 64) * 2, table=FAKE, starts=FAKE, path=FAKE, lengths=FAKE, B=1, P=3,
         Hkv=1, D=64, pages=4, page=64, max_pages=4, dtype=BF):
    st = None if strides is None else I64x6(*strides)
    return lib.gdr2_kv_keep(k, v, st, table, starts, path, lengths, B, P, Hkv, D, pages, page, max_pages, dtype, None)


def pages(lib, lengths=FAKE, counts=FAKE, table=FAKE, free=FAKE, num_free=FAKE, new=FAKE, cu=FAKE, slots=FAKE, B=1,
          tokens=1, pages=4, page=64, max_pages=4):
    return lib.gdr2_kv_pages(lengths, counts, table, free, num_free, new, cu, slots, B, tokens, pages, page, max_pages, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_prompt_refusals(lib, call):
    last = {"ws": 0} if call is bwd else {"window": -1}  # the refusal that a call right in all else ends with
    end = WS if call is bwd else VALUE
    need = ["q", "k", "v", "o"] + (["lse", "dout", "dq", "dk", "dv"] if call is bwd else [])
    assert call(lib, **last) == end
    for name in need:
        assert call(lib, **{name: 0}) == NULL, name
    for name in [n for n in need if n != "lse"] + ["rest"] + (["ws"] if call is bwd else []):
        assert call(lib, **{name: FAKE + 8}) == ALIGN, name
    assert call(lib, lse=FAKE + 2) == ALIGN and call(lib, lse=FAKE + 4, **last) == end
    assert call(lib, rest=0, **last) == end
    assert call(lib, strides=(128, 64, 64, 64, 60, 64)) == ALIGN and call(lib, strides=(-8, 8, 8, 8, 8, 8)) == ALIGN
    assert call(lib, strides=(512, 64) * 3, **last) == end
    assert call(lib, Hq=3, Hkv=2) == SHAPE and call(lib, N=-1) == SHAPE and call(lib, T=-1) == SHAPE
    assert call(lib, Hq=3, Hkv=0) == SHAPE
    assert call(lib, D=96) == UNSUP and call(lib, dtype=9) == UNSUP
    assert call(lib, T=2 ** 31 - 1) == SHAPE and call(lib, N=1 << 12, T=1 << 20) == SHAPE
    assert call(lib, N=1 << 20, T=1, Hq=8) == SHAPE  # 2^23 workgroups
    for s in (math.inf, math.nan, -math.inf):
        assert call(lib, scale=s) == VALUE
    assert call(lib, window=-1) == VALUE
    for none in (dict(N=0), dict(T=0), dict(Hq=0, Hkv=0), dict(N=0, cu=FAKE)):
        assert call(lib, **none, **{n: 0 for n in need}) == OK


def test_prompt_workspace_sizes(lib):
    f = g2.gdr2_attn_bwd_workspace_bytes
    assert f(2, 100, 4, 4, 64) == f(1, 200, 4, 4, 64) == f(7, 200, 4, 4, 64, packed=True) == 200 * 4 * 8
    assert f(1, 200, 8, 2, 64) == 200 * 8 * 8 + 4 * 200 * 2 * 64 * 8    # parts of dK and dV, a query head each
    assert f(8, 4096, 64, 32, 64) == 8 * 4096 * 64 * 8                  # enough walks without
    assert f(1, 0, 4, 2, 64) == 0 and f(1, 64, 3, 2, 64) == 0 and f(1, 64, 2, 2, 96) == 0
    n = f(1, 64, 2, 1, 64)
    assert bwd(lib, ws_bytes=n - 1) == WS


def test_prompt_workspace_parts_are_aligned(lib):
    # parts of dK and dV, written and read 16 bytes at a time, behind an odd number of rows
    f = g2.gdr2_attn_bwd_workspace_bytes
    for T, Hq, rows in ((33, 3, 800), (1, 3, 32), (2, 3, 48), (7, 5, 288)):
        assert rows % 16 == 0 and 0 <= rows - T * Hq * 8 < 16
        assert f(1, T, Hq, 1, 64) == rows + 2 * Hq * T * 64 * 4
        assert bwd(lib, T=T, Hq=Hq, ws_bytes=f(1, T, Hq, 1, 64) - 1) == WS


def test_tree_refusals(lib):
    need = g2.gdr2_attn_tree_workspace_bytes(1, 3, 2, 1, 64)
    assert need > 0 and g2.gdr2_attn_tree_workspace_bytes(0, 3, 2, 1, 64) == 0
    assert g2.gdr2_attn_tree_workspace_bytes(1, 65, 2, 1, 64) == 0 and g2.gdr2_attn_tree_workspace_bytes(1, 0, 2, 1, 64) == 0
    assert g2.gdr2_attn_tree_workspace_bytes(5, 3, 64, 32, 64) == need  # by the drafts and heads of a key head alone
    for name in ("q", "parents", "k", "v", "table", "starts", "o", "strides"):
        assert tree(lib, **{name: None if name == "strides" else 0}) == NULL, name
    for name in ("q", "k", "v", "o", "ws"):
        assert tree(lib, **{name: FAKE + 8}) == ALIGN, name
    for name in ("parents", "table", "starts", "lse"):
        assert tree(lib, **{name: FAKE + 2}) == ALIGN, name
    assert tree(lib, strides=(8192, 128, 60, 8192, 128, 64)) == ALIGN
    assert tree(lib, Hq=3, Hkv=2) == SHAPE and tree(lib, B=-1) == SHAPE and tree(lib, T=-1) == SHAPE
    assert tree(lib, T=65) == SHAPE and tree(lib, B=1 << 20, T=64, Hq=64) == SHAPE
    assert tree(lib, max_pages=1 << 25) == SHAPE          # 2^31 places in a table
    assert tree(lib, B=1 << 12, max_pages=1 << 18) == SHAPE  # 2^31 places in the line of rows
    assert tree(lib, D=96) == UNSUP and tree(lib, dtype=9) == UNSUP
    for page in (0, 8, 24, -16, 1 << 21):
        assert tree(lib, page=page) == VALUE, page
    assert tree(lib, window=-1) == VALUE and tree(lib, scale=math.nan) == VALUE
    assert tree(lib, ws=0) == WS and tree(lib, ws_bytes=need - 1) == WS
    for none in (dict(B=0), dict(T=0), dict(Hq=0, Hkv=0)):
        assert tree(lib, **none, q=0, parents=0, o=0, ws=0) == OK


def test_keep_and_pages_refusals(lib):
    for name in ("k", "v", "table", "starts", "path", "strides"):
        assert keep(lib, **{name: None if name == "strides" else 0}) == NULL, name
    for name in ("k", "v"):
        assert keep(lib, **{name: FAKE + 8}) == ALIGN, name
    for name in ("table", "starts", "path", "lengths"):
        assert keep(lib, **{name: FAKE + 2}) == ALIGN, name
    assert keep(lib, P=65) == SHAPE and keep(lib, P=-1) == SHAPE and keep(lib, B=-1) == SHAPE
    assert keep(lib, B=2 ** 31 - 1) == SHAPE and keep(lib, D=32) == UNSUP and keep(lib, page=20) == VALUE
    assert keep(lib, B=0, k=0, v=0, starts=0) == OK
    for name in ("lengths", "counts", "table", "free", "num_free", "new", "cu"):
        assert pages(lib, **{name: 0}) == NULL, name
        assert pages(lib, **{name: FAKE + 2}) == ALIGN, name
    assert pages(lib, slots=FAKE + 4) == ALIGN
    for name in ("B", "tokens", "pages", "max_pages"):
        assert pages(lib, **{name: -1}) == SHAPE, name
    assert pages(lib, max_pages=1 << 25) == SHAPE
    for page in (0, 8, 24, -16, 1 << 21):
        assert pages(lib, page=page) == VALUE, page


def test_reference_of_attention_against_autograd():
    gen = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(23, h, 8, generator=gen, dtype=torch.float64) for h in (4, 2, 2, 4))
    cu = [3, 10, 10, 22]
    for window in (0, 1, 4):
        x = [t.clone().requires_grad_() for t in (q, k, v)]
        o, lse, size = ref.attention(*x, cu, -0.4, window)
        (o * do).sum().backward()
        got = ref.gradients(q, k, v, do, cu, -0.4, window)
        for a, b in zip(got[:3], x):
            assert (a - b.grad).abs().max() < 1e-12
        for a, b in zip(got[:3], got[3:6]):
            assert (a.abs() <= b + 1e-12).all()
        # a row by hand
        t, h = 17, 3
        seen = range(max(10, t - window + 1) if window else 10, t + 1)
        w = torch.stack([torch.exp(-0.4 * q[t, h] @ k[j, h // 2]) for j in seen])
        assert (o[t, h] - sum(w[i] * v[j, h // 2] for i, j in enumerate(seen)) / w.sum()).abs().max() < 1e-12
        assert abs(lse[t, h] - w.sum().log()) < 1e-12 and not o[:3].any() and not o[22:].any()


def test_reference_of_trees_and_pages():
    assert ref.lineage([-1, 0, 0, 2], 3) == [3, 2, 0] and ref.lineage([-1, 1, 1], 2) is None
    assert ref.lineage([-2, 0], 1) is None
    rng = random.Random(0)
    for _ in range(50):  # pages: each page has one owner, before and after
        P, B, page = 20, 4, 16
        ids = list(range(P))
        rng.shuffle(ids)
        lengths = [rng.randint(0, 60) for _ in range(B)]
        table = [[ids.pop() for _ in range(-(-n // page))] for n in lengths]
        table = [r + [-1] * (5 - len(r)) for r in table]
        counts = [rng.choice([-1, 0, 1, 5, 40]) for _ in range(B)]
        new, cu, slots, after, stack, top = ref.pages(lengths, counts, table, ids + [0] * (P - len(ids)), len(ids), page, 60)
        owned = [p for r in after for p in r if p >= 0] + stack[:top]
        assert sorted(owned) == list(range(P))
        placed = [x for x in slots if x >= 0]
        assert len(placed) == len(set(placed)) == sum(n - m for n, m, c in zip(new, lengths, counts) if c > 0)


def test_binding_checks_before_any_call():
    cpu = torch.zeros(1, 4, 2, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    for f in (lambda: g2.gdr2_attn_fwd(cpu, cpu, cpu), lambda: g2.gdr2_attn_bwd(cpu, cpu, cpu, cpu, cpu, cpu),
              lambda: g2.gdr2_attn_tree(cpu, i, cpu, cpu, i, i), lambda: g2.gdr2_kv_keep(cpu, cpu, i, i, i),
              lambda: g2.gdr2_kv_pages(i[0], i[0], i, i[0], i[0, :1], page_size=16, max_tokens=4)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused(grad):
    # not dropped, with a derivative of zero as the result, where no gradient is wanted
    import torch.autograd.forward_ad as fw
    x = torch.randn(1, 4, 2, 64)
    gate, state = torch.randn(1, 4, 2), torch.randn(1, 2, 64, 64)
    with torch.set_grad_enabled(grad), fw.dual_level():
        dual = lambda t: fw.make_dual(t, torch.ones_like(t))
        for i in range(3):
            args = [dual(t) if i == j else t for j, t in enumerate((x, x, x))]
            with pytest.raises(NotImplementedError):
                g2.GDR2AttnFunction.apply(*args)
        plain = (x, x, x, gate, gate, state)
        for i in range(6):
            args = [dual(t) if i == j else t for j, t in enumerate(plain)]
            with pytest.raises(NotImplementedError):
                g2.GDR2ScalarFunction.apply(*args)
        for call in (lambda: g2.GDR2AttnFunction.apply(x, x, x), lambda: g2.GDR2ScalarFunction.apply(*plain)):
            with pytest.raises(ValueError):
                call()  # without a tangent: CPU tensors
    with pytest.raises(NotImplementedError):
        torch.func.jvp(lambda t: g2.GDR2AttnFunction.apply(t, t, t), (x,), (x,))
