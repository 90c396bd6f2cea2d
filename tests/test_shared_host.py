"""Argument checks of page planning and the shared-latent calls (host only: no CUDA call)."""
import ctypes

import pytest

import decode_attention_stief_b200 as stief
from decode_attention_stief_b200 import build as stief_build

OK, INVALID, ALIGN, CAPACITY, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    stief_build.build_library()
    return stief.library()


def _call(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*[a[k] for k in order], None, None)


PLAN = dict(new=FAKE, lens=FAKE, table=FAKE, free=FAKE, count=FAKE, slots=FAKE, q=FAKE, kv=FAKE, lens_out=FAKE,
            count_out=FAKE, ws=FAKE, ws_bytes=256, B=4, num_pages=8, page_size=64, max_pages=2, max_tokens=10)


@pytest.mark.parametrize("kw,code", [
    (dict(new=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(count=None), INVALID), (dict(count_out=None), INVALID), (dict(B=0), INVALID), (dict(B=8193), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_size=63), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_pages=1 << 25), INVALID), (dict(max_pages=1 << 25), INVALID), (dict(max_tokens=-1), INVALID),
    (dict(new=FAKE + 2), ALIGN), (dict(slots=FAKE + 1), ALIGN), (dict(kv=FAKE + 3), ALIGN), (dict(ws=FAKE + 8), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=255), WORKSPACE),
])
def test_plan_argument_errors(lib, kw, code):
    assert _call(lib.stief_plan_pages, list(PLAN), PLAN, kw) == code


APPEND = dict(c=FAKE, pe=FAKE, slots=FAKE, pages=FAKE, N=4, r=512, dr=64, sc=512, sp=64, num_pages=8, page_size=64)


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), INVALID), (dict(pe=None), INVALID), (dict(slots=None), INVALID), (dict(pages=None), INVALID),
    (dict(N=-1), INVALID), (dict(r=0), INVALID), (dict(r=520), INVALID), (dict(r=24), INVALID), (dict(r=528), INVALID),
    (dict(dr=80), INVALID), (dict(dr=8), INVALID), (dict(dr=-16), INVALID), (dict(sc=504), INVALID), (dict(sp=56), INVALID),
    (dict(sc=-512), INVALID), (dict(page_size=32), INVALID), (dict(sc=516), ALIGN), (dict(sp=68), ALIGN),
    (dict(c=FAKE + 8), ALIGN), (dict(pe=FAKE + 2), ALIGN), (dict(slots=FAKE + 2), ALIGN), (dict(N=0, c=None), OK),
])
def test_append_argument_errors(lib, kw, code):
    assert _call(lib.stief_append_shared_paged, list(APPEND), APPEND, kw) == code


DECODE = dict(q=FAKE, pages=FAKE, table=FAKE, lens=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, Hq=32, r=512, dr=64,
              num_pages=8, page_size=64, max_pages=4, most=256, scale=0.1)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(pages=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(B=0), INVALID), (dict(B=65536), INVALID), (dict(Hq=0), INVALID), (dict(Hq=257), INVALID),
    (dict(r=8), INVALID), (dict(dr=72), INVALID), (dict(page_size=96), INVALID), (dict(num_pages=0), INVALID),
    (dict(most=-1), INVALID), (dict(most=257), CAPACITY), (dict(scale=float("nan")), INVALID),
    (dict(B=65535, max_pages=1 << 24, most=1 << 30), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=FAKE + 8), ALIGN), (dict(pages=FAKE + 2), ALIGN),
    (dict(out=FAKE + 4), ALIGN), (dict(table=FAKE + 2), ALIGN), (dict(lens=FAKE + 1), ALIGN), (dict(ws=FAKE + 8), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
])
def test_decode_argument_errors(lib, kw, code):
    assert _call(lib.stief_decode_shared_paged, list(DECODE), DECODE, kw) == code


EXPAND = dict(pages=FAKE, table=FAKE, start=FAKE, W_K=FAKE, W_V=FAKE, k=FAKE, v=FAKE, pe=FAKE, B=2, N=100, H=8, d=128,
              r=512, dr=64, num_pages=8, page_size=64, max_pages=4)


@pytest.mark.parametrize("kw,code", [
    (dict(pages=None), INVALID), (dict(table=None), INVALID), (dict(start=None), INVALID), (dict(W_K=None), INVALID),
    (dict(W_V=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(pe=None), INVALID),
    (dict(B=0), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(H=257), INVALID), (dict(d=64), INVALID),
    (dict(r=20), INVALID), (dict(dr=65), INVALID), (dict(page_size=1), INVALID), (dict(W_K=FAKE + 2), ALIGN),
    (dict(k=FAKE + 8), ALIGN), (dict(pe=FAKE + 8), ALIGN), (dict(start=FAKE + 2), ALIGN), (dict(N=0, k=None), OK),
])
def test_expand_argument_errors(lib, kw, code):
    assert _call(lib.stief_expand_shared_paged, list(EXPAND), EXPAND, kw) == code


PREFILL = dict(q=FAKE, k=FAKE, v=FAKE, pe=FAKE, qs=FAKE, ks=FAKE, out=FAKE, B=2, Hq=8, Hkv=2, d=128, dr=64, Nq=100,
               Nkv=120, most=60, scale=0.1)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(pe=None), INVALID),
    (dict(qs=None), INVALID), (dict(ks=None), INVALID), (dict(out=None), INVALID), (dict(B=0), INVALID),
    (dict(Hq=9), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=512, Hkv=512), INVALID), (dict(d=64), INVALID),
    (dict(dr=24), INVALID), (dict(Nq=-1), INVALID), (dict(Nkv=-1), INVALID), (dict(most=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN), (dict(pe=FAKE + 4), ALIGN),
    (dict(out=FAKE + 2), ALIGN), (dict(qs=FAKE + 2), ALIGN), (dict(Nq=0, q=None), OK), (dict(most=0), OK),
    (dict(B=65535, Hq=256, Hkv=256, Nq=1 << 20, most=1 << 20), INVALID),
])
def test_prefill_argument_errors(lib, kw, code):
    assert _call(lib.stief_prefill_attention, list(PREFILL), PREFILL, kw) == code


def test_workspace_sizes(lib):
    assert stief.stief_plan_workspace_bytes() == 256
    assert stief.stief_decode_shared_workspace_bytes(4, 128, 512) > 0
    for bad in ((0, 32, 512), (1, 0, 512), (1, 257, 512), (1, 32, 8), (1, 32, 528)):
        assert stief.stief_decode_shared_workspace_bytes(*bad) == 0
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_binding_refuses_before_any_cuda_call():
    """Wrong types and CPU tensors are refused with the reason, with or without a GPU."""
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros((2, 64, 48), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="new_tokens must be on a CUDA device"):
        stief.stief_plan_pages(i, i, i.view(2, 2), i, i[:1], None, None, None, None, i[:1], i, 64)
    with pytest.raises(TypeError, match="seq_lens|new_tokens"):
        stief.stief_plan_pages(i.float(), i, i.view(2, 2), i, i[:1], None, None, None, None, i[:1], i, 64)
    with pytest.raises((ValueError, TypeError), match="c_new"):
        stief.stief_append_shared_paged(b[0], None, i, b)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        stief.stief_decode_shared_paged(None, b, i, i, b, i, 3, 0.1)
    with pytest.raises(ValueError, match="pages must be on a CUDA device"):
        stief.stief_expand_shared_paged(b, i, i, b, b, b, b)
    with pytest.raises(ValueError, match="q must be on a CUDA device"):
        stief.stief_prefill_attention(b, b, b, i, i, b, 3, 0.1)
