"""stief_plan_pages and stief_append_shared_paged against their definitions, exactly."""
import numpy as np
import pytest
import torch

import decode_attention_stief_b200 as stief
from shared_util import bf, plan_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def _state(rng, B, hi, thi, page_size, max_pages, spare=5):
    lens = rng.integers(0, hi + 1, B)
    new = rng.integers(0, thi + 1, B)
    held = -(-lens // page_size)
    num = int(held.sum() + (-(-(lens + new) // page_size) - held).sum()) + spare
    ids = rng.permutation(num).astype(np.int32)
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, : held[b]] = ids[at: at + held[b]]
        at += held[b]
    free = np.full(num, -9, np.int32)
    free[: num - at] = ids[at:]
    return new, lens, table, free, num - at


def _run(new, lens, table, free, count, page_size, max_tokens, ws=None, in_place=False):
    B = len(new)
    ws = stief.plan_workspace() if ws is None else ws
    t, ln, ct = _i(table), _i(lens), _i([count])
    slots = None if max_tokens is None else torch.full((max_tokens,), 77, dtype=torch.int32, device=DEV)
    qs, ks = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(B + 1, dtype=torch.int32, device=DEV)
    lo, co = (ln, ct) if in_place else (torch.empty_like(ln), torch.empty_like(ct))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stief.stief_plan_pages(_i(new), ln, t, _i(free), ct, slots, qs, ks, lo, co, ws, page_size, dev_status=status)
    bits = int(status.item())
    assert int(ws.count_nonzero()) == 0
    return (t.cpu().numpy(), None if slots is None else slots.tolist(), qs.tolist(), ks.tolist(), lo.tolist(),
            int(co.item()), bits)


def _same(got, want):
    assert np.array_equal(got[0], want[0])
    if got[1] is not None:
        assert got[1] == list(want[1])
    assert got[2:] == tuple(want[2:])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi,thi,page_size", [(1, 0, 1, 64), (1, 63, 2, 64), (7, 300, 1, 64), (64, 1000, 200, 128),
                                                (1025, 130, 90, 64), (8192, 200, 3, 192)])
def test_plan_matches_its_definition(B, hi, thi, page_size, in_place):
    rng = np.random.default_rng(B + hi)
    s = _state(rng, B, hi, thi, page_size, (hi + thi) // page_size + 2)
    n = int(s[0].sum()) + 13
    _same(_run(*s, page_size, n, in_place=in_place), plan_reference(*s, page_size, n))


def test_plan_over_many_ctas_in_place():
    """More slots than one CTA writes: the lengths are updated only once every CTA has read them."""
    rng = np.random.default_rng(3)
    s = _state(rng, 300, 2000, 4000, 64, 100)
    n = int(s[0].sum()) + 20001
    want = plan_reference(*s, 64, n)
    ws = stief.plan_workspace()
    for _ in range(5):
        _same(_run(*s, 64, n, ws=ws, in_place=True), want)


def test_plan_without_optional_outputs():
    rng = np.random.default_rng(4)
    s = _state(rng, 9, 500, 70, 64, 12)
    _same(_run(*s, 64, None), plan_reference(*s, 64, None))
    t, ct = _i(s[2]), _i([s[4]])
    stief.stief_plan_pages(_i(s[0]), _i(s[1]), t, _i(s[3]), ct, None, None, None, None, ct, stief.plan_workspace(), 64)
    want = plan_reference(*s, 64, None)
    assert np.array_equal(t.cpu().numpy(), want[0]) and int(ct.item()) == want[5]


def test_plan_refusals():
    """Each refused sequence keeps its length and entries; the others get theirs."""
    ps, cap_pages = 64, 4
    #        ok  neg L  L>cap  T<0  L+T>cap  rest  tail unmapped  ok
    lens = [10, -1, 300, 5, 250, 64, 70, 63]
    new = [100, 1, 1, -4, 7, 0, 3, 2]
    table = np.full((8, cap_pages), -1, np.int32)
    table[0, 0], table[4], table[5, 0], table[6, 0], table[7, 0] = 3, [4, 5, 6, 7], 8, 9, 10
    free = np.array([20, 21, 22, 23] + [-5] * 26, np.int32)
    for max_tokens in (None, 200):
        want = plan_reference(new, lens, table, free, 4, ps, max_tokens)
        assert want[6] == 5 and want[4] == [110, -1, 300, 5, 250, 64, 70, 65]
        _same(_run(new, lens, table, free, 4, ps, max_tokens), want)


def test_plan_runs_out_of_pages_and_of_tokens():
    ps = 64
    table = np.full((5, 6), -1, np.int32)
    table[3, 0] = 2
    lens, new, free = [0, 0, 0, 5, 0], [64, 200, 1, 20, 64], np.arange(10, 22, dtype=np.int32)[::-1].copy()
    for count in (0, 1, 3, 5, 6, 99, -2):
        want = plan_reference(new, lens, table, free, count, ps, 400)
        _same(_run(new, lens, table, free, count, ps, 400), want)
    for max_tokens in (1, 64, 264, 284, 285, 349):
        want = plan_reference(new, lens, table, free, 12, ps, max_tokens)
        _same(_run(new, lens, table, free, 12, ps, max_tokens), want)


def test_plan_captured_decode_loop():
    """One captured in-place step, replayed: the lengths and the table grow as if called."""
    ps, B, steps = 64, 33, 200
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 100, B)
    new, lens, table, free, count = _state(rng, B, 100, 0, ps, 6, spare=B * 5)
    new = np.ones(B, np.int64)
    t, ln, ct, fr = _i(table), _i(lens), _i([count]), _i(free)
    one, ws = _i(new), stief.plan_workspace()
    slots = torch.empty(B, dtype=torch.int32, device=DEV)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        stief.stief_plan_pages(one, ln, t, fr, ct, slots, None, None, ln, ct, ws, ps)
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    lens = [int(n) for n in lens]
    for _ in range(steps):
        table, want_slots, _, _, lens, count, bits = plan_reference(new, lens, table, free, count, ps, B)
        assert bits == 0
    assert np.array_equal(t.cpu().numpy(), table) and ln.tolist() == lens and int(ct.item()) == count
    assert slots.tolist() == want_slots


@pytest.mark.parametrize("N,r,dr", [(1, 512, 64), (3, 16, 0), (130, 96, 16), (5000, 512, 64), (777, 128, 48)])
def test_append_rows(N, r, dr):
    gen = torch.Generator().manual_seed(N)
    ps, num = 64, N // 64 + 3
    both = bf(N, r + dr + 24, gen=gen).to(DEV)  # rows inside a wider matrix
    c, pe = both[:, 8: 8 + r], both[:, r + 16: r + 16 + dr]
    slots = torch.randperm(num * ps, generator=gen)[:N].to(torch.int32)
    slots[::5] = -1 - slots[::5] % 3
    pool = bf(num, ps, r + dr, gen=gen).to(DEV)
    want = pool.clone().view(-1, r + dr)
    kept = (slots >= 0).to(DEV)
    want[slots.to(DEV)[kept].long()] = torch.cat([c, pe], 1)[kept]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stief.stief_append_shared_paged(c, pe if dr else None, slots.to(DEV), pool, dev_status=status)
    assert torch.equal(pool.view(-1, r + dr).view(torch.int16), want.view(torch.int16)) and int(status.item()) == 0


def test_append_slot_past_the_pool():
    pool = torch.zeros((2, 64, 48), dtype=torch.bfloat16, device=DEV)
    c, pe = bf(3, 32).to(DEV), bf(3, 16).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stief.stief_append_shared_paged(c, pe, _i([127, 128, 2 ** 31 - 1]), pool, dev_status=status)
    assert int(status.item()) == stief.DEV_CAPACITY_OVERFLOW
    assert torch.equal(pool[1, 63], torch.cat([c[0], pe[0]])) and int(pool.count_nonzero()) <= 48
    stief.stief_append_shared_paged(c[:0], pe[:0], _i([]), pool)  # no rows: nothing to do
