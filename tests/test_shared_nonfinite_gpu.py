"""stief_decode_shared_paged and stief_expand_shared_paged with NaN and infinities in rows that ARE
read: they reach the outputs that the definition says, and no others, in each form of the call (one
CTA a sequence, whole sequences, split ones with each way of joining the parts)."""
import pytest
import torch

import decode_attention_stief_b200 as stief
from shared_util import attention, bf, check, pool_of, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")

# (lengths, heads, rank): the odd row stands in the sequence given last
FORMS = {"one CTA": ([200, 64, 130], 16, 128, 0), "whole": ([200, 1, 77] * 60, 8, 64, 3), "sixteen warps": ([9100], 24, 512, 0),
         "four, 128 dims": ([2000, 3000, 1, 700], 48, 512, 1), "four, all dims": ([64] * 20 + [6000] + [300] * 19, 32, 512, 20),
         "a warp a head": ([10] * 20 + [7000, 0] + [257] * 20, 128, 384, 20)}


def _case(form, seed):
    lens, Hq, r, b = FORMS[form]
    gen = torch.Generator().manual_seed(seed)
    pool, table = pool_of(lens, 64, r + 16, gen)
    q = bf(len(lens), Hq, r + 16, gen=gen).to(DEV)
    return lens, r, b, q, pool.to(DEV), table.to(DEV)


def _decode(q, pool, table, lens, r):
    out = torch.full((q.shape[0], q.shape[1], r), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stief.stief_decode_shared_paged(q, pool, table, torch.tensor(lens, dtype=torch.int32, device=DEV), out,
                                    stief.shared_workspace_for(q.shape[0], q.shape[1], r), max(lens), 0.06,
                                    dev_status=status)
    assert int(status.item()) == 0
    return out


def _row(pool, table, b, t):
    return pool[int(table[b, t // 64]), t % 64]


def _others(got, want, b):
    keep = torch.arange(got.shape[0], device=DEV) != b
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_nan_in_a_row(form, where):
    lens, r, b, q, pool, table = _case(form, 1)
    want = _decode(q, pool, table, lens, r)
    t = {"first": 0, "middle": lens[b] // 2, "last": lens[b] - 1}[where]
    _row(pool, table, b, t)[r + 5] = float("nan")  # a position value: every head's score
    got = _decode(q, pool, table, lens, r)
    assert got[b].isnan().all()
    _others(got, want, b)


@pytest.mark.parametrize("form", list(FORMS))
def test_nan_in_a_query(form):
    lens, r, b, q, pool, table = _case(form, 2)
    want = _decode(q, pool, table, lens, r)
    h = q.shape[1] // 2
    q[b, h, 3] = float("nan")
    got = _decode(q, pool, table, lens, r)
    assert got[b, h].isnan().all()
    got[b, h] = want[b, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("form", list(FORMS))
def test_infinite_scores(form):
    """One row scores +inf for the even heads (NaN) and -inf for the odd ones (no weight)."""
    lens, r, b, q, pool, table = _case(form, 3)
    q[b, ::2, r] = 1.0
    q[b, 1::2, r] = -1.0
    t = lens[b] // 3
    want = _decode(q, pool, table, lens, r)
    _row(pool, table, b, t)[r] = float("inf")
    got = _decode(q, pool, table, lens, r)
    _others(got, want, b)
    assert got[b, ::2].isnan().all()
    rows = rows_of(pool.cpu(), table.cpu(), b, lens[b]).to(DEV)
    rows = rows[torch.arange(lens[b], device=DEV) != t][None]
    x, bound = attention(q[b, 1::2].double()[:, None], rows, rows[..., :r], 0.06)
    check(got[b, 1::2], x[:, 0], bound[:, 0])


@pytest.mark.parametrize("form", list(FORMS))
def test_rows_of_nothing_but_minus_infinity(form):
    lens, r, b, q, pool, table = _case(form, 4)
    want = _decode(q, pool, table, lens, r)
    for t in range(lens[b]):
        _row(pool, table, b, t)[r + 1] = float("-inf")
    q[b, :, r + 1] = 1.0
    got = _decode(q, pool, table, lens, r)
    assert got[b].isnan().all()
    _others(got, want, b)


def test_expanded_rows_keep_nan_and_infinities_to_themselves():
    gen = torch.Generator().manual_seed(5)
    pool, table = pool_of([300, 70], 64, 64 + 16, gen)
    pool, table = pool.to(DEV), table.to(DEV)
    W = bf(3, 128, 64, gen=gen, scale=0.125).to(DEV)
    start = torch.tensor([0, 300, 370], dtype=torch.int32, device=DEV)

    def run():
        k, v = (torch.zeros((370, 3, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        pe = torch.zeros((370, 16), dtype=torch.bfloat16, device=DEV)
        stief.stief_expand_shared_paged(pool, table, start, W, W, k, v, pe)
        return k, v, pe

    want = run()
    _row(pool, table, 0, 130)[7], _row(pool, table, 1, 3)[64 + 2] = float("nan"), float("inf")
    _row(pool, table, 0, 131)[7] = float("inf")
    k, v, pe = run()
    assert k[130].isnan().all() and v[130].isnan().all() and pe[303, 2] == float("inf")
    sign = W[:, :, 7].sign().float() * float("inf")
    assert torch.equal(k[131].float(), sign) and torch.equal(v[131].float(), sign)
    pe[303, 2] = want[2][303, 2]
    for x, y in zip((k, v, pe), want):
        rows = [i for i in range(370) if i not in (130, 131)]
        assert torch.equal(x[rows], y[rows])
    assert torch.equal(pe, want[2])
