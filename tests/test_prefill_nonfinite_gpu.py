"""stief_prefill_attention with NaN and infinities among the queries and keys that ARE seen: every
form of the kernel gives what the definition gives, whatever the number of tiles.

A score of NaN or +inf makes its row NaN (inf - inf), a score of -inf weighs nothing, and a row
whose scores are all -inf is 0 / 0.  Rows that do not see the odd key are as without it.
"""
import pytest
import torch

import decode_attention_stief_b200 as stief
from shared_util import attention, bf, check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")

# (queries, keys, heads, KV heads, position values): eight, four and two CTAs share a tile's keys, a
# CTA a tile, and pairs of CTAs
FORMS = {"split8": (3, 5000, 8, 1, 0), "split8 packed": (40, 5000, 8, 1, 16), "split8 positions": (1, 1037, 4, 4, 64),
         "split4": (130, 8250, 24, 24, 64), "split2": (300, 1100, 40, 40, 0), "one": (300, 300, 4, 2, 0),
         "one positions": (77, 90, 8, 1, 16), "pairs": (513, 1400, 40, 40, 64)}


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(form, seed):
    nq, nk, Hq, Hkv, dr = FORMS[form]
    gen = torch.Generator().manual_seed(seed)
    shapes = ((nq, Hq, 128 + dr), (nk, Hkv, 128), (nk, Hkv, 128), (nk, dr))
    return [bf(*s, gen=gen).to(DEV) for s in shapes]


def _run(q, k, v, pe, scale):
    """The output, and the definition's with its bounds: rows in 64 bits, NaN where they are NaN."""
    nq, Hq, w = q.shape
    nk, Hkv, _ = k.shape
    out = torch.full((nq, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    status = _i([0])
    stief.stief_prefill_attention(q, k, v, _i([0, nq]), _i([0, nk]), out, nq, scale,
                                  k_pe=pe if pe.shape[1] else None, dev_status=status)
    assert int(status.item()) == 0
    kk = torch.cat([k, pe[:, None].expand(-1, Hkv, -1)], 2).double()
    kk, vv = (x.repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (kk, v.double()))
    hidden = torch.arange(nk, device=DEV)[None, :] > torch.arange(nq, device=DEV)[:, None] + nk - nq
    qq = q.double().transpose(0, 1)
    scores = (qq @ kk.transpose(1, 2) * scale).masked_fill(hidden, -torch.inf)
    dead = torch.softmax(scores, -1).isnan().any(-1)  # [Hq, nq]
    return out.transpose(0, 1), dead, (qq, kk, vv, hidden)


def _same(got, dead, parts, scale, odd=None):
    """NaN in every value of the dead rows, the definition's values in the others (computed with the
    odd keys left out, which no live row gives a weight)."""
    qq, kk, vv, hidden = parts
    if odd is not None:
        hidden = hidden.clone()
        hidden[:, odd] = True
        kk = kk.clone()
        kk[:, odd] = 0.0
    want, bound = attention(torch.where(qq.isfinite(), qq, 0.0), kk, vv, scale, hidden)
    assert got[dead].isnan().all()
    check(got[~dead], want[~dead], bound[~dead])


def _heads(parts, of):
    return tuple(x[of] for x in parts[:3]) + (parts[3],)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_nan_in_a_seen_key(form, where):
    q, k, v, pe = _inputs(form, 1)
    nq, nk = q.shape[0], k.shape[0]
    at = {"first": 0, "middle": nk // 2, "last": nk - 1 - nq // 2}[where]
    k[at, 0, 5] = float("nan")
    got, dead, parts = _run(q, k, v, pe, 0.1)
    assert dead.any()
    g = q.shape[1] // k.shape[1]  # heads of the KV head with the odd key, and the others
    assert not dead[g:].any()
    _same(got[:g], dead[:g], _heads(parts, slice(0, g)), 0.1, odd=at)
    if g < q.shape[1]:
        _same(got[g:], dead[g:], _heads(parts, slice(g, None)), 0.1)


@pytest.mark.parametrize("form", [f for f in FORMS if FORMS[f][4]])
def test_nan_in_a_seen_position_value(form):
    q, k, v, pe = _inputs(form, 2)
    at = k.shape[0] // 3
    pe[at, 3] = float("nan")
    got, dead, parts = _run(q, k, v, pe, 0.1)
    assert dead.any()
    _same(got, dead, parts, 0.1, odd=at)


@pytest.mark.parametrize("form", list(FORMS))
def test_nan_in_a_query(form):
    q, k, v, pe = _inputs(form, 3)
    q[q.shape[0] // 2, 0, 7] = float("nan")
    got, dead, parts = _run(q, k, v, pe, 0.1)
    assert int(dead.sum()) == 1
    _same(got, dead, parts, 0.1)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_infinite_scores(form, scale):
    """One key scores +inf for half of the heads (NaN rows) and -inf for the others (no weight)."""
    q, k, v, pe = _inputs(form, 4)
    at = k.shape[0] // 2
    k[at, :, 0] = float("inf")
    q[:, :, 0] = 1.0
    q[:, ::2, 0] = -1.0
    got, dead, parts = _run(q, k, v, pe, scale)
    _same(got, dead, parts, scale, odd=at)


@pytest.mark.parametrize("form", list(FORMS))
def test_rows_of_nothing_but_minus_infinity(form):
    q, k, v, pe = _inputs(form, 5)
    k[:, :, 0] = float("inf")
    q[:, :, 0] = 1.0
    q[0, 0, 0] = q[-1, -1, 0] = -1.0
    got, dead, _ = _run(q, k, v, pe, 0.1)
    assert dead.all() and got.isnan().all()


@pytest.mark.parametrize("form", list(FORMS))
def test_nan_and_infinity_in_a_value_that_every_query_sees(form):
    q, k, v, pe = _inputs(form, 6)
    v[0, :, 3], v[0, :, 4] = float("nan"), float("inf")
    got, dead, (qq, kk, vv, hidden) = _run(q, k, v, pe, 0.1)
    seen = ~hidden[:, 0]
    assert got[:, seen, 3].isnan().all() and not got[:, :, 5:].isnan().any()
    assert (got[:, seen, 4] == float("inf")).all()
    vv = vv.clone()
    vv[:, 0, 3:5] = 0.0
    want, bound = attention(qq, kk, vv, 0.1, hidden)
    check(got[:, :, 5:], want[:, :, 5:], bound[:, :, 5:])
