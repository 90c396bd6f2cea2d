"""stief_prefill_attention with NaN and infinities in value rows that some queries of the same
sequence do not see: they reach the queries that do, and no others, in each form of the kernel."""
import pytest
import torch

import decode_attention_stief_b200 as stief
from shared_util import attention, bf, check
from test_prefill_nonfinite_gpu import FORMS, _i, _inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _run(q, k, v, pe, qs, ks, scale):
    out = torch.full((q.shape[0], q.shape[1], 128), 7.0, dtype=torch.bfloat16, device=DEV)
    status = _i([0])
    stief.stief_prefill_attention(q, k, v, _i(qs), _i(ks), out, max(b - a for a, b in zip(qs, qs[1:])), scale,
                                  k_pe=pe if pe.shape[1] else None, dev_status=status)
    assert int(status.item()) == 0
    return out


def _want(q, k, v, pe, scale):
    """The definition over the keys that a query sees, in 64 bits: [Hq, nq, 128] of finite sums and their
    bounds, and of the sums of the seen values that are not finite (0: none)."""
    nq, Hq, _ = q.shape
    nk, Hkv, _ = k.shape
    kk = torch.cat([k, pe[:, None].expand(-1, Hkv, -1)], 2).double()
    kk, vv = (x.repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (kk, v.double()))
    hidden = torch.arange(nk, device=DEV)[None, :] > torch.arange(nq, device=DEV)[:, None] + nk - nq
    clean = torch.where(vv.isfinite(), vv, 0.0)
    o, bound = attention(q.double().transpose(0, 1), kk, clean, scale, hidden)
    odd = torch.zeros_like(o)
    for j in (~v.isfinite()).flatten(1).any(1).nonzero().flatten().tolist():
        term = torch.where(vv[:, j].isfinite(), 0.0, vv[:, j])
        odd = odd + torch.where(hidden[:, j][None, :, None], 0.0, term[:, None, :])
    return o, bound, odd


def _check(got, o, bound, odd):
    got = got.transpose(0, 1)
    fine = odd == 0
    check(got[fine], o[fine], bound[fine])
    assert torch.equal(got[~fine].double().nan_to_num(nan=3.0), odd[~fine].nan_to_num(nan=3.0))


@pytest.mark.parametrize("form", list(FORMS))
def test_single_values(form):
    """NaN and infinities in a few places near the diagonal and before it."""
    q, k, v, pe = _inputs(form, 11)
    nq, nk = q.shape[0], k.shape[0]
    for n, (back, dim, x) in enumerate([(0, 3, "nan"), (nq // 2, 4, "inf"), (nq // 3, 5, "-inf"), (nq // 3 + 1, 5, "inf"),
                                        (nq - 1, 127, "nan"), (min(nk - 1, nq + 40), 64, "inf")]):
        v[nk - 1 - back, :, dim] = float(x)
    got = _run(q, k, v, pe, [0, nq], [0, nk], 0.1)
    _check(got, *_want(q, k, v, pe, 0.1))


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("part", [0.5, 0.9])
def test_every_value_from_a_token_on(form, part):
    """All values of the last tokens are NaN, as after a token that went wrong."""
    q, k, v, pe = _inputs(form, 12)
    nq, nk = q.shape[0], k.shape[0]
    at = nk - nq + int(nq * part)
    v[at:] = float("nan")
    got = _run(q, k, v, pe, [0, nq], [0, nk], -0.1)
    see = torch.arange(nq, device=DEV) + nk - nq >= at
    assert got[see].isnan().all()
    clean = v.clone()
    clean[at:] = 0.0
    o, bound, _ = _want(q, k, clean, pe, -0.1)
    check(got.transpose(0, 1)[:, ~see], o[:, ~see], bound[:, ~see])


@pytest.mark.parametrize("form", list(FORMS))
def test_every_value_is_nan(form):
    q, k, v, pe = _inputs(form, 13)
    v.fill_(float("nan"))
    assert _run(q, k, v, pe, [0, q.shape[0]], [0, k.shape[0]], 0.1).isnan().all()


@pytest.mark.parametrize("Hq,Hkv,dr", [(4, 2, 0), (6, 2, 16), (40, 40, 64)])
def test_ragged_sequences(Hq, Hkv, dr):
    """Several sequences with odd values near their ends, cached tokens before some, queries that see
    nothing in one; scores far apart, so that the running reference moves."""
    nq, nk = [130, 1, 77, 300], [130, 90, 70, 900]
    gen = torch.Generator().manual_seed(14)
    q, k, v, pe = (bf(*s, gen=gen).to(DEV) for s in ((508, Hq, 128 + dr), (1190, Hkv, 128), (1190, Hkv, 128), (1190, dr)))
    q[:, :, 0] = 20.0
    k[:, :, 0] = torch.linspace(0.0, 12.0, 1190, device=DEV)[:, None].to(torch.bfloat16)
    qs, ks = [0, 130, 131, 208, 508], [0, 130, 220, 290, 1190]
    for b in range(4):
        v[ks[b + 1] - 1, :, 1], v[ks[b + 1] - min(50, nq[b]), :, 2] = float("nan"), float("-inf")
    got = _run(q, k, v, pe, qs, ks, 0.3)
    for b in range(4):
        i, j = slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1])
        _check(got[i], *_want(q[i], k[j], v[j], pe[j], 0.3))


def test_captured_call_with_odd_values_later():
    """The rows are looked at on the GPU: a graph captured with finite values does the same."""
    q, k, v, pe = _inputs("one", 15)
    nq, nk = q.shape[0], k.shape[0]
    qs, ks, out = _i([0, nq]), _i([0, nk]), torch.zeros((nq, q.shape[1], 128), dtype=torch.bfloat16, device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        stief.stief_prefill_attention(q, k, v, qs, ks, out, nq, 0.1)
    for at in (None, 100, 255):
        if at is not None:
            v[at, :, 9] = float("nan")
        graph.replay()
        torch.cuda.synchronize()
        _check(out, *_want(q, k, v, pe, 0.1))
