"""stief_prefill_attention against a 64-bit form, and the operators run together."""
import numpy as np
import pytest
import torch

import decode_attention_stief_b200 as stief
import oracle
import stief_inputs as si
from gpu_util import assert_decode_close, f64
from shared_util import attention, bf, check, plan_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _starts(lens, at=0):
    got = [at]
    for n in lens:
        got.append(got[-1] + n)
    return got


def _inputs(nq, nk, Hq, Hkv, dr, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    Q, K = sum(nq) + pad, sum(nk) + pad
    q, k, v = bf(Q, Hq, 128 + dr, gen=gen), bf(K, Hkv, 128, gen=gen), bf(K, Hkv, 128, gen=gen)
    pe = bf(K, dr, gen=gen)
    return [x.to(DEV) for x in (q, k, v, pe)]


def _prefill(q, k, v, pe, qs, ks, max_q, scale, expect=0):
    out = torch.full((q.shape[0], q.shape[1], 128), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stief.stief_prefill_attention(q, k, v, _i(qs), _i(ks), out, max_q, scale, k_pe=pe if pe.shape[1] else None,
                                  dev_status=status)
    assert int(status.item()) == expect
    return out


def _check(got, q, k, v, pe, qs, ks, scale, only=None):
    Hq, Hkv = q.shape[1], k.shape[1]
    for b in range(len(qs) - 1) if only is None else only:
        nq, nk = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        if nq == 0:
            continue
        kk = torch.cat([k[ks[b]: ks[b + 1]], pe[ks[b]: ks[b + 1], None].expand(-1, Hkv, -1)], 2)
        kk, vv = (x.double().repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (kk, v[ks[b]: ks[b + 1]]))
        last = torch.arange(nq, device=DEV)[:, None] + nk - nq
        hidden = torch.arange(nk, device=DEV)[None, :] > last
        want, bound = attention(q[qs[b]: qs[b + 1]].double().transpose(0, 1), kk, vv, scale, hidden)
        check(got[qs[b]: qs[b + 1]].transpose(0, 1), want, bound)


@pytest.mark.parametrize("Hq,Hkv,dr", [(1, 1, 0), (4, 2, 64), (8, 1, 16), (5, 5, 48), (6, 2, 32)])
@pytest.mark.parametrize("nq,nk", [([1], [1]), ([77], [77]), ([128, 129, 1], [128, 129, 1]), ([300], [555]),
                                   ([5, 0, 64, 1], [200, 3, 64, 0]), ([260, 40], [100, 39]), ([513], [513])])
def test_prefill(nq, nk, Hq, Hkv, dr):
    """Whole prompts, chunks behind cached tokens, more queries than keys, empty sequences; the
    rows around the sequences hold NaN or stay as they were."""
    q, k, v, pe = _inputs(nq, nk, Hq, Hkv, dr, sum(nq) + dr, pad=9)
    qs, ks = _starts(nq, 4), _starts(nk, 3)
    for x, s in ((q, qs), (k, ks), (v, ks), (pe, ks)):
        x[: s[0]] = float("nan")
        x[s[-1]:] = float("nan")
    scale = 1.5 / (128 + dr) ** 0.5
    got = _prefill(q, k, v, pe, qs, ks, max(nq), scale)
    _check(got, q, k, v, pe, qs, ks, scale)
    assert torch.all(got[: qs[0]] == 7.0) and torch.all(got[qs[-1]:] == 7.0)


@pytest.mark.parametrize("n,Hq,Hkv,dr", [(2049, 4, 4, 64), (3000, 8, 2, 0)])
def test_prefill_long(n, Hq, Hkv, dr):
    q, k, v, pe = _inputs([n], [n + 700], Hq, Hkv, dr, n)
    got = _prefill(q, k, v, pe, [0, n], [0, n + 700], n, 0.1)
    _check(got, q, k, v, pe, [0, n], [0, n + 700], 0.1)


@pytest.mark.parametrize("scale", [1.0, -0.5, 0.0])
def test_prefill_peaked_and_flat_scores(scale):
    q, k, v, pe = _inputs([400], [400], 4, 2, 64, 77)
    k *= torch.linspace(0.2, 4.0, 400, device=DEV)[:, None, None].to(torch.bfloat16)
    got = _prefill(q, k, v, pe, [0, 400], [0, 400], 400, scale)
    _check(got, q, k, v, pe, [0, 400], [0, 400], scale)


@pytest.mark.parametrize("Hq,Hkv,dr", [(1, 1, 64), (4, 2, 64), (8, 1, 16), (5, 5, 48), (6, 2, 32), (256, 1, 16)])
@pytest.mark.parametrize("nq,nk", [([1], [1]), ([77], [77]), ([128, 129, 1], [128, 129, 1]), ([300], [555]),
                                   ([5, 0, 64, 1], [200, 3, 64, 0]), ([260, 40], [100, 39]), ([513], [513]),
                                   ([257, 31, 383], [321, 1031, 2000])])
def test_prefill_within_long_arrays(nq, nk, Hq, Hkv, dr):
    """The same kinds of batches at the head of arrays of many more rows (a padded batch), which hold
    NaN there: a long walk over the keys is expected, and CTAs work in pairs."""
    q, k, v, pe = _inputs(nq, nk, Hq, Hkv, dr, sum(nq) + dr, pad=9)
    more = 1024 * len(nk)
    k, v, pe = (torch.cat([x, torch.full((more, *x.shape[1:]), float("nan"), dtype=x.dtype, device=DEV)])
                for x in (k, v, pe))
    qs, ks = _starts(nq, 4), _starts(nk, 3)
    for x, s in ((q, qs), (k, ks), (v, ks), (pe, ks)):
        x[: s[0]] = float("nan")
        x[s[-1]:] = float("nan")
    scale = 1.5 / (128 + dr) ** 0.5
    got = _prefill(q, k, v, pe, qs, ks, max(nq), scale)
    _check(got, q, k, v, pe, qs, ks, scale)
    assert torch.all(got[: qs[0]] == 7.0) and torch.all(got[qs[-1]:] == 7.0)


@pytest.mark.parametrize("scale", [1.0, -0.5, 0.0])
def test_prefill_late_peaks_over_a_long_walk(scale):
    q, k, v, pe = _inputs([400], [1400], 4, 4, 64, 79)
    k *= torch.linspace(0.2, 4.0, 1400, device=DEV)[:, None, None].to(torch.bfloat16)
    k[:, :, 0] = torch.linspace(0.0, 9.0, 1400, device=DEV)[:, None].to(torch.bfloat16) * (1 if scale > 0 else -1)
    q[:, :, 0] = 20.0
    got = _prefill(q, k, v, pe, [0, 400], [0, 1400], 400, scale)
    _check(got, q, k, v, pe, [0, 400], [0, 1400], scale)


def test_prefill_bad_rows_over_a_long_walk():
    q, k, v, pe = _inputs([50, 50], [1160, 1160], 2, 2, 16, 5)
    good = _prefill(q, k, v, pe, [0, 50, 100], [0, 1160, 2320], 50, 0.1)
    for qs, ks, most in (([0, 50, 101], [0, 1160, 2320], 60), ([0, 50, 100], [0, 1160, 2321], 50),
                         ([0, 50, 40], [0, 1160, 2320], 50), ([0, 50, 100], [0, 1160, 1159], 50)):
        got = _prefill(q, k, v, pe, qs, ks, most, 0.1, expect=stief.DEV_BAD_LENGTH)
        assert torch.equal(got[:50], good[:50]) and torch.all(got[50:] == 7.0)
    for _ in range(20):  # the same every time
        assert torch.equal(_prefill(q, k, v, pe, [0, 50, 100], [0, 1160, 2320], 50, 0.1), good)


@pytest.mark.parametrize("nq,nk,Hq,Hkv", [
    ([1], [1037], 4, 4), ([3], [5000], 8, 1), ([900], [600], 1, 1), ([1, 1, 1], [5000, 3, 0], 4, 2),       # eight CTAs a tile
    ([130], [8250], 24, 24), ([17, 0, 90], [2000, 700, 1100], 6, 6), ([513], [513], 3, 3),
    ([200, 130], [1300, 1100], 8, 8), ([64] * 6, [640 + 77 * i for i in range(6)], 20, 5), ([70, 450], [64, 1090], 5, 5),  # four
    ([300], [1100], 40, 40), ([260, 40], [2100, 39], 76, 38)])                                             # two
@pytest.mark.parametrize("dr", [0, 16, 64])
def test_prefill_keys_split_over_ctas(nq, nk, Hq, Hkv, dr):
    """Few tiles of queries and long walks; rows of no sequence hold NaN, and some queries, or some of
    the CTAs of a tile, see no key."""
    q, k, v, pe = _inputs(nq, nk, Hq, Hkv, dr, sum(nk) + dr, pad=9)
    qs, ks = _starts(nq, 4), _starts(nk, 3)
    for x, s in ((q, qs), (k, ks), (v, ks), (pe, ks)):
        x[: s[0]] = float("nan")
        x[s[-1]:] = float("nan")
    scale = 1.5 / (128 + dr) ** 0.5
    got = _prefill(q, k, v, pe, qs, ks, max(nq), scale)
    _check(got, q, k, v, pe, qs, ks, scale)
    assert torch.all(got[: qs[0]] == 7.0) and torch.all(got[qs[-1]:] == 7.0)
    for _ in range(5):  # the same every time
        again = _prefill(q, k, v, pe, qs, ks, max(nq), scale)
        assert torch.equal(again[qs[0]: qs[-1]], got[qs[0]: qs[-1]])


@pytest.mark.parametrize("nq", [2, 150])
@pytest.mark.parametrize("at", [0, 1000, 2399])
def test_prefill_one_key_outweighs_a_split_walk(nq, at):
    """All the weight lies in the keys of one of a tile's CTAs, the others' parts vanish."""
    q, k, v, pe = _inputs([nq], [2400 + nq], 4, 4, 16, at + nq)
    q[:, :, 0], k[:, :, 0] = 30.0, 0.0
    k[at, :, 0] = 40.0
    got = _prefill(q, k, v, pe, [0, nq], [0, 2400 + nq], nq, 1.0)
    _check(got, q, k, v, pe, [0, nq], [0, 2400 + nq], 1.0)
    assert torch.equal(got, v[at].expand(nq, 4, 128))


@pytest.mark.parametrize("Hq,Hkv,dr", [(40, 40, 64), (160, 40, 48), (96, 48, 16)])
@pytest.mark.parametrize("nq,nk", [([257, 31, 383], [321, 1031, 2000]), ([300, 200], [555, 100]), ([513], [513])])
def test_prefill_many_heads_within_long_arrays(nq, nk, Hq, Hkv, dr):
    """As many tiles as keep the GPU busy, and a long walk expected: CTAs in pairs."""
    q, k, v, pe = _inputs(nq, nk, Hq, Hkv, dr, sum(nq) + dr, pad=9)
    more = 1024 * len(nk)
    k, v, pe = (torch.cat([x, torch.full((more, *x.shape[1:]), float("nan"), dtype=x.dtype, device=DEV)])
                for x in (k, v, pe))
    qs, ks = _starts(nq, 4), _starts(nk, 3)
    for x, s in ((q, qs), (k, ks), (v, ks), (pe, ks)):
        x[: s[0]] = float("nan")
        x[s[-1]:] = float("nan")
    scale = 1.5 / (128 + dr) ** 0.5
    got = _prefill(q, k, v, pe, qs, ks, max(nq), scale)
    _check(got, q, k, v, pe, qs, ks, scale)
    assert torch.all(got[: qs[0]] == 7.0) and torch.all(got[qs[-1]:] == 7.0)
    for _ in range(5):
        again = _prefill(q, k, v, pe, qs, ks, max(nq), scale)
        assert torch.equal(again[qs[0]: qs[-1]], got[qs[0]: qs[-1]])


@pytest.mark.parametrize("scale", [1.0, -0.5, 0.0])
def test_prefill_many_heads_late_peaks(scale):
    q, k, v, pe = _inputs([400], [1400], 40, 40, 64, 80)
    k *= torch.linspace(0.2, 4.0, 1400, device=DEV)[:, None, None].to(torch.bfloat16)
    k[:, :, 0] = torch.linspace(0.0, 9.0, 1400, device=DEV)[:, None].to(torch.bfloat16) * (1 if scale > 0 else -1)
    q[:, :, 0] = 20.0
    got = _prefill(q, k, v, pe, [0, 400], [0, 1400], 400, scale)
    _check(got, q, k, v, pe, [0, 400], [0, 1400], scale)


def test_prefill_split_captured_with_new_lengths():
    """A graph captured for a long walk, replayed with shorter ones: some CTAs of a tile get nothing."""
    q, k, v, pe = _inputs([60], [3000], 4, 4, 64, 19)
    qs, ks, out = _i([0, 60]), _i([0, 3000]), torch.zeros((60, 4, 128), dtype=torch.bfloat16, device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        stief.stief_prefill_attention(q, k, v, qs, ks, out, 60, 0.1, k_pe=pe)
    for n, m in ((60, 3000), (31, 700), (1, 65), (60, 40), (2, 1), (7, 0)):
        qs.copy_(_i([0, n]))
        ks.copy_(_i([0, m]))
        graph.replay()
        torch.cuda.synchronize()
        _check(out, q, k, v, pe, [0, n], [0, m], 0.1)


@pytest.mark.parametrize("scale", [1.0, -0.5])
@pytest.mark.parametrize("nq,dr", [(400, 0), (30, 16), (400, 16)])
def test_prefill_late_peaks(nq, dr, scale):
    """The largest scores come last and far above the first ones: the running reference moves."""
    q, k, v, pe = _inputs([nq], [400], 8, 2, dr, 78)
    k *= torch.linspace(0.2, 4.0, 400, device=DEV)[:, None, None].to(torch.bfloat16)
    k[:, :, 0] = torch.linspace(0.0, 9.0, 400, device=DEV)[:, None].to(torch.bfloat16) * (1 if scale > 0 else -1)
    q[:, :, 0] = 20.0
    got = _prefill(q, k, v, pe, [0, nq], [0, 400], nq, scale)
    _check(got, q, k, v, pe, [0, nq], [0, 400], scale)


@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (12, 4), (128, 1), (256, 1), (64, 2), (130, 65)])
@pytest.mark.parametrize("dr", [0, 16])
def test_prefill_shared_heads(Hq, Hkv, dr):
    """Groups of query heads that fill a tile's rows, part of them, or do not divide them; sequences
    that end inside a tile, with fewer queries than a tile has room for and with more."""
    for nq, nk in (([9, 1, 0, 33], [9, 90, 5, 20]), ([1] * 4, [1, 64, 65, 300]), ([130], [131])):
        q, k, v, pe = _inputs(nq, nk, Hq, Hkv, dr, Hq + dr, pad=2)
        qs, ks = _starts(nq, 1), _starts(nk, 1)
        got = _prefill(q, k, v, pe, qs, ks, max(nq), 0.1)
        _check(got, q, k, v, pe, qs, ks, 0.1)
        assert torch.all(got[: qs[0]] == 7.0) and torch.all(got[qs[-1]:] == 7.0)


@pytest.mark.parametrize("B,nk", [(6, 700), (2, 700), (3, 100)])
def test_prefill_short_chunks_with_positions(B, nk):
    """Chunks within one tile of queries: many, few, and few over few keys."""
    nq = [128, 1, 65, 17, 0, 100][:B]
    keys = [nk + b for b in range(B)]
    q, k, v, pe = _inputs(nq, keys, 32, 32, 64, B + nk)
    qs, ks = _starts(nq), _starts(keys)
    got = _prefill(q, k, v, pe, qs, ks, 128, 0.09)
    _check(got, q, k, v, pe, qs, ks, 0.09)


def test_prefill_masked_places_hold_nan_and_infinities():
    """Keys and values that no query of a sequence sees belong to its neighbours in the arrays:
    what stands there must not matter."""
    q, k, v, pe = _inputs([70, 70], [70, 70], 4, 4, 16, 3)
    k[70:], v[70:], pe[70:], q[70:] = float("inf"), float("nan"), float("-inf"), float("nan")
    got = _prefill(q, k, v, pe, [0, 70, 140], [0, 70, 140], 70, 0.1)
    _check(got, q, k, v, pe, [0, 70, 140], [0, 70, 140], 0.1, only=[0])


def test_prefill_bad_rows():
    q, k, v, pe = _inputs([50, 50], [60, 60], 2, 2, 0, 5)
    good = _prefill(q, k, v, pe, [0, 50, 100], [0, 60, 120], 50, 0.1)
    for qs, ks, most in (([0, 50, 101], [0, 60, 120], 60), ([0, 50, 100], [0, 60, 121], 50), ([0, 50, 40], [0, 60, 120], 50),
                         ([0, 50, 100], [0, 60, 59], 50)):
        got = _prefill(q, k, v, pe, qs, ks, most, 0.1, expect=stief.DEV_BAD_LENGTH)
        assert torch.equal(got[:50], good[:50]) and torch.all(got[50:] == 7.0)
    got = _prefill(q, k, v, pe, [0, 51, 100], [0, 60, 120], 50, 0.1, expect=stief.DEV_BAD_LENGTH)
    assert torch.all(got[:51] == 7.0)
    none = _prefill(q, k[:0], v[:0], pe[:0], [0, 50, 100], [0, 0, 0], 50, 0.1)
    assert torch.all(none == 0)


def test_prefill_captured_with_new_lengths():
    q, k, v, pe = _inputs([200], [200], 4, 4, 64, 9)
    qs, ks, out = _i([0, 200]), _i([0, 200]), torch.zeros((200, 4, 128), dtype=torch.bfloat16, device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        stief.stief_prefill_attention(q, k, v, qs, ks, out, 200, 0.1, k_pe=pe)
    for n in (200, 131, 1):
        qs.copy_(_i([0, n]))
        ks.copy_(_i([0, n]))
        graph.replay()
        torch.cuda.synchronize()
        _check(out, q, k, v, pe, [0, n], [0, n], 0.1)


# ------------------------------------------------------------------------------- together

def test_prompt_then_decode_steps_over_one_pool():
    """A serving run: plan, append and expand a ragged batch of prompts, attend, then decode steps
    of plan, append and absorbed attention.  Both forms answer the same model: each step's output
    is checked against the expanded definition in 64 bits, the absorbed one through its folded
    query and value maps."""
    gen = torch.Generator().manual_seed(11)
    H, r, dr, ps, B, steps = 8, 96, 32, 64, 4, 70
    prompts = [61, 1, 200, 128]
    scale = 1.2 / (128 + dr) ** 0.5
    W_K, W_V = (bf(H, 128, r, gen=gen, scale=r ** -0.5).to(DEV) for _ in range(2))
    num = 24
    pool = torch.full((num, ps, r + dr), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, 6), -1, dtype=torch.int32, device=DEV)
    free, count, lens = _i(list(range(num))), _i([num]), _i([0] * B)
    ws = stief.plan_workspace()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qs, ks = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(B + 1, dtype=torch.int32, device=DEV)
    history = [[] for _ in range(B)]

    def step(new):
        n = sum(new)
        slots = torch.empty(n + 3, dtype=torch.int32, device=DEV)  # a padded batch
        stief.stief_plan_pages(_i(new), lens, table, free, count, slots, qs, ks, lens, count, ws, ps, dev_status=status)
        rows = bf(n + 3, r + dr, gen=gen).to(DEV)
        stief.stief_append_shared_paged(rows[:, :r], rows[:, r:], slots, pool, dev_status=status)
        at = 0
        for b, t in enumerate(new):
            history[b].append(rows[at: at + t])
            at += t
        return n

    n = step(prompts)
    k, v = (torch.empty((n, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pe = torch.empty((n, dr), dtype=torch.bfloat16, device=DEV)
    stief.stief_expand_shared_paged(pool, table, ks, W_K, W_V, k, v, pe, dev_status=status)
    q = bf(n, H, 128 + dr, gen=gen).to(DEV)
    out = torch.empty((n, H, 128), dtype=torch.bfloat16, device=DEV)
    stief.stief_prefill_attention(q, k, v, qs, ks, out, max(prompts), scale, k_pe=pe, dev_status=status)
    starts = _starts(prompts)
    assert qs.tolist() == starts and ks.tolist() == starts
    rows = torch.cat([h[0] for h in history])
    assert torch.equal(pe, rows[:, r:])
    _check(out, q, k, v, pe, starts, starts, scale)

    dws = stief.shared_workspace_for(B, H, r)
    for s in range(steps):
        new = [1, 1, 0 if s % 3 else 1, 1]  # a request that rests on some steps
        step(new)
        qf = bf(B, H, 128 + dr, gen=gen).to(DEV)
        folded = torch.einsum("bhd,hdr->bhr", qf[..., :128].double(), W_K.double())
        ql = torch.cat([folded.to(torch.bfloat16), qf[..., 128:]], 2).contiguous()
        ol = torch.empty((B, H, r), dtype=torch.bfloat16, device=DEV)
        stief.stief_decode_shared_paged(ql, pool, table, lens, ol, dws, 6 * ps, scale, dev_status=status)
        for b in range(B):
            rows = torch.cat(history[b]).double()
            assert rows.shape[0] == int(lens[b])
            want, bound = attention(ql[b].double()[:, None], rows[None], rows[None, :, :r], scale)
            check(ol[b], want[:, 0], bound[:, 0])
            # the expanded form of the same step, through the folded query as the kernel got it:
            # keys c W_K^T are what the folded query stands for, values c W_V^T what o~ maps to
            full = torch.einsum("hr,hdr->hd", want[:, 0], W_V.double())
            got = torch.einsum("hr,hdr->hd", ol[b].double(), W_V.double())
            room = torch.einsum("hr,hdr->hd", bound[:, 0], W_V.double().abs())
            assert ((got - full).abs() <= room + 1e-12).all()
    assert int(status.item()) == 0
    assert int(count.item()) == num - sum(-(-int(x) // ps) for x in lens.tolist())


def test_plan_drives_the_paged_fused_step():
    """The plan maps pages for this library's per-head paged caches: plan, then the fused step (which
    advances the lengths itself and must not look a page up before the plan has written it)."""
    B, Hq, Hkv, rK, rV, ps, max_pages, steps = 3, 8, 2, 64, 48, 64, 4, 150
    P_K, P_V = si.bases_bf16(7, Hkv, 128, rK, rV)
    num = B * max_pages
    kp = torch.zeros((num, Hkv, ps, rK), dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros((num, Hkv, ps, rV), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(num, generator=torch.Generator().manual_seed(4)).to(torch.int32).to(DEV)
    count, lens, one = _i([num]), _i([0] * B), _i([1] * B)
    ws, pws = stief.workspace_for(B, Hq, Hkv, rV, max_pages * ps), stief.plan_workspace()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gk, gv = P_K.to(DEV), P_V.to(DEV)
    out = torch.empty((B, Hq, 128), dtype=torch.bfloat16, device=DEV)
    k_new, v_new = si.full_kv(70, B, Hkv, steps, 128)
    ko, vo = np.zeros((B, Hkv, max_pages * ps, rK)), np.zeros((B, Hkv, max_pages * ps, rV))
    olens = np.zeros(B, np.int32)
    kd, vd = k_new.to(DEV), v_new.to(DEV)
    for s in range(steps):
        q = si.queries(s, B, Hq, 128)
        kn, vn = kd[:, :, s].contiguous(), vd[:, :, s].contiguous()
        qd = q.to(DEV)
        stief.stief_plan_pages(one, lens, table, free, count, None, None, None, None, count, pws, ps, dev_status=status)
        stief.stief_append_decode_paged(qd, kn, vn, gk, gv, kp, vp, table, lens, out, ws, max_pages * ps,
                                        dev_status=status)
        ko, vo, olens, _ = oracle.compress_append(f64(k_new[:, :, s: s + 1]), f64(v_new[:, :, s: s + 1]), f64(P_K),
                                                  f64(P_V), ko, vo, olens)
        if s % 25 == 0 or s in (63, 64, 65, 128):
            assert_decode_close(out.cpu(), oracle.decode(f64(q), f64(P_K), f64(P_V), ko, vo, olens))
    assert int(status.item()) == 0 and lens.tolist() == [steps] * B
    new, have = [1] * B, [0] * B
    want, left = np.full((B, max_pages), -1, np.int32), num
    for _ in range(steps):
        want, _, _, _, have, left, _ = plan_reference(new, have, want, free.tolist(), left, ps)
    assert np.array_equal(table.cpu().numpy(), want)


def test_both_ways_into_the_library():
    """The binding's two ways (the extension, and Python: other streams, prepare) make the same
    call, and refuse the same arguments for the same reasons."""
    q, k, v, pe = _inputs([130], [130], 4, 2, 16, 21)
    qs, out = _i([0, 130]), [torch.zeros((130, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    stief.stief_prefill_attention(q, k, v, qs, qs, out[0], 130, 0.1, k_pe=pe)
    stief.stief_prefill_attention(q, k, v, qs, qs, out[1], 130, 0.1, k_pe=pe, stream=torch.cuda.current_stream())
    call = stief.prepare(stief.stief_prefill_attention, q, k, v, qs, qs, out[2], 130, 0.1, k_pe=pe)
    assert int(out[2].count_nonzero()) == 0  # prepared, not called
    call()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    for stream in (None, torch.cuda.current_stream()):
        for bad, error in ((dict(q=q.float()), TypeError), (dict(k=k.transpose(0, 1)), ValueError),
                           (dict(v=v[:, :1].contiguous()), ValueError), (dict(qs=qs.cpu()), ValueError),
                           (dict(qs=qs[:1]), ValueError), (dict(out=out[0][:5]), ValueError), (dict(out=None), TypeError),
                           (dict(scale=float("nan")), stief.StiefError), (dict(most=-1), stief.StiefError)):
            a = dict(q=q, k=k, v=v, qs=qs, out=out[0], most=130, scale=0.1)
            a.update(bad)
            with pytest.raises(error):
                stief.stief_prefill_attention(a["q"], a["k"], a["v"], a["qs"], qs, a["out"], a["most"], a["scale"],
                                              k_pe=pe, stream=stream)
        pool, table = torch.zeros((3, 64, 48), dtype=torch.bfloat16, device=DEV), _i([[0, 1]])
        ql, ol, ln = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((1, 4, 48), (1, 4, 32), (1,)))
        ws = stief.shared_workspace_for(1, 4, 32)
        for bad, error in ((dict(ln=ln), TypeError), (dict(ws=ws[:8]), stief.StiefError), (dict(most=129), stief.StiefError),
                           (dict(ol=ol[:, :3].contiguous()), ValueError)):
            a = dict(ln=_i([5]), ws=ws, most=100, ol=ol)
            a.update(bad)
            with pytest.raises(error):
                stief.stief_decode_shared_paged(ql, pool, table, a["ln"], a["ol"], a["ws"], a["most"], 0.1, stream=stream)
