"""stief_decode_shared_paged and stief_expand_shared_paged against 64-bit forms."""
import pytest
import torch

import decode_attention_stief_b200 as stief
from shared_util import U, attention, bf, check, pool_of, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _decode(q, pool, table, lens, r, scale, max_seq_len=None, expect=0, ws=None, stream=None):
    B, Hq, _ = q.shape
    out = torch.full((B, Hq, r), float("nan"), dtype=torch.bfloat16, device=DEV)
    if ws is None:  # its contents must not matter
        ws = stief.shared_workspace_for(B, Hq, r)
        ws.fill_(255)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    most = max([n for n in lens if n < 1 << 30] + [0]) if max_seq_len is None else max_seq_len
    stief.stief_decode_shared_paged(q, pool, table, _i(lens), out, ws, most, scale, dev_status=status, stream=stream)
    assert int(status.item()) == expect
    return out


def _want(q, pool, table, lens, r, scale):
    """64-bit outputs and bounds, [B, Hq, r] each (computed on the GPU in fp64)."""
    o, e = [], []
    for b, n in enumerate(lens):
        rows = rows_of(pool.cpu(), table.cpu(), b, n).to(DEV)[None]
        x, y = attention(q[b].double()[:, None], rows, rows[..., :r], scale)
        o.append(x[:, 0])
        e.append(y[:, 0])
    return torch.stack(o), torch.stack(e)


def _case(lens, Hq, r, dr, ps, seed, q_scale=1.0, **kw):
    gen = torch.Generator().manual_seed(seed)
    pool, table = pool_of(lens, ps, r + dr, gen, **kw)
    q = bf(len(lens), Hq, r + dr, gen=gen, scale=q_scale)
    return q.to(DEV), pool.to(DEV), table.to(DEV)


@pytest.mark.parametrize("r,dr", [(512, 64), (512, 0), (16, 0), (96, 0), (64, 16), (128, 64), (192, 48), (320, 32),
                                  (448, 64), (496, 64)])
@pytest.mark.parametrize("Hq", [1, 16, 40])
def test_decode_ranks_and_heads(r, dr, Hq):
    lens = [1, 0, 64, 65, 200, 63, 130]
    q, pool, table = _case(lens, Hq, r, dr, 64, r + dr + Hq)
    scale = 1.5 / (r + dr) ** 0.5
    check(_decode(q, pool, table, lens, r, scale), *_want(q, pool, table, lens, r, scale))


@pytest.mark.parametrize("Hq", [7, 32, 63, 64, 65, 100, 128, 200, 256])
def test_decode_head_counts(Hq):
    lens = [300, 5, 777]
    q, pool, table = _case(lens, Hq, 256, 64, 128, Hq)
    check(_decode(q, pool, table, lens, 256, 0.09), *_want(q, pool, table, lens, 256, 0.09))


@pytest.mark.parametrize("lens,ps", [([20000], 64), ([4097, 1, 9000], 256), ([64 * 148 + 1], 192), ([1] * 400, 64),
                                     ([777] * 150, 128), ([0, 0, 0], 64), ([100000], 1024)])
def test_decode_splits_and_batches(lens, ps):
    q, pool, table = _case(lens, 16, 128, 32, ps, sum(lens) % 1000 + 1)
    got = _decode(q, pool, table, lens, 128, 0.11, max_seq_len=max(lens) + 40 if ps > 64 else None)
    check(got, *_want(q, pool, table, lens, 128, 0.11))


@pytest.mark.parametrize("Hq", [128, 24])
def test_decode_ragged_batch_full_rank(Hq):
    lens = [(i * 397) % 2100 for i in range(40)]
    q, pool, table = _case(lens, Hq, 512, 64, 64, Hq)
    check(_decode(q, pool, table, lens, 512, 0.06), *_want(q, pool, table, lens, 512, 0.06))


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
def test_decode_peaked_and_flat_scores(scale):
    """Scores in the hundreds, whose running maximum keeps rising; a negative scale; all alike."""
    lens = [1500, 3, 640]
    q, pool, table = _case(lens, 32, 256, 64, 64, 5)
    ramp = torch.linspace(0.2, 4.0, pool.shape[0] * 64, device=DEV).view(-1, 64, 1)
    pool = (pool.float() * ramp).to(torch.bfloat16)
    check(_decode(q, pool, table, lens, 256, scale), *_want(q, pool, table, lens, 256, scale))


def test_decode_rising_maximum_rescales():
    """Each 64-token page scores above the page before it by far more than any threshold."""
    r, n = 64, 64 * 12
    pool = bf(12, 64, r, gen=torch.Generator().manual_seed(2))
    q = torch.zeros(1, 20, r)
    q[:, :, 0] = 1.0
    for j in range(12):
        pool[j, :, 0] = 40.0 * j + torch.arange(64) * 0.25
    table = _i([list(range(12))])
    q, pool = q.to(torch.bfloat16).to(DEV), pool.to(DEV)
    check(_decode(q, pool, table, [n], r, 0.7), *_want(q, pool, table, [n], r, 0.7))


def test_decode_bad_lengths_and_unmapped_pages():
    lens = [130, 70, 100]
    q, pool, table = _case(lens, 16, 64, 0, 64, 9)
    want, bound = _want(q, pool, table, lens, 64, 0.2)
    for bad in (-1, 131, 2 ** 31 - 1, -2 ** 31):
        got = _decode(q, pool, table, [130, bad, 100], 64, 0.2, max_seq_len=130, expect=stief.DEV_BAD_LENGTH)
        check(got[[0, 2]], want[[0, 2]], bound[[0, 2]])
        assert torch.all(got[1].float() == 0)
    for page in (-1, pool.shape[0], 2 ** 31 - 1, -2 ** 31):  # rows of an unmapped page read as zeros
        table[0, 1] = page
        check(_decode(q, pool, table, lens, 64, 0.2), *_want(q, pool, table, lens, 64, 0.2))


def test_decode_is_the_same_every_time_and_captured():
    lens = [3000, 10, 0, 900]
    q, pool, table = _case(lens, 128, 512, 64, 64, 31)
    first = _decode(q, pool, table, lens, 512, 0.06)
    ws = stief.shared_workspace_for(4, 128, 512)
    ln, out = _i(lens), torch.empty_like(first)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        stief.stief_decode_shared_paged(q, pool, table, ln, out, ws, 3000, 0.06)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    shorter = [2931, 9, 0, 0]  # a captured call takes the lengths as they are at replay
    ln.copy_(_i(shorter))
    graph.replay()
    torch.cuda.synchronize()
    check(out, *_want(q, pool, table, shorter, 512, 0.06))


def test_decode_two_streams():
    a, b = _case([2500], 32, 256, 0, 64, 1), _case([1800, 40], 64, 128, 64, 64, 2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    wa, wb = stief.shared_workspace_for(1, 32, 256), stief.shared_workspace_for(2, 64, 128)
    la, lb = _i([2500]), _i([1800, 40])
    xa = torch.empty((1, 32, 256), dtype=torch.bfloat16, device=DEV)
    xb = torch.empty((2, 64, 128), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        stief.stief_decode_shared_paged(*a, la, xa, wa, 2500, 0.08, stream=s)
        stief.stief_decode_shared_paged(*b, lb, xb, wb, 1800, 0.08, stream=t)
    torch.cuda.synchronize()
    check(xa, *_want(*a, [2500], 256, 0.08))
    check(xb, *_want(*b, [1800, 40], 128, 0.08))


def _expand(pool, table, start, W_K, W_V, N, dr, expect=0):
    H = W_K.shape[0]
    k, v = (torch.full((N, H, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pe = torch.full((N, dr), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stief.stief_expand_shared_paged(pool, table, start, W_K, W_V, k, v, pe if dr else None, dev_status=status)
    assert int(status.item()) == expect
    return k, v, pe


@pytest.mark.parametrize("lens,H,r,dr,ps", [([1], 1, 16, 0, 64), ([64, 0, 65, 1, 127], 3, 96, 16, 64),
                                            ([700, 300], 8, 512, 64, 128), ([0, 129], 5, 192, 0, 192),
                                            ([1000], 16, 320, 32, 64), ([1] * 70, 2, 64, 64, 64)])
def test_expand(lens, H, r, dr, ps):
    gen = torch.Generator().manual_seed(H + r)
    pool, table = pool_of(lens, ps, r + dr, gen)
    W_K, W_V = bf(H, 128, r, gen=gen, scale=r ** -0.5).to(DEV), bf(H, 128, r, gen=gen, scale=r ** -0.5).to(DEV)
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    total, N = start[-1], start[-1] + 5  # rows behind the last sequence stay as they were
    k, v, pe = _expand(pool.to(DEV), table.to(DEV), _i(start), W_K, W_V, N, dr)
    rows = torch.cat([rows_of(pool, table, b, n) for b, n in enumerate(lens)]).to(DEV)
    for got, W in ((k, W_K), (v, W_V)):
        w = W.double().reshape(H * 128, r)
        want = (rows[:, :r] @ w.T).view(total, H, 128)
        size = (rows[:, :r].abs() @ w.abs().T).view(total, H, 128)
        check(got[:total], want, U * want.abs() + (r / 16 + 4) * 2.0 ** -23 * size + 1e-30)
        assert torch.all(got[total:] == 7.0)
    assert torch.equal(pe[:total].double(), rows[:, r:]) and torch.all(pe[total:] == 7.0)


def test_expand_more_rows_than_room_and_unmapped():
    gen = torch.Generator().manual_seed(1)
    pool, table = pool_of([100, 90], 64, 64, gen)
    W = bf(2, 128, 64, gen=gen, scale=0.125).to(DEV)
    full = _expand(pool.to(DEV), table.to(DEV), _i([0, 100, 190]), W, W, 190, 0)
    part = _expand(pool.to(DEV), table.to(DEV), _i([0, 100, 190]), W, W, 150, 0, expect=stief.DEV_BAD_LENGTH)
    assert torch.equal(full[0][:150], part[0])
    table[1, 0] = -3
    k, v, _ = _expand(pool.to(DEV), table.to(DEV), _i([0, 100, 190]), W, W, 190, 0)
    assert torch.all(k[100:164] == 0) and torch.all(v[100:164] == 0) and torch.equal(k[164:], full[0][164:])


@pytest.mark.parametrize("lens,Hq,r,dr", [
    ([9100], 24, 512, 64), ([8300, 0], 5, 256, 0),                                    # very many parts
    ([2000, 3000, 1, 700], 48, 512, 64), ([1500, 0, 900], 128, 96, 32),               # four warps, 128 dims each
    ([64] * 20 + [6000] + [300] * 19, 32, 512, 64), ([500] * 30 + [9000], 16, 192, 16),  # four warps, all dims
    ([10] * 20 + [7000, 0] + [257] * 20, 128, 384, 0)])                               # a warp a head
def test_decode_many_parts(lens, Hq, r, dr):
    q, pool, table = _case(lens, Hq, r, dr, 64, sum(lens) + Hq)
    scale = 1.5 / (r + dr) ** 0.5
    got = _decode(q, pool, table, lens, r, scale)
    check(got, *_want(q, pool, table, lens, r, scale))
    assert torch.equal(got, _decode(q, pool, table, lens, r, scale))
