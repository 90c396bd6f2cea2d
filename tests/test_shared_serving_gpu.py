"""The shared-latent calls as a server makes them: a captured step replayed, several streams at
once, very large pools and batches, pages that sequences share."""
import pytest
import torch

import decode_attention_stief_b200 as stief
import stief_inputs as si
from shared_util import U, attention, bf, check, pool_of, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _empty(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV)


def test_captured_decode_step_replayed():
    """Plan, append and decode captured as one step; the graph advances the lengths and takes pages
    by itself, replay after replay."""
    gen = torch.Generator().manual_seed(5)
    B, H, r, dr, ps, steps, num = 6, 40, 128, 64, 64, 140, 40
    pool, table = torch.full((num, ps, r + dr), float("nan"), dtype=torch.bfloat16, device=DEV), _i([[-1] * 4] * B)
    free, count, lens, new = _i(list(range(num))), _i([num]), _i([0] * B), _i([1, 1, 1, 0, 1, 1])
    q, rows, out = _empty(B, H, r + dr), _empty(5, r + dr), _empty(B, H, r)
    slots, status = torch.empty(8, dtype=torch.int32, device=DEV), _i([0])
    pws, ws = stief.plan_workspace(), stief.shared_workspace_for(B, H, r)
    c, pe = rows[:, :r], rows[:, r:]
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        stief.stief_plan_pages(new, lens, table, free, count, slots, None, None, lens, count, pws, ps, dev_status=status)
        stief.stief_append_shared_paged(c, pe, slots[:5], pool, dev_status=status)
        stief.stief_decode_shared_paged(q, pool, table, lens, out, ws, 4 * ps, 0.07, dev_status=status)
    history = [[] for _ in range(B)]
    for s in range(steps):
        x, y = bf(5, r + dr, gen=gen).to(DEV), bf(B, H, r + dr, gen=gen).to(DEV)
        rows.copy_(x)
        q.copy_(y)
        graph.replay()
        for n, b in enumerate((0, 1, 2, 4, 5)):
            history[b].append(x[n])
        if s in (0, 1, 62, 63, 64, 65, 127, 128, steps - 1):
            for b in (0, 5):
                k = torch.stack(history[b]).double()[None]
                want, bound = attention(y[b].double()[:, None], k, k[..., :r], 0.07)
                check(out[b], want[:, 0], bound[:, 0])
            assert torch.all(out[3].float() == 0)
    assert lens.tolist() == [steps] * 3 + [0] + [steps] * 2 and int(status.item()) == 0
    assert int(count.item()) == num - 5 * -(-steps // ps)


def test_many_streams_at_once():
    """All the kernels that hold tensor memory, and the older ones that do, running side by side on
    streams of their own: each gives what it gives alone."""
    gen = torch.Generator().manual_seed(8)
    pool, table = pool_of([3000, 400, 90], 64, 576, gen)
    pool, table, lens = pool.to(DEV), table.to(DEV), _i([3000, 400, 90])
    small, stable = pool_of([700, 64], 64, 96, gen)
    small, stable = small.to(DEV), stable.to(DEV)
    W = bf(8, 128, 512, gen=gen, scale=0.05).to(DEV)
    Ws = bf(8, 128, 96, gen=gen, scale=0.1).to(DEV)
    q0, q64, k, v, pe = (bf(*s, gen=gen).to(DEV) for s in ((900, 8, 128), (900, 8, 192), (1000, 2, 128), (1000, 2, 128),
                                                          (1000, 64)))
    qd, qs, qsd = bf(3, 128, 576, gen=gen).to(DEV), _i([0, 900]), bf(2, 16, 96, gen=gen).to(DEV)
    ks, st3, st2, slens = _i([0, 1000]), _i([0, 3000, 3400, 3490]), _i([0, 700, 764]), _i([700, 64])
    P_K, P_V = (x.to(DEV) for x in si.bases_bf16(1, 8, 128, 64, 64))
    kn, vn = (x.to(DEV) for x in si.full_kv(2, 1, 8, 2000, 128))

    def work(n):
        ws, wss = stief.shared_workspace_for(3, 128, 512), stief.shared_workspace_for(2, 16, 96)
        outs = [_empty(3, 128, 512), _empty(900, 8, 128), _empty(900, 8, 128), _empty(3490, 8, 128), _empty(3490, 8, 128),
                _empty(3490, 64), _empty(764, 8, 128), _empty(764, 8, 128), torch.zeros((1, 8, 2048, 64), dtype=torch.bfloat16, device=DEV),
                torch.zeros((1, 8, 2048, 64), dtype=torch.bfloat16, device=DEV), _empty(2, 16, 96)]
        l0 = _i([0])
        calls = [lambda: stief.stief_decode_shared_paged(qd, pool, table, lens, outs[0], ws, 3000, 0.06),
                 lambda: stief.stief_prefill_attention(q0, k, v, qs, ks, outs[1], 900, 0.1),
                 lambda: stief.stief_prefill_attention(q64, k, v, qs, ks, outs[2], 900, 0.1, k_pe=pe),
                 lambda: stief.stief_expand_shared_paged(pool, table, st3, W, W, outs[3], outs[4], outs[5]),
                 lambda: stief.stief_expand_shared_paged(small, stable, st2, Ws, Ws, outs[6], outs[7]),
                 lambda: (l0.zero_(), stief.stief_compress_append(kn, vn, P_K, P_V, outs[8], outs[9], l0)),
                 lambda: stief.stief_decode_shared_paged(qsd, small, stable, slens, outs[10], wss, 700, 0.1)]
        return [calls[(i + n) % len(calls)] for i in range(len(calls))], outs

    sets = [work(n) for n in range(4)]
    for f in sets[0][0]:
        f()
    torch.cuda.synchronize()
    want = [x.clone() for x in sets[0][1]]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(25):
        for s, (calls, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                for f in calls:
                    f()
    torch.cuda.synchronize()
    for _, outs in sets:
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_offsets_past_32_bits():
    """A pool of more than 4 GB whose used pages lie at its end, and keys and values of more than 4
    GB whose sequence does."""
    gen = torch.Generator().manual_seed(9)
    r, dr, ps, lens = 512, 64, 1024, [1500, 700]
    num = (4 << 30) // (ps * 576 * 2) + 8
    pool = _empty(num, ps, 576)
    table = _i([[num - 1, num - 4], [num - 2, -1]])
    slots = torch.cat([torch.arange(n) % ps + ps * table.cpu()[b, torch.arange(n) // ps] for b, n in enumerate(lens)])
    rows = bf(2200, 576, gen=gen).to(DEV)
    stief.stief_append_shared_paged(rows[:, :r], rows[:, r:], slots.to(torch.int32).to(DEV), pool)
    q, out = bf(2, 32, 576, gen=gen).to(DEV), _empty(2, 32, r)
    stief.stief_decode_shared_paged(q, pool, table, _i(lens), out, stief.shared_workspace_for(2, 32, r), 1500, 0.06)
    at = 0
    for b, n in enumerate(lens):
        k = rows[at: at + n].double()[None]
        want, bound = attention(q[b].double()[:, None], k, k[..., :r], 0.06)
        check(out[b], want[:, 0], bound[:, 0])
        at += n
    W, k, v, pe = bf(1, 128, r, gen=gen, scale=0.05).to(DEV), _empty(2200, 1, 128), _empty(2200, 1, 128), _empty(2200, 64)
    stief.stief_expand_shared_paged(pool, table, _i([0, 1500, 2200]), W, W, k, v, pe)
    want, size = rows[:, :r].double() @ W[0].double().T, rows[:, :r].double().abs() @ W[0].double().abs().T
    check(k[:, 0], want, U * want.abs() + (r / 16 + 4) * 2.0 ** -23 * size)
    assert torch.equal(k, v) and torch.equal(pe, rows[:, r:])
    del pool
    torch.cuda.empty_cache()
    n, H = (4 << 30) // (32 * 256) + 300, 32
    k, v = _empty(n, H, 128), _empty(n, H, 128)
    k[-300:], v[-300:] = bf(300, H, 128, gen=gen).to(DEV), bf(300, H, 128, gen=gen).to(DEV)
    q, out = _empty(n, H, 128), _empty(n, H, 128)
    q[-200:] = bf(200, H, 128, gen=gen).to(DEV)
    out[-201] = 7.0
    stief.stief_prefill_attention(q, k, v, _i([n - 200, n]), _i([n - 300, n]), out, 200, 0.1)
    hidden = torch.arange(300, device=DEV)[None, :] > torch.arange(200, device=DEV)[:, None] + 100
    want, bound = attention(q[-200:].double().transpose(0, 1), k[-300:].double().transpose(0, 1),
                            v[-300:].double().transpose(0, 1), 0.1, hidden)
    check(out[-200:].transpose(0, 1), want, bound)
    assert torch.all(out[-201] == 7.0)


def test_largest_batch():
    """65535 sequences of 0 to 2 tokens: decode and expand."""
    B, r = 65535, 16
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 3, (B,), generator=gen).to(torch.int32)
    pool = _empty(B, 64, r)
    two = bf(B, 2, r, gen=gen).to(DEV)
    pool.fill_(float("nan"))
    pool[:, :2] = two
    table, q, out = torch.arange(B, dtype=torch.int32, device=DEV).flip(0)[:, None].contiguous(), bf(B, 1, r, gen=gen).to(DEV), _empty(B, 1, r)
    ws = stief.shared_workspace_for(B, 1, r)
    for most in (2, 64 * 5):  # one kernel, and two
        big = table if most == 2 else torch.cat([table, torch.full((B, 4), -1, dtype=torch.int32, device=DEV)], 1)
        out.fill_(float("nan"))
        stief.stief_decode_shared_paged(q, pool, big, lens.to(DEV), out, ws, most, 0.5)
        rows = two.flip(0).double()
        n = lens.to(DEV)
        x = (q.double() @ rows.transpose(1, 2))[:, 0] * 0.5
        x = x.masked_fill(torch.arange(2, device=DEV)[None, :] >= n[:, None], -torch.inf)
        p = torch.softmax(x, -1).nan_to_num(0.0)
        want, mag = (p[:, None] @ rows)[:, 0], (p[:, None] @ rows.abs())[:, 0]
        check(out[:, 0], want, (U + 1e-5) * (mag + want.abs()) + U * want.abs() + 1e-30)
    start = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).to(torch.int32)])
    N = int(start[-1])
    W, k, v = bf(1, 128, r, gen=gen, scale=0.25).to(DEV), _empty(N, 1, 128), _empty(N, 1, 128)
    stief.stief_expand_shared_paged(pool, table, start.to(DEV), W, W, k, v)
    have = torch.arange(2, device=DEV)[None, :] < lens.to(DEV)[:, None]
    rows = two.flip(0)[have].double()
    want, size = rows @ W[0].double().T, rows.abs() @ W[0].double().abs().T
    check(k[:, 0], want, U * want.abs() + 5 * 2.0 ** -23 * size + 1e-30)
    assert torch.equal(k, v)


def test_shared_pages_and_one_query_prompts():
    """Sequences that share a prefix's pages; one new query behind a long past (a decode step in the
    expanded form)."""
    gen = torch.Generator().manual_seed(4)
    pool, table = pool_of([640, 100], 64, 128, gen, extra_pages=2)
    shared = table.clone()
    shared[1, :9] = table[0, :9]
    shared[1, 9:11] = table[1, :2]
    q, out, lens = bf(2, 24, 128, gen=gen).to(DEV), _empty(2, 24, 64), [640, 9 * 64 + 100]
    stief.stief_decode_shared_paged(q, pool.to(DEV), shared.to(DEV), _i(lens), out, stief.shared_workspace_for(2, 24, 64), 700, 0.1)
    for b, n in enumerate(lens):
        k = rows_of(pool, shared, b, n).to(DEV)[None]
        want, bound = attention(q[b].double()[:, None], k, k[..., :64], 0.1)
        check(out[b], want[:, 0], bound[:, 0])
    for dr in (0, 64):
        q, k, v, pe = (bf(*s, gen=gen).to(DEV) for s in ((3, 8, 128 + dr), (5200, 2, 128), (5200, 2, 128), (5200, dr)))
        out, ks = _empty(3, 8, 128), [0, 5000, 5001, 5200]
        stief.stief_prefill_attention(q, k, v, _i([0, 1, 2, 3]), _i(ks), out, 1, 0.1, k_pe=pe if dr else None)
        for b in range(3):
            kk = torch.cat([k[ks[b]: ks[b + 1]], pe[ks[b]: ks[b + 1], None].expand(-1, 2, -1)], 2).double()
            kk, vv = (x.repeat_interleave(4, 1).transpose(0, 1) for x in (kk, v[ks[b]: ks[b + 1]].double()))
            want, bound = attention(q[b: b + 1].double().transpose(0, 1), kk, vv, 0.1)
            check(out[b][:, None], want, bound)


def test_paired_prompts_beside_single_tiles():
    """Prompts whose CTAs work in pairs, prompts whose CTAs do not, and some whose CTAs share a tile's
    keys, on streams of their own: an SM of a pair may hold another kernel's CTA where its neighbour
    holds none."""
    gen = torch.Generator().manual_seed(12)
    # (queries, keys, heads, KV heads, position values); the last two work in pairs
    shapes = [(1500, 1500, 4, 4, 64), (300, 100, 3, 1, 0), (1100, 2100, 5, 5, 16), (700, 900, 7, 7, 0),
              (129, 5000, 37, 1, 64), (90, 90, 29, 29, 16), (700, 1300, 40, 40, 64), (200, 2100, 150, 75, 16)]
    runs = []
    for nq, nk, Hq, Hkv, dr in shapes:
        t = [bf(*s, gen=gen).to(DEV) for s in ((nq, Hq, 128 + dr), (nk, Hkv, 128), (nk, Hkv, 128), (nk, dr))]
        runs.append((t, _i([0, nq]), _i([0, nk]), nq, _empty(nq, Hq, 128), _i([0])))

    def call(t, qs, ks, nq, out, status):
        stief.stief_prefill_attention(t[0], t[1], t[2], qs, ks, out, nq, 0.08, k_pe=t[3] if t[3].shape[1] else None,
                                      dev_status=status)

    for run in runs:
        call(*run)
    torch.cuda.synchronize()
    want = [run[4].clone() for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    for n in range(40):
        for i, (s, run) in enumerate(zip(streams, runs)):
            with torch.cuda.stream(s):
                for _ in range(1 + (n + i) % 3):
                    call(*run)
    torch.cuda.synchronize()
    for run, x in zip(runs, want):
        assert int(run[5].item()) == 0 and torch.equal(run[4], x)
