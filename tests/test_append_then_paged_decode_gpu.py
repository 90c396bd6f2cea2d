"""Rows that stief_append_shared_paged has just written, read by the next call of the stream: a paged
decode over per-head pools of one KV head, which lie in memory as shared pools do, requests cache
rows before its dependency wait unless it knows that the kernel before it wrote some."""
import pytest
import torch

import decode_attention_stief_b200 as stief
import stief_inputs as si
from shared_util import bf

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("n", [200, 4000, 60000])
def test_decode_sees_rows_appended_right_before_it(n):
    r, ps, Hq = 64, 64, 4
    num = -(-n // ps) + 2
    gen = torch.Generator().manual_seed(n)
    P_K, P_V = (x.to(DEV) for x in si.bases_bf16(3, 1, 128, r, r))
    kp, vp = (torch.zeros((num, ps, r), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rows_k, rows_v = (bf(n, r, gen=gen).to(DEV) for _ in range(2))
    pages = torch.randperm(num, generator=gen).to(torch.int32)
    at = torch.arange(n)
    slots = (pages[at // ps] * ps + at % ps).to(torch.int32).to(DEV)
    table, lens = pages[None].contiguous().to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    q = si.queries(5, 1, Hq, 128).to(DEV)
    ws = stief.workspace_for(1, Hq, 1, r, n)
    out = torch.empty((1, Hq, 128), dtype=torch.bfloat16, device=DEV)

    def step(wait):
        kp.zero_()
        vp.zero_()
        stief.stief_append_shared_paged(rows_k, None, slots, kp)
        stief.stief_append_shared_paged(rows_v, None, slots, vp)
        if wait:
            torch.cuda.synchronize()
        stief.stief_decode_attention_paged(q, P_K, P_V, kp.view(num, 1, ps, r), vp.view(num, 1, ps, r), table, lens, out,
                                           ws, n)
        return out.clone()

    want = step(True)
    assert all(torch.equal(step(False), want) for _ in range(50))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):  # (back to back, however slow the host)
        got = step(False)
    for _ in range(50):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
