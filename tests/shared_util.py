"""64-bit forms of the page planning and shared-latent operators, straight from their formulas,
and the error bounds their kernels are held to.

Roundings counted (u = 2^-8, half a bf16 step relative to the value): the weights of a softmax
are rounded to bf16 before the second product, numerator and denominator at most alike, so a
weighted sum moves by at most u * sum_t p_t (|v_t| + |o|); the output is rounded once, u * |o|.
Sums of n products on the tensor cores are n / 16 additions in fp32 whose adder may truncate, and
four for the products of one group: (n / 16 + 4) * 2^-23 of the sum of absolute products.  An
error e of a score (with exp's own 2^-21) moves every weight by at most the factor 1 + 2 e.
"""
import numpy as np
import torch

U = 2.0 ** -8
DEV = "cuda"


def bf(*shape, gen=None, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * scale).to(torch.bfloat16)


def pool_of(lens, page_size, w, gen, spare=3, extra_pages=1, fill=float("nan")):
    """A pool (random rows below each length, `fill` everywhere else) and a block table whose
    unused entries are ids outside the pool."""
    pages = [-(-n // page_size) for n in lens]
    num = sum(pages) + spare
    ids = torch.randperm(num, generator=gen)
    table = torch.full((len(lens), max(1, max(pages)) + extra_pages), -7, dtype=torch.int32)
    table[:, -1] = num + 5
    pool = torch.full((num, page_size, w), fill, dtype=torch.bfloat16)
    at = 0
    for b, n in enumerate(lens):
        for j in range(pages[b]):
            pg = int(ids[at])
            at += 1
            table[b, j] = pg
            k = min(page_size, n - j * page_size)
            pool[pg, :k] = bf(k, w, gen=gen)
    return pool, table


def rows_of(pool, table, b, n):
    """Rows [0, n) of sequence b in 64 bits (pages outside the pool read as zeros)."""
    ps, got = pool.shape[1], []
    for j in range(-(-n // ps)):
        pg = int(table[b, j])
        got.append(pool[pg].double() if 0 <= pg < pool.shape[0] else torch.zeros_like(pool[0], dtype=torch.float64))
    return torch.cat(got)[:n] if got else torch.zeros((0, pool.shape[2]), dtype=torch.float64)


def attention(q, k, v, scale, hidden=None):
    """softmax(scale q k^T) v for q [H, n, w], k [H|1, m, w], v [H|1, m, d] in 64 bits, zeros for a
    query that sees nothing, and the bound of the kernels' error for each output value."""
    x = (q @ k.transpose(-1, -2)) * scale
    size = (q.abs() @ k.abs().transpose(-1, -2)) * abs(scale)
    if hidden is not None:
        x = x.masked_fill(hidden, -np.inf)
        size = size.masked_fill(hidden, 0.0)
    if x.shape[-1] == 0:
        o = torch.zeros((*q.shape[:2], v.shape[-1]), dtype=torch.float64, device=q.device)
        return o, torch.zeros_like(o)
    p = torch.softmax(x, -1).nan_to_num(0.0)
    o, mag = p @ v, p @ v.abs()
    e = (q.shape[-1] / 16 + 4) * 2.0 ** -23 * size.amax(-1, keepdim=True) + 2.0 ** -21
    # the sum over m weighted rows in fp32, rescaled once a tile of 64 at most
    e = 2 * e + (k.shape[-2] / 16 + 8) * 2.0 ** -23
    return o, (U + e) * (mag + o.abs()) + U * o.abs() + 1e-30


def check(got, want, bound):
    got = got.double().to(want.device)
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), "non-finite output"
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"off by more than the bound: {worst:.3e} over, at {int(over.argmax())}"


def plan_reference(new, lens, table, free, count, page_size, max_tokens=None):
    """The plan's definition, one sequence at a time: table, slots, q_start, kv_start, lens, left,
    status bits."""
    num, cap = len(free), table.shape[1] * page_size
    table, lens, bits = table.copy(), [int(n) for n in lens], 0
    if not 0 <= count <= num:
        bits, count = 4, min(max(count, 0), num)
    slots = [-1] * (max_tokens or 0)
    q_start, kv_start, asked, used, out = [0], [0], 0, 0, []
    for b, (have, take) in enumerate(zip(lens, (int(t) for t in new))):
        bad = have < 0 or have > cap or take < 0
        end = q_start[-1] + max(take, 0)
        ok = not bad
        if bad:
            bits |= 4
        else:
            first = -(-have // page_size)
            last = -(-(have + take) // page_size)
            ok = have + take <= cap and (max_tokens is None or end <= max_tokens)
            if ok and take and have % page_size:
                ok = 0 <= table[b, first - 1] < num
            if ok and last > first:
                asked += last - first
                ok = asked <= count
                if ok:
                    for j in range(first, last):
                        table[b, j] = free[count - 1 - used]
                        used += 1
            if not ok:
                bits |= 1
        if ok and max_tokens is not None:
            for i in range(take):
                pg = int(table[b, (have + i) // page_size])
                if 0 <= pg < num:
                    slots[q_start[-1] + i] = pg * page_size + (have + i) % page_size
        out.append(have + take if ok else have)
        q_start.append(end)
        kv_start.append(kv_start[-1] + (0 if have < 0 or have > cap else out[-1]))
    return table, slots, q_start, kv_start, out, count - used, bits
