"""Cases of the page planning and shared-latent attention operators, with their plain forms.

Five operators of a serving step over page pools:

- "plan":    block tables, slot maps and row offsets from the requests' lengths;
- "append":  new latent rows written into the pool through the slot map;
- "decode":  absorbed attention of one query token a sequence over the shared latents;
- "expand":  keys and values of every head computed from the shared latents (the expanded form);
- "prefill": causal attention of ragged prompts over expanded (or any per-head) keys and values.

A cache row is ``r`` latent values, from which the keys and the values of every head come, and
``dr`` position values that every head's keys share.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
D = 128  # head dimension of queries, expanded keys and values


def _spread(n, lo, hi, k=0):
    """n lengths between lo and hi (both met when n > 1), spread evenly and out of order."""
    if n == 1:
        return [hi]
    got = [lo + (hi - lo) * ((i * 7919 + 13 * k) % n) // (n - 1) for i in range(n)]
    got[got.index(max(got))] = hi
    return got


def listed():
    return [
        # one decode step of a serving batch: every request takes one token (latency)
        dict(name="plan step", op="plan", B=64, lo=1, hi=8192, tlo=1, thi=1, ps=64, table=256),
        # admission of many ragged prompts at once, with idle requests (0 tokens) among them
        dict(name="plan prompts", op="plan", B=512, lo=0, hi=4096, tlo=0, thi=2048, ps=128, table=64),
        # the rows of one decode step
        dict(name="append step", op="append", n=64, r=512, dr=64, ps=64),
        # the rows of a large prefill batch, some padding rows (slot -1) at the end
        dict(name="append prompts", op="append", n=32768, r=512, dr=64, ps=128),
        # a few short conversations, small model: latency
        dict(name="decode short", op="decode", B=5, lo=0, hi=200, Hq=16, r=128, dr=0, ps=64),
        # one sequence at 32k tokens, 32 query heads
        dict(name="decode 32k", op="decode", B=1, lo=32768, hi=32768, Hq=32, r=512, dr=64, ps=64),
        # a ragged batch of 64 at up to 4096 tokens, many heads: bytes and products both count
        dict(name="decode batch", op="decode", B=64, lo=511, hi=4096, Hq=128, r=512, dr=64, ps=128),
        # keys and values of a 4096-token prompt
        dict(name="expand 4k", op="expand", B=1, lo=4096, hi=4096, Hq=32, r=512, dr=64, ps=64),
        # three short ragged prompts, a small rank
        dict(name="expand ragged", op="expand", B=3, lo=33, hi=501, Hq=8, r=96, dr=0, ps=64),
        # one short prompt
        dict(name="prefill short", op="prefill", B=1, lo=77, hi=77, past=0, Hq=8, Hkv=8, dr=0),
        # ragged chunks that attend to up to 1000 cached tokens besides, grouped heads
        dict(name="prefill chunks", op="prefill", B=8, lo=65, hi=1500, past=1000, Hq=32, Hkv=8, dr=0),
        # one 8192-token prompt in the expanded form, with the shared position values
        dict(name="prefill 8k", op="prefill", B=1, lo=8192, hi=8192, past=0, Hq=32, Hkv=32, dr=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "expand", "prefill"])
    ps = rng.choice([64, 128, 256])
    r, dr = rng.choice([64, 96, 128, 192, 256, 384, 512]), rng.choice([0, 32, 64])
    if op == "plan":
        B = _log(rng, 1, 2048)
        hi, thi = _log(rng, 1, 8192), _log(rng, 1, max(2, 1000000 // B) if B > 128 else 4096)
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, tlo=rng.randint(0, thi), thi=thi, ps=ps,
                    table=(hi + thi) // ps + 1 + rng.randint(0, 40))
    if op == "append":
        return dict(op=op, n=_log(rng, 1, 32768), r=r, dr=dr, ps=ps)
    if op == "decode":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, min(131072, 262144 // B))
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hq=rng.choice([1, 8, 12, 16, 32, 40, 64, 128]),
                    r=r, dr=dr, ps=ps)
    if op == "expand":
        B = _log(rng, 1, 16)
        hi = _log(rng, 1, 8192 // B)
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hq=rng.choice([1, 4, 8, 16, 32]), r=r, dr=dr, ps=ps)
    B = _log(rng, 1, 16)
    hi = _log(rng, 1, 6000 // B)
    Hkv, g = rng.choice([(1, 4), (2, 8), (4, 1), (8, 4), (16, 1), (32, 1)])
    return dict(op="prefill", B=B, lo=rng.randint(0, hi), hi=hi, past=rng.choice([0, 0, _log(rng, 1, 2000)]),
                Hq=Hkv * g, Hkv=Hkv, dr=dr)


# ------------------------------------------------------------------------------------ inputs

def _starts(lens):
    got = [0]
    for n in lens:
        got.append(got[-1] + n)
    return got


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(case, lens, gen):
    """A pool whose pages the sequences hold in random order, and its block table."""
    ps, w = case["ps"], case["r"] + case["dr"]
    pages = [-(-n // ps) for n in lens]
    num = sum(pages) + 7
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32, device=DEV)
    ids = torch.randperm(num, generator=gen, device=DEV).to(torch.int32)
    held = torch.arange(table.shape[1], device=DEV)[None, :] < _int(pages)[:, None]
    table[held] = ids[: sum(pages)]
    pool = torch.randn((num, ps, w), generator=gen, device=DEV, dtype=torch.float32).to(BF)
    return pool, table


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(BF)

    s = dict(case)
    if op == "plan":
        B, ps = case["B"], case["ps"]
        lens, new = _spread(B, case["lo"], case["hi"]), _spread(B, case["tlo"], case["thi"], 5)
        held = [-(-n // ps) for n in lens]
        need = sum(-(-(n + t) // ps) for n, t in zip(lens, new))
        num = need + 5
        ids = torch.randperm(num, generator=gen, device=DEV).to(torch.int32)
        table = torch.full((B, case["table"]), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(case["table"], device=DEV)[None, :] < _int(held)[:, None]] = ids[: sum(held)]
        free = torch.zeros(num, dtype=torch.int32, device=DEV)  # a stack; the held pages are not on it
        free[: num - sum(held)] = ids[sum(held):]
        total = sum(new)
        s.update(new_tokens=_int(new), lens=_int(lens), table=table, free=free, count=_int([num - sum(held)]),
                 max_tokens=total + (total + 7) // 8)
    elif op == "append":
        n, ps = case["n"], case["ps"]
        num = -(-n // ps) + 4
        slots = torch.randperm(num * ps, generator=gen, device=DEV)[:n].to(torch.int32)
        slots[n - n // 16:] = -1
        s.update(c=normal(n, case["r"]), pe=normal(n, case["dr"]), slots=slots,
                 pool=torch.zeros((num, ps, case["r"] + case["dr"]), dtype=BF, device=DEV))
    elif op == "decode":
        lens = _spread(case["B"], case["lo"], case["hi"])
        pool, table = _pool(case, lens, gen)
        w = case["r"] + case["dr"]
        s.update(pool=pool, table=table, lens=_int(lens), q=normal(case["B"], case["Hq"], w), scale=1.5 / math.sqrt(w))
    elif op == "expand":
        lens = _spread(case["B"], case["lo"], case["hi"])
        pool, table = _pool(case, lens, gen)
        r, H = case["r"], case["Hq"]
        s.update(pool=pool, table=table, start=_int(_starts(lens)), n=sum(lens),
                 W_K=normal(H, D, r, scale=r ** -0.5), W_V=normal(H, D, r, scale=r ** -0.5))
    else:
        lens = _spread(case["B"], case["lo"], case["hi"])
        kv = [n + p for n, p in zip(lens, _spread(case["B"], 0, case["past"], 3))]
        q, k = _starts(lens), _starts(kv)
        s.update(q=normal(q[-1], case["Hq"], D + case["dr"]), k=normal(k[-1], case["Hkv"], D),
                 v=normal(k[-1], case["Hkv"], D), pe=normal(k[-1], case["dr"]), q_start=_int(q), kv_start=_int(k),
                 max_q=max(lens), max_kv=max(kv), scale=1.5 / math.sqrt(D + case["dr"]))
    return s


# ------------------------------------------------------------------------------- plain forms

def _rows(s, b, t):
    """Pool rows (page, row) of tokens t of sequences b."""
    return s["table"].long()[b, t // s["ps"]], t % s["ps"]


def _softmax(x, seen):
    """Weights over the last axis of the positions that are seen; none for a row that sees nothing."""
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    return x / x.sum(-1, keepdim=True).clamp_min(1e-38)


def _plain_plan(s):
    ps, T, L, table = s["ps"], s["new_tokens"].long(), s["lens"].long(), s["table"]
    n = s["max_tokens"]
    q_start = torch.cat([T.new_zeros(1), T.cumsum(0)])
    had = (L + ps - 1) // ps
    need = (L + T + ps - 1) // ps - had
    upto = need.cumsum(0)
    count = s["count"].long()
    ok = (need == 0) | (upto <= count)
    ok &= (L + T <= table.shape[1] * ps) & (q_start[1:] <= n)
    lens = torch.where(ok, L + T, L)
    kv_start = torch.cat([T.new_zeros(1), lens.cumsum(0)])
    at = torch.arange(table.shape[1], device=DEV)[None, :] - had[:, None]
    new = (at >= 0) & (at < need[:, None]) & ok[:, None]
    taken = s["free"].long()[(count - 1 - ((upto - need)[:, None] + at)).clamp(0, s["free"].numel() - 1)]
    table = torch.where(new, taken, table.long())
    i = torch.arange(n, device=DEV)
    b = torch.searchsorted(q_start[1:], i, right=True).clamp_max(T.numel() - 1)
    t = L[b] + i - q_start[b]
    page = table[b, (t // ps).clamp(0, table.shape[1] - 1)]
    slots = torch.where((i < q_start[-1]) & ok[b], page * ps + t % ps, -1)
    left = count - torch.where(ok, upto, 0).amax()
    return [x.to(torch.int32) for x in (table, slots, q_start, kv_start, lens, left)]


def _plain_append(s):
    rows = s["pool"].view(-1, s["pool"].shape[2])
    kept = s["slots"] >= 0
    rows[s["slots"][kept].long()] = torch.cat([s["c"], s["pe"]], 1)[kept]
    return s["pool"]


def _plain_decode(s):
    B, r = s["B"], s["r"]
    t = torch.arange(max(1, s["hi"]), device=DEV)[None, :].expand(B, -1)
    page, row = _rows(s, torch.arange(B, device=DEV)[:, None], t)
    rows = s["pool"][page.clamp_min(0), row].float()
    seen = t < s["lens"][:, None]
    x = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * s["scale"]
    return torch.matmul(_softmax(x, seen[:, None, :]), rows[:, :, :r]).to(BF)


def _plain_expand(s):
    start, r = s["start"].long(), s["r"]
    i = torch.arange(s["n"], device=DEV)
    b = torch.searchsorted(start[1:], i, right=True)
    page, row = _rows(s, b, i - start[b])
    rows = s["pool"][page, row]
    k = torch.einsum("nr,hdr->nhd", rows[:, :r].float(), s["W_K"].float())
    v = torch.einsum("nr,hdr->nhd", rows[:, :r].float(), s["W_V"].float())
    return [k.to(BF), v.to(BF), rows[:, r:].contiguous()]


def _padded(x, start, most):
    """Ragged rows [N, ...] as [B, most, ...], and which of them there are."""
    n = start[1:] - start[:-1]
    i = torch.arange(most, device=DEV)[None, :]
    at = (start[:-1, None] + i).clamp_max(max(0, x.shape[0] - 1))
    return x[at], i < n[:, None]


def _plain_prefill(s):
    q_start, kv_start = s["q_start"].long(), s["kv_start"].long()
    g = s["Hq"] // s["Hkv"]
    if not s["max_q"]:
        return torch.zeros((0, s["Hq"], D), dtype=BF, device=DEV)
    q, is_q = _padded(s["q"].float(), q_start, s["max_q"])
    k, is_k = _padded(s["k"].float().repeat_interleave(g, 1), kv_start, s["max_kv"])
    v, _ = _padded(s["v"].float().repeat_interleave(g, 1), kv_start, s["max_kv"])
    pe, _ = _padded(s["pe"].float(), kv_start, s["max_kv"])
    q, k, v = q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2)
    x = torch.matmul(q[..., :D], k.transpose(2, 3))
    if s["dr"]:
        x += torch.matmul(q[..., D:], pe[:, None].transpose(2, 3))
    x *= s["scale"]
    nq, nk = (q_start[1:] - q_start[:-1])[:, None, None], (kv_start[1:] - kv_start[:-1])[:, None, None]
    i = torch.arange(s["max_q"], device=DEV)[None, :, None]
    j = torch.arange(s["max_kv"], device=DEV)[None, None, :]
    seen = (j <= i + nk - nq) & is_k[:, None, :]
    o = torch.matmul(_softmax(x, seen[:, None]), v)
    return o.transpose(1, 2)[is_q].to(BF)


# -------------------------------------------------------------------------- the framework's

def _own_plan(s, stief):
    if "slots" not in s:
        B, n = s["B"], s["max_tokens"]
        s.update(slots=torch.empty(n, dtype=torch.int32, device=DEV), q_start=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                 kv_start=torch.empty(B + 1, dtype=torch.int32, device=DEV), lens_out=torch.empty(B, dtype=torch.int32, device=DEV),
                 left=torch.empty(1, dtype=torch.int32, device=DEV), ws=stief.plan_workspace())
    stief.stief_plan_pages(s["new_tokens"], s["lens"], s["table"], s["free"], s["count"], s["slots"], s["q_start"],
                           s["kv_start"], s["lens_out"], s["left"], s["ws"], s["ps"])
    return [s[k] for k in ("table", "slots", "q_start", "kv_start", "lens_out", "left")]


def _own_decode(s, stief):
    if "out" not in s:
        s.update(out=torch.empty((s["B"], s["Hq"], s["r"]), dtype=BF, device=DEV),
                 ws=stief.shared_workspace_for(s["B"], s["Hq"], s["r"]))
    return stief.stief_decode_shared_paged(s["q"], s["pool"], s["table"], s["lens"], s["out"], s["ws"],
                                           s["hi"], s["scale"])


def _own_expand(s, stief):
    if "k" not in s:
        s.update(k=torch.empty((s["n"], s["Hq"], D), dtype=BF, device=DEV), v=torch.empty((s["n"], s["Hq"], D), dtype=BF, device=DEV),
                 pe=torch.empty((s["n"], s["dr"]), dtype=BF, device=DEV))
    stief.stief_expand_shared_paged(s["pool"], s["table"], s["start"], s["W_K"], s["W_V"], s["k"], s["v"], s["pe"])
    return [s["k"], s["v"], s["pe"]]


def _own_prefill(s, stief):
    if "out" not in s:
        s.update(out=torch.empty((s["q"].shape[0], s["Hq"], D), dtype=BF, device=DEV))
    return stief.stief_prefill_attention(s["q"], s["k"], s["v"], s["q_start"], s["kv_start"], s["out"], s["max_q"],
                                         s["scale"], k_pe=s["pe"] if s["dr"] else None)


def run(state):
    op = state["op"]
    if own:
        import decode_attention_stief_b200 as stief
        if op == "append":
            stief.stief_append_shared_paged(state["c"], state["pe"], state["slots"], state["pool"])
            return state["pool"]
        return {"plan": _own_plan, "decode": _own_decode, "expand": _own_expand, "prefill": _own_prefill}[op](state, stief)
    return {"plan": _plain_plan, "append": _plain_append, "decode": _plain_decode, "expand": _plain_expand,
            "prefill": _plain_prefill}[op](state)


# ------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "plan":
        B, ps = case["B"], case["ps"]
        lens, new = _spread(B, case["lo"], case["hi"]), _spread(B, case["tlo"], case["thi"], 5)
        pages = sum(-(-(n + t) // ps) - -(-n // ps) for n, t in zip(lens, new))
        n = sum(new) + (sum(new) + 7) // 8
        return {"bytes": 4 * (2 * B + B + 2 * pages + n + 2 * (B + 1) + B + 2), "flops": 0}
    r, dr = case.get("r", 0), case["dr"]
    if op == "append":
        n = case["n"] - case["n"] // 16
        return {"bytes": 4 * case["n"] + 4 * n * (r + dr), "flops": 0}
    lens = _spread(case["B"], case["lo"], case["hi"])
    N, H = sum(lens), case["Hq"]
    if op == "decode":
        return {"bytes": 2 * N * (r + dr) + 2 * case["B"] * H * (2 * r + dr) + 4 * N // case["ps"],
                "flops": 2 * H * N * (2 * r + dr)}
    if op == "expand":
        return {"bytes": 2 * N * (r + dr) + 4 * H * D * r + 4 * N * H * D + 2 * N * dr, "flops": 4 * N * r * H * D}
    kv = [n + p for n, p in zip(lens, _spread(case["B"], 0, case["past"], 3))]
    pairs = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(lens, kv))
    return {"bytes": 2 * N * H * (2 * D + dr) + 2 * sum(kv) * (2 * D * case["Hkv"] + dr), "flops": 2 * H * pairs * (2 * D + dr)}


# ------------------------------------------------------- the definition, one sequence at a time

def _exact_plan(s):
    ps, count, n = s["ps"], int(s["count"]), s["max_tokens"]
    lens, new = s["lens"].tolist(), s["new_tokens"].tolist()
    table, free = s["table"].tolist(), s["free"].tolist()
    cap, asked, used = len(table[0]) * ps, 0, 0
    slots, q_start, kv_start, out = [-1] * n, [0], [0], []
    for b, (have, take) in enumerate(zip(lens, new)):
        first, last = -(-have // ps), -(-(have + take) // ps)
        fits = have + take <= cap and q_start[-1] + take <= n
        if fits and last > first:
            asked += last - first
            fits = asked <= count
            if fits:
                for j in range(first, last):
                    table[b][j] = free[count - 1 - used]
                    used += 1
        if fits:
            for i in range(take):
                t = have + i
                slots[q_start[-1] + i] = table[b][t // ps] * ps + t % ps
        out.append(have + take if fits else have)
        q_start.append(q_start[-1] + take)
        kv_start.append(kv_start[-1] + out[-1])
    return [_int(x) for x in (table, slots, q_start, kv_start, out, [count - used])]


def _sequence(s, b, n):
    """The n rows of sequence b in 64 bits, page by page."""
    ids = s["table"][b, : -(-n // s["ps"])].long()
    return s["pool"].index_select(0, ids).flatten(0, 1)[:n].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(s)
    if op == "append":
        pool = s["pool"].clone()
        slots = s["slots"].tolist()
        at = [(i, t // case["ps"], t % case["ps"]) for i, t in enumerate(slots) if t >= 0]
        i, page, row = torch.tensor(at, device=DEV).unbind(1) if at else [torch.zeros(0, dtype=torch.long, device=DEV)] * 3
        pool[page, row, : case["r"]] = s["c"][i]
        pool[page, row, case["r"]:] = s["pe"][i]
        return pool.double()
    if op == "decode":
        out = torch.zeros((case["B"], case["Hq"], case["r"]), dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                rows = _sequence(s, b, n)
                out[b] = torch.softmax(s["q"][b].double() @ rows.T * s["scale"], -1) @ rows[:, : case["r"]]
        return out
    if op == "expand":
        start = s["start"].tolist()
        rows = torch.cat([_sequence(s, b, start[b + 1] - start[b]) for b in range(case["B"])])
        r, H = case["r"], case["Hq"]
        k, v = ((rows[:, :r] @ s[m].double().reshape(H * D, r).T).reshape(-1, H, D) for m in ("W_K", "W_V"))
        return [k, v, rows[:, r:]]
    out = torch.zeros((s["q"].shape[0], case["Hq"], D), dtype=torch.float64, device=DEV)
    qs, ks, g = s["q_start"].tolist(), s["kv_start"].tolist(), case["Hq"] // case["Hkv"]
    for b in range(case["B"]):
        nq, nk = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        if not nq or not nk:
            continue
        last = torch.arange(nq, device=DEV) + nk - nq  # the last key that each query sees
        hidden = torch.arange(nk, device=DEV) > last[:, None]
        for h in range(case["Hq"]):
            q = s["q"][qs[b]: qs[b + 1], h].double()
            k = torch.cat([s["k"][ks[b]: ks[b + 1], h // g], s["pe"][ks[b]: ks[b + 1]]], 1).double()
            x = (q @ k.T * s["scale"]).masked_fill_(hidden, -math.inf)
            out[qs[b]: qs[b + 1], h] = torch.softmax(x, -1) @ s["v"][ks[b]: ks[b + 1], h // g].double()
    return out
