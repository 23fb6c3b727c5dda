"""The paged-cache operators' measured cases: append, decode attention (with and
without the accumulated attention weight), eviction's selection and its moves.

A cache is K, V pools [n_pages, heads, page, 128], a page table [seqs,
max_pages], row counts ``lens`` [seqs], and per row the accumulated attention
weight ``mass`` and the token position ``pos``, [seqs, heads, max_pages * page].
Row r of (sequence s, KV head h) is slot r % page of page table[s, r // page].
"""
from __future__ import annotations

import math

import torch

own = False

D = 128
SINKS = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step's K/V row of 32 sequences x 8 KV heads: the smallest call, all latency
        dict(name="append_step", op="append", seqs=32, heads=8, page=64, lo=1024, hi=2047, n=1, n_lo=1,
             dtype="bf16", layout="hpd"),
        # four prompts of a batch padded to the longest, from a projection's [tokens, heads, d] output
        dict(name="append_prompt", op="append", seqs=4, heads=8, page=16, lo=0, hi=0, n=8192, n_lo=3001,
             dtype="bf16", layout="phd"),
        # one fp32 unit over a 2k prompt: a short call on one KV head
        dict(name="attend_2k_f32", op="attend", seqs=1, heads=1, g=1, page=16, lo=2048, hi=2048, mass=False,
             dtype="f32", layout="hpd"),
        # a ragged fp32 batch, seven query heads to a KV head, pages shared by the heads row by row
        dict(name="attend_ragged_f32", op="attend", seqs=24, heads=4, g=7, page=32, lo=1, hi=12001, mass=False,
             dtype="f32", layout="phd"),
        # one sequence at 128k: the cache's length has to be split
        dict(name="attend_128k", op="attend", seqs=1, heads=8, g=4, page=128, lo=131071, hi=131071, mass=False,
             dtype="bf16", layout="hpd"),
        # 256 units at a 32k prompt while 1024 tokens are decoded: the largest call
        dict(name="attend_32k", op="attend", seqs=32, heads=8, g=4, page=64, lo=32768, hi=33791, mass=False,
             dtype="bf16", layout="hpd"),
        # the same units held at a budget of 1024 with up to 320 tokens past it, weights accumulated for the eviction
        dict(name="weigh_budget", op="attend", seqs=32, heads=8, g=4, page=16, lo=1025, hi=1344, mass=True,
             dtype="bf16", layout="hpd"),
        # ragged prompts not yet evicted, eight query heads to a KV head
        dict(name="weigh_ragged", op="attend", seqs=8, heads=8, g=8, page=64, lo=1, hi=33791, mass=True,
             dtype="bf16", layout="phd"),
        # eviction every 320 steps, 1344 rows to 1024
        dict(name="select_period", op="select", seqs=32, heads=8, page=16, lo=1344, hi=1344, budget=1024, recent=256),
        # eviction after 128k prompts, to 2048
        dict(name="select_128k", op="select", seqs=4, heads=8, page=64, lo=100003, hi=131071, budget=2048, recent=512),
        dict(name="apply_period", op="apply", seqs=32, heads=8, page=16, lo=1344, hi=1344, budget=1024, recent=256,
             dtype="bf16", layout="hpd"),
        # eviction after 32k prompts, to 1024: nearly every row of the budget moves
        dict(name="apply_32k", op="apply", seqs=16, heads=8, page=64, lo=30011, hi=32768, budget=1024, recent=256,
             dtype="bf16", layout="phd"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "select", "apply"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, seqs=_log_int(rng, 1, 64), heads=_log_int(rng, 1, 8), page=rng.choice([16, 32, 48, 64, 128]))
    most = 3_000_000 // (c["seqs"] * c["heads"])  # rows of a (sequence, head): well below the largest case
    if op == "append":
        n = _log_int(rng, 1, min(16384, max(1, most // 8)))
        hi = _log_int(rng, 1, 4096)
        c.update(lo=rng.randint(0, hi), hi=hi, n=n, n_lo=rng.randint(0, n), dtype=dtype, layout=rng.choice(["hpd", "phd"]))
    elif op == "attend":
        hi = _log_int(rng, 1, min(131072, most))
        c.update(g=rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16]), lo=rng.randint(0, hi), hi=hi,
                 mass=rng.random() < 0.5, dtype=dtype, layout=rng.choice(["hpd", "phd"]))
    else:
        hi = _log_int(rng, 64, min(131072, most))
        budget = _log_int(rng, 32, max(32, hi - 1))
        c.update(lo=rng.randint(1, hi), hi=hi, budget=budget, recent=rng.randint(0, budget - SINKS))
        if op == "apply":
            c.update(dtype=dtype, layout=rng.choice(["hpd", "phd"]))
    return c


def _lens(case):
    """The sequences' row counts: spread over [lo, hi]; they are the case's, not the seed's."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887498949 * s) % 1.0)) for s in range(case["seqs"])]


def _counts(case):
    """How many of a padded append's n rows each sequence brings."""
    lo, hi = case["n_lo"], case["n"]
    return [hi - int((hi - lo + 1) * ((0.6180339887498949 * s) % 1.0)) for s in range(case["seqs"])]


def _n_moves(case, rows):
    """The rows that an eviction moves: the recent ones past the budget, and of the others as large a share as lies past it."""
    B, recent = case["budget"], case["recent"]
    if rows <= B:
        return 0
    late = min(recent, rows - B)
    free = B - SINKS - recent
    return min(rows - B, B - SINKS, late + int(free * (rows - B - late) / max(1, rows - SINKS - recent)))


def work(case):
    heads, page = case["heads"], case["page"]
    lens = _lens(case)
    rows, pages = sum(lens) * heads, sum(-(-n // page) for n in lens)
    if case["op"] == "append":
        elem = 2 if case["dtype"] == "bf16" else 4
        new = sum(_counts(case)) * heads
        return {"bytes": new * (4 * D * elem + 8) + 24 * case["seqs"], "flops": 0}
    if case["op"] == "attend":
        elem = 2 if case["dtype"] == "bf16" else 4
        heads_q = case["seqs"] * heads * case["g"]
        return {"bytes": rows * (2 * D * elem + (8 if case["mass"] else 0)) + heads_q * (D * elem + 4 * D + 4)
                + 4 * pages + 4 * case["seqs"], "flops": 4 * D * case["g"] * rows}
    moves = sum(_n_moves(case, n) for n in lens) * heads
    if case["op"] == "select":
        over = sum(n for n in lens if n > case["budget"]) * heads
        return {"bytes": 8 * over + 8 * moves + 4 * case["seqs"] * heads + 8 * case["seqs"], "flops": 0}
    elem = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": moves * (4 * D * elem + 16 + 8) + 4 * case["seqs"] * heads + 8 * case["seqs"], "flops": 0}


def _pool(gen, n_pages, heads, page, dtype, layout):
    if layout == "hpd":
        return torch.randn(n_pages, heads, page, D, generator=gen, device="cuda", dtype=dtype)
    return torch.randn(n_pages, page, heads, D, generator=gen, device="cuda", dtype=dtype).transpose(1, 2)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1_000_003 * int(seed) + 17)
    op, S, H, P = case["op"], case["seqs"], case["heads"], case["page"]
    lens = _lens(case)
    held = [n + c for n, c in zip(lens, _counts(case))] if op == "append" else lens
    need = [-(-n // P) for n in held]
    width = max(1, max(need))
    R = width * P
    st = dict(op=op, S=S, H=H, P=P, R=R, lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    row = torch.arange(R, device=dev)
    # pages as an allocator hands them out after many sequences have come and gone: in no order
    perm = torch.randperm(sum(need) + 3, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for s in range(S):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    st["table"] = table
    n_pages = sum(need) + 3
    if op != "select":
        dt = DTYPES[case["dtype"]]
        st["K"] = _pool(gen, n_pages, H, P, dt, case["layout"])
        st["V"] = _pool(gen, n_pages, H, P, dt, case["layout"])
    else:  # the selection reads no key and no value
        st["K"] = torch.empty(n_pages, H, P, D, device=dev, dtype=torch.bfloat16)
        st["V"] = torch.empty_like(st["K"])
    # accumulated weights fall off over several decades; evicted caches hold older positions with gaps
    st["mass"] = torch.exp(2.0 * torch.randn(S, H, R, generator=gen, device=dev) - 2.0)
    st["pos"] = row.to(torch.int32).expand(S, H, R).contiguous()
    st["seen"] = st["lens"].clone()
    st["g"] = case.get("g", 1)
    if op == "append":
        dt, n = DTYPES[case["dtype"]], case["n"]
        st["k"] = torch.randn(S, n, H, D, generator=gen, device=dev, dtype=dt).transpose(1, 2)
        st["v"] = torch.randn(S, n, H, D, generator=gen, device=dev, dtype=dt).transpose(1, 2)
        st["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
        st["start"] = st["lens"].clone()
        st["first"] = st["lens"] + torch.randint(0, 5000, (S,), generator=gen, device=dev, dtype=torch.int32)
    elif op == "attend":
        st["q"] = 1.5 * torch.randn(S, H * case["g"], D, generator=gen, device=dev)
        st["q"] = st["q"].to(DTYPES[case["dtype"]])
        st["out"] = torch.zeros(S, H * case["g"], D, device=dev)
        st["lse"] = torch.zeros(S, H * case["g"], device=dev)
        st["mass_out"] = torch.zeros(S, H, R, device=dev) if case["mass"] else None
    else:
        B = case["budget"]
        st["budget"], st["recent"] = B, case["recent"]
        st["moves"] = torch.zeros(S, H, B, 2, dtype=torch.int32, device=dev)
        st["n_moves"] = torch.zeros(S, H, dtype=torch.int32, device=dev)
        if op == "apply":
            # random rows past the budget to random rows below it, both in ascending order
            count = torch.tensor([_n_moves(case, n) for n in lens], device=dev)
            st["n_moves"].copy_(count[:, None].expand(S, H))
            length = st["lens"].long()[:, None, None]
            draw_ = torch.rand(S, H, R, generator=gen, device=dev)
            for col, ok in ((0, (row >= B) & (row < length)), (1, (row >= SINKS) & (row < B) & (row < length))):
                order = torch.where(ok, draw_, torch.full_like(draw_, 2.0)).argsort(dim=-1)[..., :B]
                taken = torch.arange(order.shape[-1], device=dev) < count[:, None, None]
                order = torch.where(taken, order, torch.full_like(order, 1 << 30)).sort(dim=-1).values
                st["moves"][..., :order.shape[-1], col] = torch.where(taken, order, 0).to(torch.int32)
    if own:
        from recallable_kv_cache_gb300 import ckv
        st["cache"] = ckv.PagedCache(st["K"], st["V"], st["table"], st["lens"], g=st["g"], mass=st["mass"],
                                     pos=st["pos"], seen=st["seen"])
    return st


# ---- the plain forms ---------------------------------------------------------
def _plain_append(st):
    S, n = st["S"], st["k"].shape[2]
    s, j = (torch.arange(n, device="cuda") < st["counts"][:, None]).nonzero(as_tuple=True)
    r = st["start"].long()[s] + j
    page, slot = st["table"][s, r // st["P"]].long(), r % st["P"]
    st["K"].transpose(1, 2)[page, slot] = st["k"][s, :, j]
    st["V"].transpose(1, 2)[page, slot] = st["v"][s, :, j]
    st["pos"][s, :, r] = (st["first"][s] + j.to(torch.int32))[:, None].expand(-1, st["H"])
    st["mass"][s, :, r] = 0.0
    st["lens"].copy_(st["start"] + st["counts"])
    st["seen"].copy_(st["first"] + st["counts"])


def _rows(pool, st):
    x = pool[st["table"].clamp(min=0).long()]  # [S, pages, H, P, D]
    return x.transpose(1, 2).reshape(st["S"], st["H"], st["R"], D).float()


def _plain_attend(st):
    S, H, g = st["S"], st["H"], st["g"]
    held = (torch.arange(st["R"], device="cuda") < st["lens"][:, None])[:, None, None, :]
    q = st["q"].float().view(S, H, g, D)
    s = torch.matmul(q, _rows(st["K"], st).transpose(2, 3)) * (1.0 / math.sqrt(D))
    s = s.masked_fill(~held, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    v = _rows(st["V"], st).masked_fill(~held.transpose(2, 3), 0.0)
    st["out"].copy_(torch.matmul(p, v).view(S, H * g, D))
    st["lse"].copy_((m + torch.log(total)).view(S, H * g))
    if st["mass_out"] is not None:
        grown = st["mass"] + p.sum(dim=2)
        st["mass_out"].copy_(torch.where(held[:, :, 0], grown, st["mass_out"]))


def _plain_select(st):
    B = st["budget"]
    row = torch.arange(st["R"], device="cuda")
    length = st["lens"].long()[:, None, None]
    held = row < length
    safe = (st["pos"] < SINKS) | (st["pos"] >= st["seen"][:, None, None] - st["recent"])
    rank = torch.where(held, 1 + safe.to(torch.int32), 0)
    by_mass = st["mass"].nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    by_mass = by_mass.sort(dim=-1, descending=True, stable=True).indices
    by_rank = rank.gather(-1, by_mass).sort(dim=-1, descending=True, stable=True).indices
    order = by_mass.gather(-1, by_rank)[..., :B]
    kept = torch.zeros_like(held.expand_as(safe)).scatter(-1, order, True) & held
    over = length > B
    chosen = torch.stack((kept & (row >= B) & over, ~kept & (row < B) & over), dim=-1)
    s, h, r, col = chosen.nonzero(as_tuple=True)
    k = chosen.cumsum(dim=2)[s, h, r, col] - 1
    st["moves"][s, h, k, col] = r.to(torch.int32)
    st["n_moves"].copy_(chosen[..., 0].sum(dim=-1))


def _plain_apply(st):
    P = st["P"]
    s, h, k = (torch.arange(st["moves"].shape[2], device="cuda") < st["n_moves"][..., None]).nonzero(as_tuple=True)
    src, dst = st["moves"][s, h, k, 0].long(), st["moves"][s, h, k, 1].long()
    p0, p1 = st["table"][s, src // P].long(), st["table"][s, dst // P].long()
    st["K"][p1, h, dst % P] = st["K"][p0, h, src % P]
    st["V"][p1, h, dst % P] = st["V"][p0, h, src % P]
    st["mass"][s, h, dst] = st["mass"][s, h, src]
    st["pos"][s, h, dst] = st["pos"][s, h, src]
    st["lens"].clamp_(max=st["budget"])


def run(st):
    op = st["op"]
    if own:
        cache = st["cache"]
        if op == "append":
            cache.append(st["k"], st["v"], counts=st["counts"], start=st["start"], first=st["first"])
        elif op == "attend":
            if st["mass_out"] is None:
                cache.decode_attn(st["q"], st["out"], lse=st["lse"])
            else:
                cache.decode_attn(st["q"], st["out"], lse=st["lse"], mass_in=st["mass"], mass_out=st["mass_out"])
        elif op == "select":
            cache.evict_select(st["budget"], SINKS, st["recent"], st["moves"], st["n_moves"])
        else:
            cache.evict_apply(st["budget"], st["moves"], st["n_moves"])
    else:
        {"append": _plain_append, "attend": _plain_attend, "select": _plain_select, "apply": _plain_apply}[op](st)
    if op == "attend":
        return {"out": st["out"], "lse": st["lse"], "mass": st["mass_out"]}
    if op == "select":
        return {"moves": st["moves"], "n_moves": st["n_moves"]}
    got = {k: st[k] for k in ("K", "V", "mass", "pos", "lens")}
    if op == "append":
        got["seen"] = st["seen"]
    return got


# ---- the definitions in 64 bits ----------------------------------------------
def exact(case, seed):
    """Each operator from its definition, a sequence (and KV head) at a time.
    The selection gives whole numbers only and has no value here."""
    if case["op"] == "select":
        return None
    st = prepare(case, seed)
    S, H, g, P = st["S"], st["H"], st["g"], st["P"]
    if case["op"] != "attend":
        got = {k: st[k].double() for k in ("K", "V", "mass")}
        for s, n in enumerate(_lens(case)):
            if case["op"] == "append":
                c = _counts(case)[s]
                at = torch.arange(n, n + c, device="cuda")
                page, slot = st["table"][s].long()[at // P], at % P
                for h in range(H):
                    got["K"][page, h, slot] = st["k"][s, h, :c].double()
                    got["V"][page, h, slot] = st["v"][s, h, :c].double()
                got["mass"][s, :, n:n + c] = 0.0
                continue
            for h in range(H):
                src, dst = st["moves"][s, h, :int(st["n_moves"][s, h])].long().unbind(1)
                p0, p1 = st["table"][s].long()[src // P], st["table"][s].long()[dst // P]
                for k in ("K", "V"):
                    got[k][p1, h, dst % P] = got[k][p0, h, src % P]
                got["mass"][s, h, dst] = got["mass"][s, h, src]
        return {**got, "pos": None, "lens": None, "seen": None}
    out = torch.zeros(S, H * g, D, dtype=torch.float64, device="cuda")
    lse = torch.full((S, H * g), -math.inf, dtype=torch.float64, device="cuda")
    mass = torch.zeros(S, H, st["R"], dtype=torch.float64, device="cuda") if case["mass"] else None
    for s, n in enumerate(_lens(case)):
        if n == 0:
            continue
        pages = st["table"][s, :-(-n // P)].long()
        for h in range(H):
            keys = st["K"][pages, h].reshape(-1, D)[:n].double()
            values = st["V"][pages, h].reshape(-1, D)[:n].double()
            logits = st["q"][s, h * g:(h + 1) * g].double() @ keys.T / math.sqrt(D)
            lse[s, h * g:(h + 1) * g] = torch.logsumexp(logits, dim=1)
            weights = torch.softmax(logits, dim=1)
            out[s, h * g:(h + 1) * g] = weights @ values
            if mass is not None:
                mass[s, h, :n] = st["mass"][s, h, :n].double() + weights.sum(dim=0)
    return {"out": out, "lse": lse, "mass": mass}
