"""Measured cases of the operators around a paged cache's batch: page tables and
slot maps made from request lengths (plan), norms and rotary positions of
queries and keys, on their own (rotate) and with the rows going into the pages
(append), and decode attention of sequences that share their leading rows
(shared).

A cache is K, V pools [n_pages, heads, page, 128], a page table [seqs,
max_pages] and row counts ``lens`` [seqs].  Row r of sequence s is slot r % page
of page table[s, r // page].
"""
from __future__ import annotations

import math

import torch

own = False

D = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode step of 32 sequences: one token each, a page now and then; the smallest call, all latency
        dict(name="plan_step", op="plan", seqs=32, page=64, lo=1024, hi=2047, n_lo=1, n=1, evicted=False),
        # a step of a large batch in which a few sequences were evicted or have ended and hand pages back
        dict(name="plan_mixed", op="plan", seqs=509, page=16, lo=0, hi=4095, n_lo=0, n=3, evicted=True),
        # ragged prompts admitted together, tens of thousands of tokens
        dict(name="plan_prompts", op="plan", seqs=48, page=32, lo=0, hi=700, n_lo=1, n=2047, evicted=True),
        # one prompt's queries and keys of a layer with 8 KV heads, before its keys are clustered
        dict(name="rotate_32k", op="rotate", tokens=32768, heads=8, g=4, rot=128, interleaved=False, norm=False,
             dtype="bf16"),
        # a fp32 unit over a 2k prompt, neighbouring channels paired, half of the head rotated, normed
        dict(name="rotate_2k_f32", op="rotate", tokens=2048, heads=1, g=1, rot=64, interleaved=True, norm=True,
             dtype="f32"),
        # a decode step's tokens: normed, rotated, rows into the pages
        dict(name="append_step", op="append", seqs=32, n_lo=1, n=1, heads=8, g=4, page=64, rot=128, interleaved=False,
             norm=True, dtype="bf16", layout="hpd"),
        # ragged prompts, positions of a long context, a quarter of the head left as it is
        dict(name="append_prompts", op="append", seqs=5, n_lo=1001, n=7993, heads=8, g=4, page=16, rot=96,
             interleaved=True, norm=True, dtype="bf16", layout="phd"),
        # eight conversations behind one instruction of 512 rows: latency
        dict(name="shared_512", op="shared", seqs=8, groups=1, prefix_lo=512, prefix=512, lo=17, hi=700, heads=8, g=4,
             page=16, dtype="bf16", layout="hpd"),
        # questions about one 32k document
        dict(name="shared_32k", op="shared", seqs=32, groups=1, prefix_lo=32768, prefix=32768, lo=1, hi=1023, heads=8,
             g=4, page=64, dtype="bf16", layout="hpd"),
        # several documents, ragged groups, seven query heads to a KV head
        dict(name="shared_ragged", op="shared", seqs=61, groups=7, prefix_lo=1000, prefix=20011, lo=0, hi=900, heads=4,
             g=7, page=48, dtype="bf16", layout="phd"),
        # many samples drawn for one 16k prompt: more query rows than one tile holds
        dict(name="shared_samples", op="shared", seqs=160, groups=1, prefix_lo=16384, prefix=16384, lo=1, hi=320, heads=8,
             g=4, page=128, dtype="bf16", layout="hpd"),
        # fp32 rows, two groups
        dict(name="shared_f32", op="shared", seqs=12, groups=2, prefix_lo=2001, prefix=4096, lo=0, hi=257, heads=2, g=4,
             page=16, dtype="f32", layout="hpd"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "rotate", "append", "shared", "shared", "shared"])
    c = dict(op=op)
    if op == "plan":
        c["seqs"] = _log_int(rng, 1, 1024)
        n = _log_int(rng, 1, max(1, min(4096, 90_000 // c["seqs"])))
        hi = _log_int(rng, 1, 16384)
        c.update(page=rng.choice([16, 32, 48, 64, 128]), lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(0, n), n=n,
                 evicted=rng.random() < 0.5)
        return c
    c.update(heads=_log_int(rng, 1, 8), g=rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 16]),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op in ("rotate", "append"):
        most = 1_000_000 // (c["heads"] * (c["g"] + 2))
        c.update(rot=rng.choice([16, 32, 64, 80, 96, 128, 128, 128]), interleaved=rng.random() < 0.5,
                 norm=rng.random() < 0.5)
        if op == "rotate":
            c["tokens"] = _log_int(rng, 1, min(32768, most))
            return c
        c["seqs"] = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, max(1, min(8192, most // c["seqs"])))
        c.update(n_lo=rng.randint(1, n), n=n)
    else:
        c["seqs"] = _log_int(rng, 1, 192)
        c["groups"] = rng.randint(1, max(1, min(c["seqs"], 8)))
        # rows of keys and values, and logits, stay below those of the largest cases
        most = min(65536, 500_000 // (c["heads"] * c["groups"]),
                   60_000_000 // (c["seqs"] * c["heads"] * c["g"]))
        prefix = _log_int(rng, 16, max(16, most))
        hi = _log_int(rng, 1, max(1, min(2048, 250_000 // (c["seqs"] * c["heads"]))))
        c.update(prefix_lo=rng.randint(0, prefix), prefix=prefix, lo=rng.randint(0, hi), hi=hi)
    c.update(page=rng.choice([16, 32, 48, 64, 128]), layout=rng.choice(["hpd", "phd"]))
    return c


GOLD = 0.6180339887498949


def _spread(lo, hi, n, at=0.5):
    """n whole numbers spread over [lo, hi]; they are the case's, not the seed's."""
    return [lo + int((hi - lo + 1) * ((at + GOLD * i) % 1.0)) for i in range(n)]


def _groups(case):
    """Where the groups begin, and the rows that each shares (whole pages)."""
    S, G, P = case["seqs"], case["groups"], case["page"]
    cuts = sorted(_spread(1, S - 1, G - 1, 0.3)) if S > 1 else [1] * (G - 1)
    prefix = [n // P * P for n in _spread(case["prefix_lo"], case["prefix"], G, 0.999)]
    return [0] + cuts + [S], prefix


def _plan_lengths(case):
    """Rows before the call, new tokens, pages in hand, pages of a prefix."""
    S, P = case["seqs"], case["page"]
    start, counts = _spread(case["lo"], case["hi"], S), _spread(case["n_lo"], case["n"], S, 0.9)
    held = [-(-n // P) for n in start]
    shared = [0] * S
    if case["evicted"]:
        for s in range(S):
            if s % 5 == 1:  # cut down to a budget since the last call, its pages still in hand
                start[s] = min(start[s], 1024)
            elif s % 17 == 3:  # has ended
                start[s] = counts[s] = 0
            elif s % 7 == 2:  # the first pages are a prefix's
                shared[s] = min(held[s], 8)
    return start, counts, held, shared


def work(case):
    op = case["op"]
    if op == "plan":
        start, counts, held, shared = _plan_lengths(case)
        need = [max(q, -(-(n + c) // case["page"])) for n, c, q in zip(start, counts, shared)]
        moved = sum(abs(a - b) for a, b in zip(need, held))
        # a token's slot map entry; pages read and written where they change hands; 5 words read, 5 written a sequence
        return {"bytes": 16 * sum(counts) + 8 * moved + 40 * case["seqs"], "flops": 0}
    elem = 2 if case["dtype"] == "bf16" else 4
    H, g = case["heads"], case["g"]
    if op == "rotate":
        n = case["tokens"]
        return {"bytes": n * (2 * H * (g + 1) * D * elem + 4), "flops": 6 * n * H * (g + 1) * case["rot"] // 2}
    if op == "append":
        n = sum(_spread(case["n_lo"], case["n"], case["seqs"], 0.9))
        return {"bytes": n * (2 * H * (g + 2) * D * elem + 16), "flops": 6 * n * H * (g + 1) * case["rot"] // 2}
    cuts, prefix = _groups(case)
    own_rows = _spread(case["lo"], case["hi"], case["seqs"])
    S, flops = case["seqs"], 4 * D * g * H * sum(own_rows)
    for i, p in enumerate(prefix):
        flops += 4 * D * g * H * p * (cuts[i + 1] - cuts[i])
    rows = sum(own_rows) + sum(p for i, p in enumerate(prefix) if cuts[i + 1] > cuts[i])
    return {"bytes": H * (rows * 2 * D * elem + S * g * (D * elem + 4 * D + 4)) + 4 * rows // case["page"] + 4 * S,
            "flops": flops}


def _pool(gen, n_pages, heads, page, dtype, layout):
    if layout == "hpd":
        return torch.randn(n_pages, heads, page, D, generator=gen, device="cuda", dtype=dtype)
    return torch.randn(n_pages, page, heads, D, generator=gen, device="cuda", dtype=dtype).transpose(1, 2)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_plan(case, st, gen):
    S, P = case["seqs"], case["page"]
    start, counts, held, shared = _plan_lengths(case)
    width = max(1, max(max(h, -(-(n + c) // P)) for n, c, h in zip(start, counts, held)))
    need = sum(max(0, max(q, -(-(n + c) // P)) - h) for n, c, h, q in zip(start, counts, held, shared))
    total = sum(held) + need + 5
    # pages as many sequences that came and went have left them: in no order, the free ones in a ring
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    column = torch.arange(width, device="cuda")
    first_page = torch.tensor([sum(held[:s]) for s in range(S)], device="cuda")
    mine = column < _ints(held)[:, None]
    st["table"] = torch.where(mine, perm[(first_page[:, None] + column).clamp(max=total - 1)], -1)
    free = total - sum(held)
    head = int(torch.randint(0, total, (1,), generator=gen, device="cuda"))
    st["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    st["free"][(head + torch.arange(free, device="cuda")) % total] = perm[sum(held):]
    st["span"] = _ints([head, free])
    st["start"], st["counts"], st["held"], st["shared"] = _ints(start), _ints(counts), _ints(held), _ints(shared)
    st["first"] = st["start"] + torch.randint(0, 5000, (S,), generator=gen, device="cuda", dtype=torch.int32)
    # room for a few tokens more than there are, as a captured step's buffers have
    st["slots"] = torch.zeros(sum(counts) + 3, 4, dtype=torch.int32, device="cuda")
    for name in ("lens", "seen", "held_out", "granted"):
        st[name] = torch.zeros(S, dtype=torch.int32, device="cuda")
    st["starts"] = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    st["span_out"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    if own:  # the plan reads no key and no value
        from recallable_kv_cache_gb300 import ckv
        pool = torch.empty(total, 1, P, D, dtype=torch.bfloat16, device="cuda")
        st["cache"] = ckv.PagedCache(pool, pool, st["table"], st["lens"], seen=st["seen"])


def _prepare_rotary(case, st, gen, tokens):
    H, g, dt = case["heads"], case["g"], DTYPES[case["dtype"]]
    st["rot"], st["interleaved"], st["g"] = case["rot"], case["interleaved"], g
    # a projection's output: the queries, keys and values of a token side by side
    qkv = torch.randn(tokens, H * (g + 2), D, generator=gen, device="cuda", dtype=dt)
    st["q"], st["k"], st["v"] = qkv[:, :H * g], qkv[:, H * g:H * (g + 1)], qkv[:, H * (g + 1):]
    st["q_out"] = torch.zeros(tokens, H * g, D, dtype=dt, device="cuda")
    for name in ("q_weight", "k_weight"):
        st[name] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None
    # base 500000 as for long contexts, the far half of the frequencies interpolated
    half = case["rot"] // 2
    inv = [500000.0 ** (-i / half) / (1.0 if 2 * i < half else 8.0) for i in range(half)]
    st["inv"] = torch.tensor(inv, dtype=torch.float64, device="cuda")
    if own:
        from recallable_kv_cache_gb300 import ckv
        st["turns"] = ckv.rotary_turns(inv).cuda()


def _prepare_append(case, st, gen):
    S, H, P = case["seqs"], case["heads"], case["page"]
    counts = _spread(case["n_lo"], case["n"], S, 0.9)
    start = _spread(0, 1000, S)
    need = [-(-(n + c) // P) for n, c in zip(start, counts)]
    width, n_pages, T = max(need), sum(need) + 3, sum(counts)
    _prepare_rotary(case, st, gen, T)
    dt = DTYPES[case["dtype"]]
    st["K"] = _pool(gen, n_pages, H, P, dt, case["layout"])
    st["V"] = _pool(gen, n_pages, H, P, dt, case["layout"])
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    column = torch.arange(width, device="cuda")
    first_page = torch.tensor([sum(need[:s]) for s in range(S)], device="cuda")
    table = torch.where(column < _ints(need)[:, None], perm[(first_page[:, None] + column).clamp(max=n_pages - 1)], -1)
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), _ints(counts).long())
    j = torch.arange(T, device="cuda") - torch.tensor([sum(counts[:s]) for s in range(S)], device="cuda")[seq]
    row = _ints(start).long()[seq] + j
    far = torch.randint(0, 120_000, (S,), generator=gen, device="cuda")  # evicted rows leave positions ahead of rows
    slot = table[seq, row // P].long() * P + row % P
    st["slots"] = torch.stack((slot, seq, row, row + far[seq]), dim=1).to(torch.int32)
    R = width * P
    st["pos"] = torch.zeros(S, H, R, dtype=torch.int32, device="cuda")
    st["mass"] = torch.rand(S, H, R, generator=gen, device="cuda")
    if own:
        from recallable_kv_cache_gb300 import ckv
        st["lens"] = _ints([n + c for n, c in zip(start, counts)])
        st["cache"] = ckv.PagedCache(st["K"], st["V"], table, st["lens"], g=case["g"], mass=st["mass"], pos=st["pos"],
                                     seen=st["lens"].clone())


def _prepare_shared(case, st, gen):
    S, H, g, P, dt = case["seqs"], case["heads"], case["g"], case["page"], DTYPES[case["dtype"]]
    cuts, prefix = _groups(case)
    own_rows = _spread(case["lo"], case["hi"], S)
    own_pages = [-(-n // P) for n in own_rows]
    of = [max(i for i in range(len(prefix)) if cuts[i] <= s) for s in range(S)]
    lens = [prefix[of[s]] + own_rows[s] for s in range(S)]
    n_pages = sum(p // P for p in prefix) + sum(own_pages) + 3
    width = max(1, max(-(-n // P) for n in lens))
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, p in enumerate(prefix):
        table[cuts[i]:cuts[i + 1], :p // P] = perm[at:at + p // P]
        at += p // P
    for s in range(S):
        table[s, prefix[of[s]] // P:-(-lens[s] // P)] = perm[at:at + own_pages[s]]
        at += own_pages[s]
    st.update(S=S, H=H, g=g, P=P, cuts=cuts, prefix=prefix, of=of, table=table, lens_host=lens, lens=_ints(lens),
              K=_pool(gen, n_pages, H, P, dt, case["layout"]), V=_pool(gen, n_pages, H, P, dt, case["layout"]))
    st["q"] = (1.5 * torch.randn(S, H * g, D, generator=gen, device="cuda")).to(dt)
    st["out"] = torch.zeros(S, H * g, D, device="cuda")
    st["lse"] = torch.zeros(S, H * g, device="cuda")
    if own:
        from recallable_kv_cache_gb300 import ckv
        st["group_starts"], st["prefix_rows"] = _ints(cuts), _ints(prefix)
        st["cache"] = ckv.PagedCache(st["K"], st["V"], table, st["lens"], g=g, shared=True)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * int(seed) + 29)
    st = dict(op=case["op"], P=case.get("page"))
    if case["op"] == "plan":
        _prepare_plan(case, st, gen)
    elif case["op"] == "rotate":
        n = case["tokens"]
        _prepare_rotary(case, st, gen, n)
        st["k_out"] = torch.zeros(n, case["heads"], D, dtype=DTYPES[case["dtype"]], device="cuda")
        # prompts laid end to end, somewhere in a long context
        st["positions"] = (torch.arange(n, device="cuda") + torch.randint(0, 120_000, (1,), generator=gen,
                                                                          device="cuda")).to(torch.int32)
    elif case["op"] == "append":
        _prepare_append(case, st, gen)
    else:
        _prepare_shared(case, st, gen)
    return st


# ---- the plain forms ---------------------------------------------------------
def _plain_plan(st):
    P, cap = st["P"], st["free"].numel()
    start, counts, held = st["start"].long(), st["counts"].long(), st["held"].long()
    need = torch.maximum((start + counts + P - 1) // P, st["shared"].long())
    take, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    run_ = take.cumsum(0)
    ok = (take == 0) | (run_ <= st["span"][1])
    take = torch.where(ok, take, 0)
    before = take.cumsum(0) - take
    column = torch.arange(st["table"].shape[1], device="cuda")
    k = column - held[:, None]
    new = (k >= 0) & (k < take[:, None])
    head, tail = st["span"][0].long(), st["span"].long().sum()
    pages = st["free"][(head + before[:, None] + k).remainder(cap)]
    k = column - need[:, None]
    back = (k >= 0) & (k < give[:, None])
    at = (tail + (give.cumsum(0) - give)[:, None] + k).remainder(cap)
    st["free"][at[back]] = st["table"][back]
    st["table"].copy_(torch.where(new, pages, st["table"]))
    granted = torch.where(ok, counts, 0)
    st["granted"].copy_(granted)
    st["held_out"].copy_(held + take - give)
    st["lens"].copy_(start + granted)
    st["seen"].copy_(st["first"] + granted)
    st["span_out"].copy_(torch.stack(((head + take.sum()) % cap, st["span"][1] - take.sum() + give.sum())))
    st["starts"][:1] = 0
    st["starts"][1:] = counts.cumsum(0)
    t = torch.arange(st["slots"].shape[0], device="cuda")
    s = (torch.searchsorted(st["starts"], t.to(torch.int32), right=True) - 1).clamp(max=start.numel() - 1)
    j = t - st["starts"][s]
    row = start[s] + j
    fine = (j < counts[s]) & ok[s]
    page = st["table"][s, torch.where(fine, row // P, 0)].long()
    entry = torch.stack((page * P + row % P, s, row, st["first"][s] + j), dim=1)
    st["slots"].copy_(torch.where(fine[:, None], entry, -1))


def _plain_rotary(x, weight, cos, sin, rot, interleaved):
    """x [tokens, heads, 128] in 32 bits: normed over the head, its first rot channels rotated."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight
    turn = x[..., :rot]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _angles(st, positions):
    angle = positions.double()[:, None, None] * st["inv"]
    return angle.cos().float(), angle.sin().float()


def _plain_rotate(st):
    cos, sin = _angles(st, st["positions"])
    st["q_out"].copy_(_plain_rotary(st["q"], st["q_weight"], cos, sin, st["rot"], st["interleaved"]))
    st["k_out"].copy_(_plain_rotary(st["k"], st["k_weight"], cos, sin, st["rot"], st["interleaved"]))


def _plain_append(st):
    slot, seq, row, position = st["slots"].long().unbind(1)
    cos, sin = _angles(st, position)
    st["q_out"].copy_(_plain_rotary(st["q"], st["q_weight"], cos, sin, st["rot"], st["interleaved"]))
    k = _plain_rotary(st["k"], st["k_weight"], cos, sin, st["rot"], st["interleaved"])
    page, at = slot // st["P"], slot % st["P"]
    st["K"].transpose(1, 2)[page, at] = k.to(st["K"].dtype)
    st["V"].transpose(1, 2)[page, at] = st["v"]
    st["pos"].transpose(1, 2)[seq, row] = position.to(torch.int32)[:, None].expand(-1, st["pos"].shape[1])
    st["mass"].transpose(1, 2)[seq, row] = 0.0


def _rows(pool, pages):
    """pages [..., n] -> [..., H, n * P, 128] in 32 bits."""
    x = pool[pages.clamp(min=0).long()].transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, D).float()


def _plain_shared(st):
    S, H, g, P = st["S"], st["H"], st["g"], st["P"]
    scale = 1.0 / math.sqrt(D)
    q = st["q"].float().view(S, H, g, D) * scale
    m = torch.full((S, H, g, 1), -math.inf, device="cuda")
    total = torch.zeros(S, H, g, 1, device="cuda")
    acc = torch.zeros(S, H, g, D, device="cuda")
    # the rows that a group shares: once for all of its queries
    for i, p in enumerate(st["prefix"]):
        a, b = st["cuts"][i], st["cuts"][i + 1]
        if p == 0 or a == b:
            continue
        pages = st["table"][a, :p // P]
        logits = torch.matmul(q[a:b].transpose(0, 1).reshape(H, -1, D), _rows(st["K"], pages).transpose(1, 2))
        top = logits.amax(dim=-1, keepdim=True)
        e = torch.exp(logits - top)
        for to, x in ((m, top), (total, e.sum(dim=-1, keepdim=True)), (acc, torch.matmul(e, _rows(st["V"], pages)))):
            to[a:b] = x.view(H, b - a, g, -1).transpose(0, 1)
    # each sequence's own rows
    skip = torch.tensor([st["prefix"][i] for i in st["of"]], device="cuda")
    width = max(1, max(-(-n // P) - st["prefix"][i] // P for n, i in zip(st["lens_host"], st["of"])))
    column = skip[:, None] // P + torch.arange(width, device="cuda")
    pages = st["table"].gather(1, column.clamp(max=st["table"].shape[1] - 1))
    kept = (skip[:, None] + torch.arange(width * P, device="cuda") < st["lens"][:, None])[:, None, None, :]
    logits = torch.matmul(q, _rows(st["K"], pages).transpose(2, 3)).masked_fill(~kept, -math.inf)
    top = torch.maximum(m, logits.amax(dim=-1, keepdim=True))
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(logits - safe)
    old = torch.exp(m - safe)
    total = total * old + e.sum(dim=-1, keepdim=True)
    acc = acc * old + torch.matmul(e, _rows(st["V"], pages).masked_fill(~kept.transpose(2, 3), 0.0))
    st["out"].copy_(torch.where(total > 0, acc / total, torch.zeros_like(acc)).view(S, H * g, D))
    st["lse"].copy_((safe + torch.log(total)).view(S, H * g))


def run(st):
    op = st["op"]
    if own:
        from recallable_kv_cache_gb300 import ckv
        if op == "plan":
            st["cache"].plan(st["counts"], st["held"], st["free"], st["span"], st["slots"], st["starts"], st["granted"],
                             shared=st["shared"], start=st["start"], first=st["first"], held_out=st["held_out"],
                             span_out=st["span_out"])
        elif op == "rotate":
            ckv.rotate(st["q"], st["k"], st["positions"], st["turns"], st["q_out"], st["k_out"],
                       interleaved=st["interleaved"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS)
        elif op == "append":
            st["cache"].append_rotated(st["q"], st["k"], st["v"], st["slots"], st["turns"], st["q_out"],
                                       interleaved=st["interleaved"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                                       eps=EPS)
        else:
            st["cache"].shared_attn(st["q"], st["out"], st["group_starts"], st["prefix_rows"], lse=st["lse"])
    else:
        {"plan": _plain_plan, "rotate": _plain_rotate, "append": _plain_append, "shared": _plain_shared}[op](st)
    names = {"plan": ("table", "free", "span_out", "held_out", "lens", "seen", "granted", "starts", "slots"),
             "rotate": ("q_out", "k_out"), "append": ("q_out", "K", "V", "pos", "mass"), "shared": ("out", "lse")}
    return {k: st[k] for k in names[op]}


# ---- the definitions in 64 bits ----------------------------------------------
def _turned(x, weight, positions, case):
    """The norm and the rotation as a complex product: channels (a, b) of pair i are a + ib times e^(i p w_i)."""
    y = x.double()
    if weight is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    w = torch.tensor([500000.0 ** (-n / half) / (1.0 if 2 * n < half else 8.0) for n in range(half)],
                     dtype=torch.float64, device="cuda")
    z = torch.complex(y[..., a], y[..., b])
    z = z * torch.polar(torch.ones_like(w), positions.double()[:, None] * w)[:, None, :]
    got = y.clone()
    got[..., a], got[..., b] = z.real, z.imag
    return got


def exact(case, seed):
    """Each operator from its definition; the plan gives whole numbers only and has no value here."""
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return {"q_out": _turned(st["q"], st["q_weight"], st["positions"], case),
                "k_out": _turned(st["k"], st["k_weight"], st["positions"], case)}
    if case["op"] == "append":
        slot, seq, row, position = st["slots"].long().unbind(1)
        got = {name: st[name].double() for name in ("K", "V", "mass")}
        k = _turned(st["k"], st["k_weight"], position, case)
        for h in range(case["heads"]):
            got["K"][slot // st["P"], h, slot % st["P"]] = k[:, h]
            got["V"][slot // st["P"], h, slot % st["P"]] = st["v"][:, h].double()
            got["mass"][seq, h, row] = 0.0
        return {**got, "q_out": _turned(st["q"], st["q_weight"], position, case), "pos": None}
    S, H, g, P = st["S"], st["H"], st["g"], st["P"]
    out = torch.zeros(S, H * g, D, dtype=torch.float64, device="cuda")
    lse = torch.full((S, H * g), -math.inf, dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lens_host"]):  # every sequence by itself, over all of its rows
        if n == 0:
            continue
        pages = st["table"][s, :-(-n // P)].long()
        keys = st["K"][pages].transpose(0, 1).reshape(H, -1, D)[:, :n].double()
        values = st["V"][pages].transpose(0, 1).reshape(H, -1, D)[:, :n].double()
        logits = torch.matmul(st["q"][s].double().view(H, g, D), keys.transpose(1, 2)) / math.sqrt(D)
        lse[s] = torch.logsumexp(logits, dim=-1).view(-1)
        out[s] = torch.matmul(torch.softmax(logits, dim=-1), values).view(-1, D)
    return {"out": out, "lse": lse}
