"""GPU parity of a paged batch's step (plans and slot maps, norms and rotary
positions, attention of sequences that share leading rows) against its oracle in
64 bits, through the public entry points.

Tolerances.  Plans are whole numbers and exact.  A rotated channel is
amplitude * (y_a cos t -+ y_b sin t): the norm's sum of squares takes 12
roundings in a row and its root is off by 2^-22, so that y is off by less than
2^-20 of itself; the angle is exact to 2^-32 of a turn and half a unit of a float
of at most pi / 4, cos and sin are within 2 units and the amplitude and the two
products add one each: less than 2^-20 |amplitude| in all.  So a channel is off
by at most 2^-19 |amplitude| (|y_a| + |y_b|), and by half a step of its type, 2^-8
(bf16) or 2^-24 (fp32) of itself.  Shared attention is held to the decode
attention's bounds: a tile of 128 rows takes 24 tensor-core steps on a sum that
starts from zero, which is less than its n / 16 + 200."""
import math

import numpy as np
import pytest
import torch

import oracle.batch as ob
import oracle.paged as po
from recallable_kv_cache_gb300 import ckv
from test_gpu_paged import D, DT, pools

pytestmark = pytest.mark.gpu
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plans
class Plan:
    """Random pages in a ring and in hand; every table entry that is not held is -1."""

    def __init__(self, start, counts, page=16, shared=None, extra=3, seed=0, width=None, n_slots=None, held=None, avail=None,
                 seen=True, heads=1):
        rng = np.random.default_rng(seed)
        S = len(start)
        self.page, self.seen_on = page, seen
        held = [-(-max(0, n) // page) for n in start] if held is None else held
        need = [-(-max(0, n + c) // page) for n, c in zip(start, counts)]
        self.width = width or max(1, max(max(need), max(held)))
        total = sum(held) + sum(max(0, a - b) for a, b in zip(need, held)) + extra
        perm = rng.permutation(total).tolist()
        table = np.full((S, self.width), -1, dtype=np.int32)
        at = 0
        for s, h in enumerate(held):
            table[s, :h] = perm[at:at + h]
            at += h
        free = perm[at:]
        free = free if avail is None else free[:avail]
        head = int(rng.integers(0, total))
        ring = np.full(total, -1, dtype=np.int32)
        for i, p in enumerate(free):
            ring[(head + i) % total] = p
        self.S, self.total = S, total
        first = rng.integers(0, 5000, S).tolist()
        self.n_slots = max(1, sum(max(0, c) for c in counts) + 2) if n_slots is None else n_slots
        self.host = dict(start=list(start), counts=list(counts), first=first, held=list(held),
                         shared=[0] * S if shared is None else list(shared), span=[head, len(free)])
        self.table, self.ring = ints(table), ints(ring)
        self.table0, self.ring0 = table, ring
        self.dev = {k: ints(v) for k, v in self.host.items()}
        self.lens, self.seen = (torch.full((S,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        self.held_out, self.granted = (torch.full((S,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        self.span_out = torch.full((2,), -7, dtype=torch.int32, device="cuda")
        self.starts = torch.full((S + 1,), -7, dtype=torch.int32, device="cuda")
        self.slots = torch.full((self.n_slots, 4), -7, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pool = torch.empty(total, heads, page, D, dtype=torch.bfloat16, device="cuda")
        self.cache = ckv.PagedCache(pool, pool, self.table, self.lens, seen=self.seen if seen else None, dev_err=self.err)

    def run(self, **kw):
        d = self.dev
        args = dict(shared=d["shared"], start=d["start"], first=d["first"] if self.seen_on else None, held_out=self.held_out,
                    span_out=self.span_out)
        args.update(kw)
        self.cache.plan(d["counts"], d["held"], self.ring, d["span"], self.slots, self.starts, self.granted, **args)

    def check(self, held_out=None, span_out=None, was=(-7, -7)):
        torch.cuda.synchronize()
        h = self.host
        want = ob.plan(self.table0, h["counts"], h["start"], h["first"] if self.seen_on else h["start"], h["shared"], h["held"],
                       self.ring0, h["span"], self.page, self.n_slots, self.total)
        assert self.table.tolist() == want["table"] and self.ring.tolist() == want["ring"]
        assert (self.held_out if held_out is None else held_out).tolist() == want["held"]
        assert (self.span_out if span_out is None else span_out).tolist() == want["span"]
        assert self.granted.tolist() == want["granted"] and self.starts.tolist() == want["starts"]
        assert self.slots.tolist() == want["slots"]
        for got, key, old in ((self.lens, "lens", was[0]), (self.seen, "seen", was[1])):
            if key == "seen" and not self.seen_on:
                continue
            for s, (x, y) in enumerate(zip(got.tolist(), want[key])):
                assert x == (old if isinstance(old, int) else old[s]) if y is None else x == y
        met = {0: set(), 2: {"index"}, 3: {"count"}}[int(self.err)]
        assert met <= want["errors"] and bool(met) == bool(want["errors"])
        return want


def rand(n, lo, hi, seed):
    return np.random.default_rng(seed).integers(lo, hi + 1, n).tolist()


PLANS = [
    # start, counts, page
    ([0], [1], 16), ([0], [0], 16), ([15], [1], 16), ([16], [1], 16), ([5], [700], 48), ([0, 0, 0], [0, 0, 0], 32),
    ([31, 32, 33], [1, 1, 1], 32), (rand(40, 0, 300, 1), rand(40, 0, 3, 2), 16), (rand(255, 0, 99, 3), [1] * 255, 16),
    (rand(257, 0, 99, 4), [1] * 257, 64), (rand(9, 0, 3, 5), rand(9, 0, 900, 6), 128),
    (rand(1024, 0, 70, 7), rand(1024, 0, 2, 8), 16), (rand(1025, 0, 70, 9), rand(1025, 0, 1, 10), 16),
    (rand(3001, 0, 40, 11), rand(3001, 0, 1, 12), 16), (rand(2500, 0, 40, 13), rand(2500, 0, 5, 14), 48),
    ([0, 100, 7], [5000, 0, 1], 16), ([0] * 3, [2047, 0, 1], 64), ([0], [2049], 16), ([3] * 200, [60] * 200, 32),
]


@pytest.mark.parametrize("start,counts,page", PLANS)
def test_plan(start, counts, page):
    p = Plan(start, counts, page, seed=len(start))
    p.run()
    p.check()


@pytest.mark.parametrize("S,n", [(7, 1), (300, 2), (60, 200), (1500, 1), (1500, 7)])
@pytest.mark.parametrize("seen", [False, True])
def test_plan_with_pages_handed_back(S, n, seen):
    """Evicted sequences, ended ones, prefixes' pages."""
    start, counts = rand(S, 0, 500, S), rand(S, 0, n, S + 1)
    held = [-(-x // 16) + y for x, y in zip(start, rand(S, 0, 12, S + 2))]
    for s in range(0, S, 5):
        start[s] = counts[s] = 0
    shared = [min(h, x) for h, x in zip(held, rand(S, 0, 3, S + 3))]
    p = Plan(start, counts, 16, shared, held=held, seed=S, seen=seen)
    p.run()
    p.check()
    # the same call again gives the same again: nothing it reads has changed
    p.run()
    p.check()


@pytest.mark.parametrize("S,avail", [(6, 0), (6, 1), (40, 9), (1100, 100), (2100, 1)])
def test_plan_with_too_few_pages(S, avail):
    p = Plan(rand(S, 0, 60, S), rand(S, 0, 40, S + 1), 16, avail=avail, seed=S)
    p.run()
    want = p.check()
    assert 0 in want["granted"]


@pytest.mark.parametrize("S", [5, 1030])
def test_plan_in_place(S):
    """lens and seen as start and first, held and span updated where they are; a
    loop of steps, then the sequences end one by one."""
    p = Plan(rand(S, 0, 50, S), [1] * S, 16, width=12, extra=9 * S, n_slots=S, seed=S)
    p.lens.copy_(p.dev["start"])
    p.seen.copy_(p.dev["first"])
    for step in range(40):
        if step % 7 == 5:
            end = torch.arange(S, device="cuda") % 11 == step % 11
            p.lens.masked_fill_(end, 0)
            p.seen.masked_fill_(end, 0)
        p.host.update(start=p.lens.tolist(), first=p.seen.tolist(), held=p.dev["held"].tolist(), span=p.dev["span"].tolist())
        p.table0, p.ring0 = p.table.cpu().numpy().copy(), p.ring.cpu().numpy().copy()
        p.run(start=None, first=None, held_out=None, span_out=None)
        p.check(held_out=p.dev["held"], span_out=p.dev["span"])


def test_plan_counts_from_lens():
    p = Plan([16, 0, 3], [16, 0, 3], 16)
    p.lens.copy_(p.dev["start"])
    p.seen.copy_(p.dev["first"])
    p.cache.plan(p.lens, p.dev["held"], p.ring, p.dev["span"], p.slots, p.starts, p.granted, shared=p.dev["shared"],
                 held_out=p.held_out, span_out=p.span_out)
    p.check()


@pytest.mark.parametrize("n_slots", [300, 5000])
@pytest.mark.parametrize("S", [3, 1100])
def test_plan_positions_from_lens(S, n_slots):
    """Positions count from the old lens, rows from other numbers, and the cache has no seen."""
    start, counts, lens = rand(S, 0, 9, 1), rand(S, 0, 1, 2), rand(S, 0, 300, 3)
    counts[1] = 100
    p = Plan(start, counts, 16, n_slots=n_slots, seen=False)
    p.lens.copy_(ints(lens))
    p.run(first=p.lens)
    h = p.host
    want = ob.plan(p.table0, counts, start, lens, h["shared"], h["held"], p.ring0, h["span"], 16, n_slots, p.total)
    torch.cuda.synchronize()
    assert p.slots.tolist() == want["slots"] and p.lens.tolist() == [n if n is not None else x for n, x in zip(want["lens"], lens)]


BAD_SEQS = [dict(start=-1), dict(counts=-1), dict(first=-1), dict(held=-1), dict(held=99), dict(shared=-1), dict(shared=9),
            dict(start=2 ** 31 - 1), dict(counts=2 ** 31 - 1), dict(first=2 ** 31 - 1), dict(counts=200)]


@pytest.mark.parametrize("bad", BAD_SEQS)
@pytest.mark.parametrize("S", [4, 1500])
def test_bad_sequences_are_left_alone(bad, S):
    p = Plan([20, 30, 40, 50] + [3] * (S - 4), [3, 4, 5, 6] + [0] * (S - 4), 16, width=8, seed=3)
    for key, value in bad.items():
        p.host[key][2] = value
        p.dev[key][2] = value
    p.run()
    p.check()
    assert int(p.err) == 3


@pytest.mark.parametrize("S", [4, 300, 1200])
@pytest.mark.parametrize("counts,n_slots,granted", [([4, 3, 3, 1], 9, [4, 3, 0, 0]), ([4, 3, 900, 0], 9, [4, 3, 0, 0]),
                                                    ([1000, 5, 1200, 3], 2100, [1000, 5, 0, 0])])
def test_slots_that_do_not_fit(S, counts, n_slots, granted):
    """Tokens past the slot map are refused; sequences without any still hand their pages back."""
    p = Plan([0] * S, counts + [0] * (S - 4), 16, n_slots=n_slots, held=[0] * (S - 1) + [0 if S == 4 else 2], seed=S)
    p.run()
    want = p.check()
    assert want["granted"][:4] == granted and int(p.err) == 3
    assert want["starts"][3] == n_slots and want["held"][-1] == 0


@pytest.mark.parametrize("span", [[-1, 2], [10 ** 6, 2], [0, -1], [0, 10 ** 6]])
def test_a_span_outside_the_ring_is_empty(span):
    p = Plan([15, 3], [1, 20], 16)
    p.host["span"] = span
    p.dev["span"].copy_(ints(span))
    p.run()
    want = p.check()
    assert want["span"] == [0, 0] and want["granted"] == [1, 0]


def test_pages_handed_back_to_a_full_ring_are_lost():
    p = Plan([0, 0], [0, 0], 16, held=[3, 2], extra=1)
    p.ring = ints(p.ring0[:4].copy())
    p.ring0 = p.ring0[:4]
    p.host["span"] = [2, 1]
    p.dev["span"].copy_(ints([2, 1]))
    p.run()
    want = p.check()
    assert want["span"] == [2, 4] and int(p.err) == 3


def test_bad_page_ids_give_no_slot():
    p = Plan([20, 5], [20, 4], 16)
    p.table[0, 1] = 10 ** 6
    p.table0 = p.table.cpu().numpy().copy()
    p.run()
    want = p.check()
    assert int(p.err) == 2 and [-1] * 4 in want["slots"][:20]


def test_plan_replayed():
    """Captured once: the step after step of a growing batch."""
    S = 33
    p = Plan([0] * S, [1] * S, 16, width=4, extra=2 * S, n_slots=S)
    p.lens.zero_()
    p.seen.zero_()
    h, sp = p.dev["held"], p.dev["span"]
    run = lambda: p.cache.plan(p.dev["counts"], h, p.ring, sp, p.slots, p.starts, p.granted)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run()
    for step in range(40):
        g.replay()
    torch.cuda.synchronize()
    assert p.lens.tolist() == [40] * S and h.tolist() == [3] * S and int(sp[1]) == 3 * S - 3 * S
    pages = p.table[:, :3].flatten().tolist()
    assert len(set(pages)) == 3 * S


# ---------------------------------------------------------------- norms and rotary positions
def check_rows(got, x, positions, turns, rot, interleaved, weight, eps, amplitude, dtype):
    """got, x [tokens, heads, 128] against the oracle row by row."""
    got, x = got.double().cpu().numpy(), x.double().cpu().numpy()
    turns = [int(t) % 2 ** 64 for t in turns.tolist()] if turns is not None else []
    w = None if weight is None else weight.double().cpu().numpy()
    for t, p in enumerate(positions):
        for h in range(x.shape[1]):
            want = ob.rotary(x[t, h], p, turns, rot, interleaved, w, eps, amplitude)
            y = np.abs(ob.rotary(x[t, h], 0, [], 0, False, w, eps))
            size = y.copy()
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                size[a] = size[b] = abs(amplitude) * (y[a] + y[b])
            bound = 2.0 ** -19 * size + HALF_STEP[dtype] * np.abs(want) * (1 + 2.0 ** -10) + 1e-37
            if w is None:
                bound[rot:] = 0.0  # untouched channels stay what they are
            assert (np.abs(got[t, h] - want) <= bound).all(), (t, h, np.abs(got[t, h] - want).max())


ROTATE = [
    # tokens, heads_q, heads_k, rot, interleaved, norm, dtype
    (1, 1, 1, 128, False, False, "bf16"), (1, 1, 1, 128, True, True, "f32"), (1, 32, 8, 128, False, True, "bf16"),
    (3, 5, 3, 64, True, False, "bf16"), (17, 4, 1, 16, False, True, "f32"), (16, 1, 1, 80, True, True, "bf16"),
    (33, 7, 2, 96, False, False, "f32"), (5, 0, 4, 112, False, True, "bf16"), (5, 3, 0, 48, True, True, "f32"),
    (9, 2, 2, 0, False, True, "bf16"), (2, 64, 8, 128, True, True, "f32"), (130, 12, 4, 32, False, True, "bf16"),
    (700, 1, 2, 128, False, True, "bf16"), (41, 16, 16, 128, True, False, "f32"),
]


@pytest.mark.parametrize("tokens,hq,hk,rot,interleaved,norm,dtype", ROTATE)
def test_rotate(tokens, hq, hk, rot, interleaved, norm, dtype):
    gen = torch.Generator().manual_seed(tokens + hq)
    q, k = ((2 * torch.randn(tokens, h, D, generator=gen)).to(DT[dtype]).cuda() if h else None for h in (hq, hk))
    w = [1 + 0.3 * torch.randn(D, generator=gen).cuda() if norm else None for _ in range(2)]
    positions = torch.randint(-5, 2 ** 20, (tokens,), generator=gen, dtype=torch.int32)
    positions[0] = 2 ** 31 - 1
    freq, amplitude = ckv.rotary_frequencies(rot or 2, 500000.0, "ramp", 4.0)
    turns = ckv.rotary_turns(freq).cuda() if rot else None
    qo, ko = (None if x is None else torch.full_like(x, 9.0) for x in (q, k))
    args = dict(interleaved=interleaved, q_weight=w[0], k_weight=w[1], eps=1e-5, amplitude=amplitude)
    ckv.rotate(q, k, positions.cuda(), turns, qo, ko, **args)
    for got, x, weight in ((qo, q, w[0]), (ko, k, w[1])):
        if x is not None:
            check_rows(got, x, positions.tolist(), turns, rot, interleaved, weight, 1e-5, amplitude, dtype)
    # in place, the same bits
    q2, k2 = (None if x is None else x.clone() for x in (q, k))
    ckv.rotate(q2, k2, positions.cuda(), turns, q2, k2, **args)
    assert all(x is None or torch.equal(x, y) for x, y in ((q2, qo), (k2, ko)))


def sample(n, seed):
    """The first and last tokens and some between."""
    return sorted({0, 1, n - 2, n - 1} | set(np.random.default_rng(seed).integers(0, n, 12).tolist()))


LONG = [
    # rows a token: queries, keys; enough tokens that a lane group has 20 to 24 of them, or all 12 of a few heads
    (32, 8, 128, False, True, "bf16"), (32, 8, 128, True, True, "f32"), (40, 8, 96, True, False, "bf16"),
    (33, 8, 64, False, False, "f32"), (8, 4, 128, True, True, "bf16"), (41, 0, 0, False, True, "f32"),
]


@pytest.mark.parametrize("hq,hk,rot,interleaved,norm,dtype", LONG)
def test_rotate_long(hq, hk, rot, interleaved, norm, dtype):
    """Prompts, where every block keeps four rows under way and takes the next as they are done."""
    gen = torch.Generator(device="cuda").manual_seed(hq + hk)
    tokens = 5003
    x = torch.randn(tokens, hq + hk, D, generator=gen, device="cuda").to(DT[dtype])
    q, k = x[:, :hq], x[:, hq:] if hk else None
    w = [1 + 0.3 * torch.randn(D, generator=gen, device="cuda") if norm else None for _ in range(2)]
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda") + 99_000
    turns = ckv.rotary_turns(ckv.rotary_frequencies(rot)[0]).cuda() if rot else None
    qo, ko = (None if x is None else torch.full_like(x, 9.0) for x in (q, k))
    args = dict(interleaved=interleaved, q_weight=w[0], k_weight=w[1])
    ckv.rotate(q, k, positions, turns, qo, ko, **args)
    at = sample(tokens, rot)
    for got, rows, weight in ((qo, q, w[0]), (ko, k, w[1])):
        if rows is not None:
            check_rows(got[at], rows[at], positions[at].tolist(), turns, rot, interleaved, weight, 1e-6, 1.0, dtype)
    # every row is what a call of few tokens, whose blocks share a token's rows out, makes of it, and in place the same
    few = [None if rows is None else torch.empty_like(rows) for rows in (q, k)]
    for t in range(0, tokens, 150):
        part = lambda rows: None if rows is None else rows[t:t + 150]
        ckv.rotate(part(q), part(k), positions[t:t + 150], turns, part(few[0]), part(few[1]), **args)
    ckv.rotate(q, k, positions, turns, q, k, **args)
    for got, rows, one in ((qo, q, few[0]), (ko, k, few[1])):
        assert rows is None or torch.equal(got, rows) and torch.equal(got, one)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_strided(dtype, interleaved):
    """A projection's output, heads of a wide row, a broadcast key, outputs inside a wider buffer."""
    gen = torch.Generator().manual_seed(5)
    qkv = torch.randn(21, 7, 136, generator=gen).to(DT[dtype]).cuda()
    q, k = qkv[:, 1:5, 8:], qkv[:1, 5:6, :128].expand(21, 3, 128)
    positions = torch.randint(0, 10 ** 6, (21,), generator=gen, dtype=torch.int32)
    turns = ckv.rotary_turns(ckv.rotary_frequencies(128)[0]).cuda()
    wide = torch.full((21, 9, 144), 5.0, dtype=DT[dtype], device="cuda")
    qo, ko = wide[:, ::2][:, :4, 8:136], torch.full((3, 21, 128), 5.0, dtype=DT[dtype], device="cuda").transpose(0, 1)
    ckv.rotate(q, k, positions.cuda(), turns, qo, ko, interleaved=interleaved)
    check_rows(qo, q, positions.tolist(), turns, 128, interleaved, None, 0, 1.0, dtype)
    check_rows(ko, k, positions.tolist(), turns, 128, interleaved, None, 0, 1.0, dtype)
    assert (wide[..., :8] == 5).all() and (wide[..., 136:] == 5).all() and (wide[:, 1::2] == 5).all()
    # a token or head by itself: torch gives such an extent any stride
    one = torch.empty_strided((1, 1, 128), (7, 3, 1), dtype=DT[dtype], device="cuda")
    one.copy_(q[3:4, :1])
    ckv.rotate(one, None, positions[3:4].cuda(), turns, one, None, interleaved=interleaved)
    assert torch.equal(one, qo[3:4, :1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotate_rows_between_each_other(dtype):
    """Outputs between the rows that are read, in one tensor: heads, tokens and projections interleaved."""
    gen = torch.Generator().manual_seed(6)
    turns = ckv.rotary_turns(ckv.rotary_frequencies(128)[0]).cuda()
    positions = torch.randint(0, 10 ** 6, (19,), generator=gen, dtype=torch.int32)
    for shape, cut in (((19, 5, 2, D), lambda x: (x[:, :, 0], x[:, :, 1])), ((19, 2, 5, D), lambda x: (x[:, 0], x[:, 1])),
                       ((5, 19, 2, D), lambda x: (x[:, :, 0].transpose(0, 1), x[:, :, 1].transpose(0, 1))),
                       ((19, 15, D), lambda x: (x[:, :10:2], x[:, 1:10:2])), ((19, 15, D), lambda x: (x[:, ::3], x[:, 1::3]))):
        x = torch.randn(*shape, generator=gen).to(DT[dtype]).cuda()
        q, o = cut(x)
        before, rows = x.clone(), q.clone()
        ckv.rotate(q, None, positions.cuda(), turns, o, None)
        check_rows(o, rows, positions.tolist(), turns, 128, False, None, 0, 1.0, dtype)
        changed = before != x
        cut(changed)[1].fill_(False)
        assert not changed.any()
    for q, o in ((x[:, :5], x[:, 1:6]), (x[:, :5], x[:, 4:9]), (x[:, :5], x[:, 5:10].flip(0)[:1].expand(19, 5, D))):
        with pytest.raises(ckv.CKVError):
            ckv.rotate(q, None, positions.cuda(), turns, o, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotate_values(dtype):
    """Zero rows, tiny ones, infinities and NaN: what the formula says, row by row."""
    x = torch.ones(6, 1, D)
    x[0] = 0.0
    x[1] = 1e-30
    x[2] = 1e18
    x[3, 0, 100] = math.inf
    x[4, 0, 3] = math.nan
    x = x.to(DT[dtype]).cuda()
    turns = ckv.rotary_turns(ckv.rotary_frequencies(64)[0]).cuda()
    positions = ints([7] * 6)
    out = torch.zeros_like(x)
    ckv.rotate(x, None, positions, turns, out, None)
    keep = [0, 1, 2, 5]
    check_rows(out[keep], x[keep], [7] * 4, turns, 64, False, None, 0, 1.0, dtype)
    assert torch.equal(out[3, 0, 64:], x[3, 0, 64:]) and out[3].isfinite().sum() == D - 1
    assert out[4].isnan().nonzero()[:, 1].tolist() == [3, 35]
    w = torch.full((D,), 2.0, device="cuda")
    ckv.rotate(x, None, positions, turns, out, None, q_weight=w, eps=1e-6)
    check_rows(out[keep], x[keep], [7] * 4, turns, 64, False, w, 1e-6, 1.0, dtype)
    assert not out[0].any()


class Append:
    def __init__(self, start, counts, heads=2, g=4, page=16, dtype="bf16", layout="hpd", state=True, seed=0):
        gen = torch.Generator().manual_seed(seed)
        S, T = len(start), sum(counts)
        need = [-(-(n + c) // page) for n, c in zip(start, counts)]
        width = max(need)
        n_pages = sum(need) + 2
        self.K, self.V = pools(n_pages, heads, page, dtype, layout, gen)
        perm = torch.randperm(n_pages, generator=gen)
        table = torch.full((S, width), -1, dtype=torch.int32)
        at = 0
        rows = []
        for s in range(S):
            table[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
            for j in range(counts[s]):
                r = start[s] + j
                rows.append([int(table[s, r // page]) * page + r % page, s, r, r + 1000 * s])
        self.rows, self.page, self.heads, self.g, self.dtype, self.T = rows, page, heads, g, dtype, T
        qkv = torch.randn(T, heads * (g + 2), D, generator=gen).to(DT[dtype]).cuda()
        self.q, self.k, self.v = qkv[:, :heads * g], qkv[:, heads * g:heads * (g + 1)], qkv[:, heads * (g + 1):]
        self.q_out = torch.full((T, heads * g, D), 3.0, dtype=DT[dtype], device="cuda") if g else None
        R = width * page
        self.pos = torch.full((S, heads, R), -5, dtype=torch.int32, device="cuda") if state else None
        self.mass = torch.full((S, heads, R), 4.0, device="cuda") if state else None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.slots = ints(rows)
        self.cache = ckv.PagedCache(self.K, self.V, table.cuda(), torch.zeros(S, dtype=torch.int32, device="cuda"), g=max(g, 1),
                                    mass=self.mass, pos=self.pos, seen=torch.zeros(S, dtype=torch.int32, device="cuda"),
                                    dev_err=self.err)
        self.weights = [1 + 0.2 * torch.randn(D, generator=gen).cuda() for _ in range(2)]

    def check(self, turns, rot, interleaved, before, left_out=()):
        torch.cuda.synchronize()
        K0, V0, pos0, mass0 = before
        kept = [t for t in range(self.T) if t not in left_out]
        at = [self.rows[t] for t in kept]
        if self.g:
            check_rows(self.q_out[kept], self.q[kept], [x[3] for x in at], turns, rot, interleaved, self.weights[0], 1e-6, 1.0,
                       self.dtype)
            assert all((self.q_out[t] == 3).all() for t in left_out)
        page, slot = [x[0] // self.page for x in at], [x[0] % self.page for x in at]
        check_rows(self.K[page, :, slot], self.k[kept], [x[3] for x in at], turns, rot, interleaved, self.weights[1], 1e-6, 1.0,
                   self.dtype)
        assert torch.equal(self.V[page, :, slot], self.v[kept])
        for pool, old in ((self.K, K0), (self.V, V0)):
            same = torch.ones(pool.shape[0], pool.shape[2], dtype=torch.bool, device="cuda")
            same[page, slot] = False
            a, b = pool.transpose(1, 2)[same], old.transpose(1, 2)[same]
            assert torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))
        if self.pos is not None:
            for x in at:
                pos0[x[1], :, x[2]] = x[3]
                mass0[x[1], :, x[2]] = 0.0
            assert torch.equal(self.pos, pos0) and torch.equal(self.mass, mass0)

    def before(self):
        return [None if x is None else x.clone() for x in (self.K, self.V, self.pos, self.mass)]


APPEND = [
    # start, counts, heads, g, page, dtype, layout, rot, interleaved, state
    ([0], [1], 1, 1, 16, "bf16", "hpd", 128, False, True), ([0, 15, 16], [1, 1, 1], 2, 4, 16, "bf16", "phd", 64, True, True),
    ([3, 0], [100, 33], 8, 4, 48, "bf16", "wide", 128, False, True), ([3, 0], [20, 5], 3, 7, 32, "f32", "kv_in_page", 96, True, False),
    ([0, 9], [130, 1], 1, 16, 64, "f32", "phd", 128, False, True), ([0] * 30, [1] * 30, 4, 0, 16, "bf16", "hpd", 32, False, True),
    ([5], [300], 2, 1, 128, "bf16", "hpd", 0, False, False),
]


@pytest.mark.parametrize("start,counts,heads,g,page,dtype,layout,rot,interleaved,state", APPEND)
def test_append_rotated(start, counts, heads, g, page, dtype, layout, rot, interleaved, state):
    a = Append(start, counts, heads, g, page, dtype, layout, state)
    turns = ckv.rotary_turns(ckv.rotary_frequencies(rot)[0]).cuda() if rot else None
    before = a.before()
    a.cache.append_rotated(a.q if g else None, a.k, a.v, a.slots, turns, a.q_out, interleaved=interleaved,
                           q_weight=a.weights[0], k_weight=a.weights[1])
    a.check(turns, rot, interleaved, before)
    assert int(a.err) == 0


@pytest.mark.parametrize("heads,g,page,dtype,layout,rot,interleaved", [
    (8, 4, 16, "bf16", "phd", 128, False), (8, 4, 64, "f32", "hpd", 96, True), (4, 8, 48, "bf16", "hpd", 128, True),
    (8, 3, 32, "f32", "phd", 128, False),
])
def test_append_long(heads, g, page, dtype, layout, rot, interleaved):
    """Prompts of 40 to 48 rows a token into pages; tokens left out among them."""
    counts = [1300, 7, 1999]
    a = Append([3, 0, 40], counts, heads, g, page, dtype, layout)
    turns = ckv.rotary_turns(ckv.rotary_frequencies(rot)[0]).cuda()
    a.slots[[100, 2000]] = -1
    a.pos.fill_(-5)
    a.cache.append_rotated(a.q, a.k, a.v, a.slots, turns, a.q_out, interleaved=interleaved, q_weight=a.weights[0],
                           k_weight=a.weights[1])
    torch.cuda.synchronize()
    rows = torch.tensor(a.rows, device="cuda")
    kept = torch.ones(a.T, dtype=torch.bool, device="cuda")
    kept[[100, 2000]] = False
    page_of, slot = rows[:, 0] // page, rows[:, 0] % page
    at = [t for t in sample(a.T, rot) if t not in (100, 2000)]
    where = rows[at, 3].tolist()
    check_rows(a.q_out[at], a.q[at], where, turns, rot, interleaved, a.weights[0], 1e-6, 1.0, dtype)
    check_rows(a.K[page_of[at], :, slot[at]], a.k[at], where, turns, rot, interleaved, a.weights[1], 1e-6, 1.0, dtype)
    assert torch.equal(a.V[page_of, :, slot][kept], a.v[kept])
    # all rows: those of the rotation by itself
    positions = rows[:, 3].int()
    qo, ko = torch.full_like(a.q, 3.0), torch.empty_like(a.k)
    ckv.rotate(a.q, a.k, positions, turns, qo, ko, interleaved=interleaved, q_weight=a.weights[0], k_weight=a.weights[1])
    assert torch.equal(a.q_out[kept], qo[kept]) and (a.q_out[~kept] == 3).all()
    assert torch.equal(a.K[page_of, :, slot][kept], ko[kept])
    pos, mass = torch.full_like(a.pos, -5), torch.full_like(a.mass, 4.0)
    pos[rows[kept, 1], :, rows[kept, 2]] = positions[kept][:, None]
    mass[rows[kept, 1], :, rows[kept, 2]] = 0.0
    assert torch.equal(a.pos, pos) and torch.equal(a.mass, mass) and int(a.err) == 0


def test_append_with_queries_in_place():
    a, b = (Append([3, 0], [40, 33], 2, 4, 16) for _ in range(2))
    turns = ckv.rotary_turns(ckv.rotary_frequencies(128)[0]).cuda()
    a.cache.append_rotated(a.q, a.k, a.v, a.slots, turns, a.q_out)
    b.cache.append_rotated(b.q, b.k, b.v, b.slots, turns, b.q)
    assert torch.equal(a.q_out, b.q) and torch.equal(a.k, b.k)
    at = a.slots[:, 0].long()
    for x, y in ((a.K, b.K), (a.V, b.V)):
        assert torch.equal(x[at // 16, :, at % 16], y[at // 16, :, at % 16])


@pytest.mark.parametrize("column,value,code", [(0, -1, 0), (0, -2, 2), (0, 10 ** 7, 2), (1, -1, 2), (1, 2, 2), (2, -1, 2),
                                               (2, 10 ** 6, 2)])
def test_tokens_without_a_place_are_left_out(column, value, code):
    a = Append([3, 0], [40, 33], 2, 4, 16)
    turns = ckv.rotary_turns(ckv.rotary_frequencies(128)[0]).cuda()
    for t in (5, 60):
        a.slots[t, column] = value
    before = a.before()
    a.cache.append_rotated(a.q, a.k, a.v, a.slots, turns, a.q_out, q_weight=a.weights[0], k_weight=a.weights[1])
    a.check(turns, 128, False, before, left_out=(5, 60))
    assert int(a.err) == code


# ---------------------------------------------------------------- shared rows
class Shared:
    """Groups of sequences on a prefix's pages and pages of their own; every row that is not held is NaN."""

    def __init__(self, groups, heads=2, g=4, page=16, dtype="bf16", layout="hpd", seed=0, q_scale=1.5, width=None):
        """groups: [(prefix rows in whole pages, [rows of its own for each member])]"""
        gen = torch.Generator().manual_seed(seed)
        lens = [p + n for p, own in groups for n in own]
        S = len(lens)
        pages = sum(p // page for p, _ in groups) + sum(-(-n // page) for _, own in groups for n in own) + 2
        width = width or max(1, max(-(-n // page) for n in lens))
        self.K, self.V = pools(pages, heads, page, dtype, layout, gen)
        perm = torch.randperm(pages, generator=gen).to(torch.int32)
        table = torch.full((S, width), 2 ** 31 - 1, dtype=torch.int32)
        held = torch.zeros(pages, page, dtype=torch.bool)
        at = s = 0
        self.starts, self.prefix = [0], []
        for p, own in groups:
            common = perm[at:at + p // page]
            held[common.long()] = True
            at += p // page
            for n in own:
                table[s, :p // page] = common
                for i in range(-(-n // page)):
                    table[s, p // page + i] = perm[at]
                    held[perm[at].long(), :min(page, n - i * page)] = True
                    at += 1
                s += 1
            self.starts.append(s)
            self.prefix.append(p)
        mask = ~held.cuda()[:, None, :, None].expand(pages, heads, page, D)
        self.K.masked_fill_(mask, float("nan"))
        self.V.masked_fill_(mask, float("nan"))
        self.S, self.heads, self.g, self.page, self.n_pages, self.dtype = S, heads, g, page, pages, dtype
        self.lens_list, self.table = lens, table.cuda()
        self.lens = ints(lens)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q = (q_scale * torch.randn(S, heads * g, D, generator=gen)).to(DT[dtype]).cuda()
        self.out = torch.full((S, heads * g, D), float("nan"), device="cuda")
        self.lse = torch.full((S, heads * g), float("nan"), device="cuda")
        self.handle = self.make()

    def make(self):
        return ckv.PagedCache(self.K, self.V, self.table, self.lens, g=self.g, dev_err=self.err, shared=True)

    def run(self, starts=None, prefix=None, **kw):
        self.handle.shared_attn(self.q, self.out, ints(self.starts if starts is None else starts),
                                ints(self.prefix if prefix is None else prefix), lse=self.lse, **kw)

    def check(self, scale=None, skip_bad=False):
        torch.cuda.synchronize()
        scale = D ** -0.5 if scale is None else scale
        out, lse = self.out.double(), self.lse.double()
        worst = 0.0
        for s, n in enumerate(self.lens_list):
            pages = self.table[s, :-(-n // self.page)].long()
            ok = ((pages >= 0) & (pages < self.n_pages)).repeat_interleave(self.page)[:n]
            pages = pages.clamp(0, self.n_pages - 1)
            k, v = (x[pages].transpose(0, 1).reshape(self.heads, -1, D)[:, :n].double()[:, ok] for x in (self.K, self.V))
            q = self.q[s].double().view(self.heads, self.g, D)
            got, z = out[s].view(self.heads, self.g, D), lse[s].view(self.heads, self.g)
            if k.shape[1] == 0:
                assert not got.any() and (z == -math.inf).all()
                continue
            logits = scale * torch.matmul(q, k.transpose(1, 2))
            want_z = torch.logsumexp(logits, dim=-1)
            p = torch.exp(logits - want_z[..., None])
            es = 2.0 ** -16 * abs(scale) * float(torch.matmul(q.abs(), k.abs().transpose(1, 2)).max())
            sums = 2.0 ** -23 * (n / 16 + 200)
            eps = 4 * es + 2.0 ** -16 + 2 * sums
            bound = eps * torch.matmul(p, v.abs()) + 1e-30
            off = (got - torch.matmul(p, v)).abs()
            assert (off <= bound).all(), (s, float((off / bound).max()))
            assert ((z - want_z).abs() <= 2 * es + 2.0 ** -19 + sums + 2.0 ** -23 * want_z.abs()).all(), s
            worst = max(worst, float(off.norm() / torch.matmul(p, v).norm()))
        return worst


SHARED = [
    # groups, heads, g, page, dtype, layout
    ([(16, [1, 1])], 1, 1, 16, "bf16", "hpd"),
    ([(128, [0, 0])], 1, 4, 16, "bf16", "hpd"),
    ([(256, [5, 0, 17])], 2, 4, 64, "bf16", "phd"),
    ([(112, [3, 4]), (144, [1, 2, 3]), (0, [7, 8])], 3, 2, 16, "bf16", "kv_in_page"),
    ([(480, [31, 1, 300])], 2, 8, 48, "bf16", "wide"),
    ([(1024, [1] * 40)], 2, 4, 128, "bf16", "hpd"),          # 160 queries a head: two blocks
    ([(512, [1] * 64), (96, [3] * 33)], 1, 8, 32, "bf16", "phd"),  # 512 queries, 264
    ([(64, [2]), (64, [1, 0]), (0, [0, 0]), (0, [0])], 2, 16, 16, "bf16", "hpd"),
    ([(5120, [9, 100])], 4, 1, 16, "bf16", "hpd"),
    ([(20000, [3, 700, 33])], 1, 7, 32, "bf16", "hpd"),
    ([(32 * (i % 5), [i % 4] * (1 + i % 3)) for i in range(90)], 2, 3, 32, "bf16", "hpd"),
    ([(288, [5, 150, 0])], 2, 4, 144, "bf16", "hpd"), ([(768, [1, 2, 300])], 1, 8, 256, "bf16", "phd"),
    ([(64, [0, 1, 2, 0]), (160, [0] * 1100)], 1, 1, 16, "bf16", "hpd"),     # more sequences than fit the prep's shared memory
    ([(16 * (i % 4), [i % 2, 1]) for i in range(300)], 1, 2, 16, "bf16", "hpd"),  # more groups than it has threads
    ([(16, [1, 1])], 1, 1, 16, "f32", "hpd"),
    ([(480, [31, 1, 300]), (96, [3, 4])], 2, 9, 48, "f32", "wide"),
    ([(2048, [100] * 9)], 2, 4, 16, "f32", "phd"),
]


@pytest.mark.parametrize("groups,heads,g,page,dtype,layout", SHARED)
def test_shared_attention(groups, heads, g, page, dtype, layout):
    c = Shared(groups, heads, g, page, dtype, layout, seed=heads + g)
    c.run()
    c.check()
    assert int(c.err) == 0


@pytest.mark.parametrize("scale", [0.0, -0.11, 0.5])
def test_shared_scale_and_strided_queries(scale):
    c = Shared([(96, [9, 17]), (0, [3])], 2, 3, 32)
    wide = torch.zeros(3, 2 * 6 + 5, 136 * 2, dtype=DT["bf16"], device="cuda")
    q = wide[:, 1:12:2, 8:136]
    q.copy_(c.q)
    c.q = q
    c.run(scale=scale)
    c.check(scale=scale)


def test_shared_peaked_and_far_scores():
    c = Shared([(1024, [100, 0, 33])], 2, 4, 16, q_scale=40.0)
    c.run()
    c.check()


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 100, 200, 207, 10 ** 9])
def test_shared_prefixes_of_any_length(prefix):
    """Rounded down to a multiple of 16, clamped to the first member's rows (all share 208)."""
    c = Shared([(208, [0, 5, 30])], 2, 4, 16)
    c.run(prefix=[prefix])
    c.check()
    assert int(c.err) == 0


@pytest.mark.parametrize("starts,prefix", [([0, 2], [64]), ([1, 3], [64]), ([0, 2, 4], [64, 64]), ([0, 0, 4, 4], [9, 64, 9]),
                                           ([4, 4], [64]), ([0, 4], [48]), ([0, 1, 2, 3, 4], [64] * 4), ([2, 4], [0])])
def test_shared_groups_of_any_kind(starts, prefix):
    """Sequences outside every group, groups of none and of one."""
    c = Shared([(64, [0, 5, 30, 100])], 2, 4, 16)
    c.run(starts, prefix)
    c.check()
    assert int(c.err) == 0


@pytest.mark.parametrize("starts,prefix", [([-3, 4], [64]), ([0, 9], [64]), ([2, 0, 4], [64, 64]), ([0, 3, 1, 4], [64, 64, 64]),
                                           ([0, 4], [-5])])
def test_shared_bad_groups_are_reported(starts, prefix):
    c = Shared([(64, [0, 5, 30, 100])], 2, 4, 16)
    c.run(starts, prefix)
    c.check()
    assert int(c.err) == 3


def test_shared_lengths_outside_the_cache():
    """A length above the capacity is clamped to it, a negative one is none, inside and outside of groups."""
    c = Shared([(64, [0, 0]), (0, [5, 7, 0])], 2, 4, 16, width=4)
    c.lens.copy_(ints([10 ** 9, 64, -3, 7, -1]))
    c.run()
    c.lens_list = [64, 64, 0, 7, 0]
    c.check()
    assert int(c.err) == 3


def test_shared_many_sequences_without_rows_of_their_own():
    """More groups than one warp has lanes, shares that pass from unit to unit, sequences without any row."""
    c = Shared([(160 + 16 * (i % 9), [0] * (2 + i % 3)) for i in range(40)] + [(0, [0, 0, 3])], 4, 8, 16, seed=3)
    c.run()
    c.check()
    assert int(c.err) == 0


def test_shared_member_shorter_than_the_prefix():
    c = Shared([(64, [0, 5, 30])], 2, 4, 16)
    c.lens[1] = 20
    c.run()
    c.lens_list[1] = 64
    c.check()
    assert int(c.err) == 3


@pytest.mark.parametrize("starts,prefix,clean", [
    ([-3, 4], [64], None), ([0, 9], [64], None), ([2, 0, 4], [64, 64], None), ([0, 3, 1, 4], [64, 64, 64], None),
    ([0, 4], [-5], None), ([0, 4], [64], [64, 69, 94, 64]), ([0, 3, 4], [70, 64], [64, 69, 94, 0]),
])
def test_shared_fp32_groups_are_looked_at(starts, prefix, clean):
    """Bad starts and prefixes are reported, and a member shorter than the prefix attends all of it,
    as with bf16 (clean: the rows that count once the last member's are set to none)."""
    c = Shared([(64, [0, 5, 30, 100])], 2, 4, 16, "f32")
    if clean:
        c.lens[3], c.lens_list = 0, clean
    c.run(starts, prefix)
    c.check()
    assert int(c.err) == (3 if clean is None or clean[3] else 0)


@pytest.mark.parametrize("short", [1, 1099])
def test_shared_fp32_shorter_member_of_many(short):
    """More sequences and groups than the look at few of them holds."""
    c = Shared([(32, [1, 0])] * 40 + [(160, [i % 3 for i in range(1100)])], 1, 2, 16, "f32")
    c.run()
    c.check()
    assert int(c.err) == 0
    c.lens[80 + short], c.lens_list[80 + short] = 33, 160
    c.run()
    c.check()
    assert int(c.err) == 3


@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
def test_shared_fp32_shorter_members_of_few(g):
    """As many groups and sequences as a block looks up by itself, every form of the fp32 tiles."""
    c = Shared([(32, [1, 0])] * 31 + [(160, [i % 3 for i in range(962)])], 1, g, 16, "f32")
    assert len(c.prefix) == 32 and c.S == 1024
    for s in (1, 61, 63, 700, 1023):
        c.lens[s], c.lens_list[s] = 5, 160 if s > 61 else 32
    c.run()
    c.check()
    assert int(c.err) == 3


@pytest.mark.parametrize("page", [16, 48, 128])
def test_shared_bad_pages_are_skipped(page):
    """Bad ids in the prefix and in a sequence's own pages; a whole tile of them."""
    c = Shared([(page * 20, [5, 300]), (page * 2, [1, 1])], 2, 4, page)
    for s in (0, 1):
        c.table[s, 3] = -1
        c.table[s, 19] = 10 ** 6
    if page <= 48:
        c.table[:2, 8:17] = 2 ** 31 - 1
    c.table[1, 21] = -7
    c.run()
    c.check()
    assert int(c.err) == 2


def test_shared_equals_itself():
    """The order in which blocks run does not change a bit."""
    c = Shared([(20000, [3, 700, 33]), (777 * 16, [1] * 20)], 2, 4, 16)
    c.run()
    first = (c.out.clone(), c.lse.clone())
    for _ in range(20):
        c.run()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_shared_first_runs_of_one_tile():
    """Units of two tiles dealt out three to a block: every other block begins with the last tile of one."""
    c = Shared([(256, [0, 0])] * 57, 4, 4, 16)
    c.run()
    c.check()
    first = c.out.clone()
    for _ in range(300):
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and int(c.err) == 0


def test_shared_exactness():
    """The error of fp32 weights, over a long prefix: the decode attention's."""
    c = Shared([(32768, [3, 100])], 2, 4, 64)
    c.run()
    assert c.check() <= 1e-6


def test_shared_rows_of_the_type_s_largest_values():
    c = Shared([(128, [3, 4])], 1, 2, 16)
    pages = c.table[0, :8].long()
    c.V[pages[2]] = torch.finfo(torch.bfloat16).max
    c.K[pages[2]] = -100.0
    c.q.fill_(1.0)
    c.run()
    c.check()


@pytest.mark.parametrize("row,own", [(3, [0, 0]), (3, [5, 40]), (70, [20, 40])])
def test_shared_nan_in_a_held_row(row, own):
    """What the decode attention makes of it, in the shared rows and in a sequence's own."""
    c = Shared([(64, own)], 2, 4, 16)
    for pool in (c.K, c.V):
        pool[c.table[0, row // 16].long(), 1, row % 16, 7] = float("nan")
        d = [torch.zeros_like(c.out), torch.zeros_like(c.lse)]
        c.run()
        c.handle.decode_attn(c.q, d[0], lse=d[1])
        assert torch.equal(c.out.isnan(), d[0].isnan()) and torch.equal(c.lse.isnan(), d[1].isnan())
        assert c.out.isnan().any()


@pytest.mark.parametrize("own", [[40000, 3], [2000, 1999], [5000] * 3])
def test_shared_long_own_rows(own):
    """Own rows of more and of fewer blocks than the join takes."""
    for heads, groups in ((1, [(64, own)]), (2, [(0, own), (0, [700])])):
        c = Shared(groups, heads, 4, 16)
        c.run()
        c.check()
        first = c.out.clone()
        c.run()
        assert torch.equal(c.out, first)


def test_shared_captured_and_on_streams():
    """Two handles over the same tensors replayed side by side, lens growing between replays."""
    c = Shared([(512, [5, 30, 100])], 2, 4, 16, width=48)
    d = Shared([(512, [5, 30, 100])], 2, 4, 16, width=48, seed=1)
    side = torch.cuda.Stream()
    graphs = []
    for x in (c, d):
        x.g_starts, x.g_prefix = ints(x.starts), ints(x.prefix)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            x.handle.shared_attn(x.q, x.out, x.g_starts, x.g_prefix, lse=x.lse)
        graphs.append(graph)
    torch.cuda.synchronize()
    for step in range(3):
        other = torch.cuda.Stream()
        for _ in range(5):
            graphs[0].replay()
            with torch.cuda.stream(other):
                graphs[1].replay()
        torch.cuda.synchronize()
        for x in (c, d):
            x.check()
            x.lens_list = [n - 1 if n > 513 else n for n in x.lens_list]
            x.lens.copy_(ints(x.lens_list))


def test_shared_lookups_follow_the_calls_before():
    """Lengths, groups, prefixes and queries written just before each call, in one replayed graph:
    every call sees its own, as a call by itself does."""
    c = Shared([(512, [5, 30, 100, 64]), (96, [7, 200])], 2, 4, 16)
    wide = [dict(starts=[0, 4, 6], prefix=[512, 96], cut=0), dict(starts=[0, 2, 6], prefix=[256, 0], cut=3),
            dict(starts=[1, 4, 6], prefix=[480, 64], cut=0), dict(starts=[0, 4, 5], prefix=[16, 96], cut=5),
            dict(starts=[3, 3, 6], prefix=[0, 0], cut=1), dict(starts=[0, 4, 6], prefix=[512, 96], cut=2)]
    starts, prefix, q = ints([0, 0, 0]), ints([0, 0]), torch.zeros_like(c.q)
    states = [(ints(x["starts"]), ints(x["prefix"]), ints([n - x["cut"] for n in c.lens_list]), c.q * (1 + i))
              for i, x in enumerate(wide)]
    outs = [torch.zeros_like(c.out) for _ in states]

    def calls():
        for (s, p, n, rows), out in zip(states, outs):
            starts.copy_(s), prefix.copy_(p), c.lens.copy_(n), q.copy_(rows)
            c.handle.shared_attn(q, out, starts, prefix)

    alone = []
    for (s, p, n, rows) in states:
        c.lens.copy_(n)
        out = torch.zeros_like(c.out)
        torch.cuda.synchronize()
        c.handle.shared_attn(rows, out, s, p)
        torch.cuda.synchronize()
        alone.append(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        calls()
    for _ in range(50):
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, alone))
    assert int(c.err) == 0


@pytest.mark.parametrize("how", ["argument", "current"])
def test_shared_handle_dropped_with_work_queued_on_another_stream(how):
    """Its workspace is not handed out while a side stream has yet to use it."""
    c = Shared([(4096, [5, 300, 100])], 2, 4, 16)
    c.run()
    out, starts, prefix = torch.zeros_like(c.out), ints(c.starts), ints(c.prefix)
    handle, side = c.make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    at, nbytes = handle.workspace.data_ptr(), handle.workspace.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some 0.2 s
        if how == "current":
            handle.shared_attn(c.q, out, starts, prefix)
    if how == "argument":
        handle.shared_attn(c.q, out, starts, prefix, stream=side)
    del handle
    others = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()
    for t in others:
        assert not t.data_ptr() <= at < t.data_ptr() + nbytes
        t.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(out, c.out)
    c.check()


def test_shared_after_a_call_with_weights():
    """One workspace for calls of both kinds, in any order."""
    c = Shared([(64, [0, 5, 30]), (0, [100])], 2, 4, 16)
    mass = torch.zeros(c.S, 2, c.table.shape[1] * 16, device="cuda")
    pos, seen = torch.zeros_like(mass, dtype=torch.int32), c.lens.clone()
    handle = ckv.PagedCache(c.K, c.V, c.table, c.lens, g=4, mass=mass, pos=pos, seen=seen, dev_err=c.err, shared=True)
    plain = torch.zeros_like(c.out)
    for _ in range(3):
        c.out.fill_(math.nan)
        handle.shared_attn(c.q, c.out, ints(c.starts), ints(c.prefix), lse=c.lse)
        c.check()
        handle.decode_attn(c.q, plain, mass_in=mass, mass_out=mass)
        assert float((plain - c.out).norm()) <= 1e-5 * float(plain.norm())
    total = mass.sum(dim=-1)
    assert torch.allclose(total, torch.full_like(total, 12.0), rtol=1e-4)
    assert int(c.err) == 0


def test_shared_wait_that_runs_out():
    """Failure detection: the wait is made to run out by the switch, the next call is right."""
    c = Shared([(512, [5, 30])], 2, 4, 16)
    try:
        ckv.paged_set_wait_limit(2_000_000, stall=True)
        c.run()
        torch.cuda.synchronize()
        assert int(c.err) == 1
    finally:
        ckv.paged_set_wait_limit()
    c.err.zero_()
    c.run()
    c.check()
    assert int(c.err) == 0


# ---------------------------------------------------------------- a batch's steps
def test_prompts_then_decode_steps_behind_a_prefix():
    """A prefix's rows, its samples' prompts, then decode steps, all through plan,
    append_rotated and shared_attn, against attention over rotated rows in 64 bits."""
    S, heads, g, page, width, prefix = 5, 2, 4, 16, 16, 64
    gen = torch.Generator().manual_seed(3)
    n_pages = S * width
    K, V = pools(n_pages, heads, page, "bf16", "phd", gen)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    zero = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
    lens, seen, held, granted, starts, err = zero(S), zero(S), zero(S), zero(S), zero(S + 1), zero(1)
    pos, mass = zero(S, heads, width * page), torch.zeros(S, heads, width * page, device="cuda")
    ring, span = torch.randperm(n_pages, generator=gen).int().cuda(), ints([0, n_pages])
    shared = zero(S)
    cache = ckv.PagedCache(K, V, table, lens, g=g, mass=mass, pos=pos, seen=seen, dev_err=err, shared=True)
    turns_host = ckv.rotary_turns(ckv.rotary_frequencies(128, 500000.0, "bands", 8.0, 8192, 1.0, 4.0)[0])
    turns = turns_host.cuda()
    ref = [([], []) for _ in range(S)]  # rotated keys (as stored) and values of each sequence

    def feed(counts):
        T = sum(counts)
        qkv = torch.randn(T, heads * (g + 2), D, generator=gen).to(torch.bfloat16).cuda()
        q, k, v = qkv[:, :heads * g], qkv[:, heads * g:heads * (g + 1)], qkv[:, heads * (g + 1):]
        slots, q_out = zero(max(T, 1), 4), torch.zeros(T, heads * g, D, dtype=torch.bfloat16, device="cuda")
        at = seen.tolist()
        cache.plan(ints(counts), held, ring, span, slots, starts, granted, shared=shared)
        cache.append_rotated(q, k, v, slots, turns, q_out)
        torch.cuda.synchronize()
        assert granted.tolist() == counts and int(err) == 0
        positions, t = [], 0
        for s, c in enumerate(counts):
            for j in range(c):
                positions.append(at[s] + j)
                r = int(slots[t, 0])
                ref[s][0].append(K[r // page, :, r % page].clone())
                ref[s][1].append(v[t])
                t += 1
        check_rows(q_out, q, positions, turns_host, 128, False, None, 0, 1.0, "bf16")
        check_rows(torch.stack([K[int(r) // page, :, int(r) % page] for r in slots[:, 0]]), k, positions, turns_host, 128,
                   False, None, 0, 1.0, "bf16")
        return q_out

    feed([prefix, 0, 0, 0, 0])
    # the others take over the first sequence's pages
    for s in range(1, S):
        table[s, :prefix // page] = table[0, :prefix // page]
        ref[s] = (list(ref[0][0]), list(ref[0][1]))
    pos[1:] = pos[:1]
    lens.fill_(prefix)
    seen.fill_(prefix)
    held.fill_(prefix // page)
    shared[1:] = prefix // page
    feed([3, 17, 0, 40, 16])
    group_starts, rows = ints([0, S]), ints([prefix])
    for step in range(20):
        q = feed([1] * S)
        out, lse = torch.zeros(S, heads * g, D, device="cuda"), torch.zeros(S, heads * g, device="cuda")
        cache.shared_attn(q, out, group_starts, rows, lse=lse)
        torch.cuda.synchronize()
        for s in range(S):
            k, v = (torch.stack(x).transpose(0, 1).double() for x in ref[s])
            logits = torch.matmul(q[s].double().view(heads, g, D), k.transpose(1, 2)) * D ** -0.5
            want = torch.matmul(torch.softmax(logits, dim=-1), v).view(heads * g, D)
            assert float((out[s].double() - want).norm() / want.norm()) < 1e-5
            assert pos[s, :, :int(lens[s])].tolist() == [list(range(len(ref[s][0])))] * heads
        if step == 10:  # one ends, hands its own pages back and starts anew behind the prefix
            lens[3] = seen[3] = prefix
            ref[3] = (ref[3][0][:prefix], ref[3][1][:prefix])
    # pages in hand and in the ring are all pages, each once
    mine = [p for s in range(S) for p in table[s, (prefix // page if s else 0):int(held[s])].tolist()]
    left = [int(ring[(int(span[0]) + i) % n_pages]) for i in range(int(span[1]))]
    assert sorted(mine + left) == list(range(n_pages))


def batch(seed, S=6, heads=2, g=4, page=16, width=12, prefix=96):
    """A batch behind a prefix, and its step as a function without host work between the calls."""
    gen = torch.Generator().manual_seed(seed)
    n_pages = S * width
    K, V = pools(n_pages, heads, page, "bf16", "hpd", gen)
    table = torch.full((S, width), -1, dtype=torch.int32)
    common = prefix // page
    table[:, :common] = torch.arange(common, dtype=torch.int32)
    x = dict(K=K, V=V, table=table.cuda(), lens=ints([prefix] * S), seen=ints([prefix] * S), held=ints([common] * S),
             ring=ints(list(range(common, n_pages))), span=ints([0, n_pages - common]), granted=ints([0] * S),
             starts=ints([0] * (S + 1)), counts=ints([1 + s % 3 for s in range(S)]), shared=ints([common] * S),
             groups=ints([0, S]), prefix=ints([prefix]), err=ints([0]))
    T = sum(1 + s % 3 for s in range(S))
    qkv = torch.randn(T, heads * (g + 2), D, generator=gen).to(torch.bfloat16).cuda()
    x.update(slots=ints([[0] * 4] * T), qkv=qkv, q_out=torch.zeros(T, heads * g, D, dtype=torch.bfloat16, device="cuda"),
             out=torch.zeros(S, heads * g, D, device="cuda"), lse=torch.zeros(S, heads * g, device="cuda"))
    turns = ckv.rotary_turns(ckv.rotary_frequencies(128)[0]).cuda()
    cache = ckv.PagedCache(K, V, x["table"], x["lens"], g=g, seen=x["seen"], dev_err=x["err"], shared=True)

    def step():
        q, k, v = qkv[:, :heads * g], qkv[:, heads * g:heads * (g + 1)], qkv[:, heads * (g + 1):]
        cache.plan(x["counts"], x["held"], x["ring"], x["span"], x["slots"], x["starts"], x["granted"], shared=x["shared"])
        cache.append_rotated(q, k, v, x["slots"], turns, x["q_out"])
        cache.shared_attn(x["q_out"][:S], x["out"], x["groups"], x["prefix"], lse=x["lse"])
        # the rows of the step go into the next one's, so that steps depend on one another
        qkv[:S, :heads * g].add_(x["out"].to(torch.bfloat16))

    return x, step


def test_steps_captured_and_side_by_side():
    """Two batches' steps replayed at once, on streams of their own, against the same steps called one by one."""
    alone = []
    for seed in (1, 2):
        x, step = batch(seed)
        for _ in range(12):
            step()
        torch.cuda.synchronize()
        alone.append(x)
    both, graphs = [], []
    for seed in (1, 2):
        x, step = batch(seed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            step()
        both.append((x, step))
        graphs.append((graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(12):
        for graph, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for x, (y, _) in zip(alone, both):
        assert int(x["err"]) == 0 and x["granted"].tolist() == [1 + s % 3 for s in range(6)]
        assert x["out"].isfinite().all()
        for name in x:
            assert torch.equal(x[name], y[name]), name


def test_offsets_above_32_bits():
    """Pools of 5 GB each, with the rows at their ends; token strides of 4 GB."""
    heads, g, page, n_pages, S, prefix = 8, 2, 128, 20000, 2, 128
    K, V = (torch.zeros(n_pages, heads, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(0)
    at = [19999, 19997, 16500]
    for pool in (K, V):
        pool[at] = torch.randn(3, heads, page, D, generator=gen).to(torch.bfloat16).cuda()
    table, lens, err = ints([[19999, 19997], [19999, 16500]]), ints([200, 133]), ints([0])
    cache = ckv.PagedCache(K, V, table, lens, g=g, dev_err=err, shared=True)
    q = torch.randn(S, heads * g, D, generator=gen).to(torch.bfloat16).cuda()
    out, want = (torch.zeros(S, heads * g, D, device="cuda") for _ in range(2))
    cache.shared_attn(q, out, ints([0, S]), ints([prefix]))
    for s in range(S):
        k, v = (x[table[s].long()].transpose(0, 1).reshape(heads, -1, D)[:, :int(lens[s])].double() for x in (K, V))
        p = torch.softmax(torch.matmul(q[s].double().view(heads, g, D), k.transpose(1, 2)) * D ** -0.5, dim=-1)
        want[s] = torch.matmul(p, v).view(heads * g, D).float()
    assert float((out - want).norm() / want.norm()) < 1e-5 and int(err) == 0
    del cache

    step = 2 ** 31
    wide = torch.empty(step + 4096, dtype=torch.bfloat16, device="cuda")
    q, o = (wide.as_strided((2, 4, D), (step, D, 1), x) for x in (0, 1024))
    rows = torch.randn(2, 4, D, generator=gen).to(torch.bfloat16).cuda()
    q.copy_(rows)
    turns = ckv.rotary_turns(ckv.rotary_frequencies(128)[0]).cuda()
    ckv.rotate(q, None, ints([5, 70000]), turns, o, None)
    check_rows(o, rows, [5, 70000], turns, 128, False, None, 0, 1.0, "bf16")
    cache = ckv.PagedCache(K, V, table, lens, g=1, dev_err=err)
    slots = ints([[19998 * page + 3, 0, 0, 9], [n_pages * page - 1, 1, 1, 8]])
    k = rows.repeat(1, 2, 1)
    cache.append_rotated(None, k, k, slots, turns, None)
    torch.cuda.synchronize()
    assert int(err) == 0
    check_rows(torch.stack([K[19998, :, 3], K[19999, :, 127]]), k, [9, 8], turns, 128, False, None, 0, 1.0, "bf16")
    assert torch.equal(V[19998, :, 3], k[0]) and torch.equal(V[19999, :, 127], k[1])


# ---------------------------------------------------------------- refusals of the handle
def test_refusals():
    c = Shared([(64, [1, 2])], 2, 4, 16)
    plain = ckv.PagedCache(c.K, c.V, c.table, c.lens, g=4)
    two, one = ints([0, 2]), ints([64])
    with pytest.raises(ValueError, match="shared=True"):
        plain.shared_attn(c.q, c.out, two, one)
    for args, error in (((c.q[:1], c.out, two, one), ValueError), ((c.q.float(), c.out, two, one), TypeError),
                        ((c.q, c.out.half(), two, one), TypeError), ((c.q, c.out, two.long(), one), TypeError),
                        ((c.q, c.out, one, one), ValueError), ((c.q, c.out, two, one[None]), ValueError),
                        ((c.q, c.out, two.cpu(), one), ValueError), ((c.q.cpu(), c.out, two, one), ValueError)):
        with pytest.raises(error):
            c.handle.shared_attn(*args)
    with pytest.raises(ckv.CKVError):  # more groups than sequences
        c.handle.shared_attn(c.q, c.out, ints([0, 1, 2, 2]), ints([0, 0, 0]))
    a = Append([0], [3], 2, 4)
    turns = ckv.rotary_turns([1.0] * 64).cuda()
    good = dict(q=a.q, k=a.k, v=a.v, slots=a.slots, turns=turns, q_out=a.q_out)
    for bad, error in ((dict(q=a.q.float()), TypeError), (dict(q_out=None), ValueError), (dict(k=a.k[:2]), ValueError),
                       (dict(slots=a.slots[:, :3]), ValueError), (dict(slots=a.slots.long()), TypeError),
                       (dict(turns=turns.double()), TypeError), (dict(turns=turns.cpu()), ValueError),
                       (dict(turns=turns[:3]), ckv.CKVError), (dict(v=a.v.transpose(1, 2)), ValueError),
                       (dict(q_weight=torch.ones(64, device="cuda")), ValueError),
                       (dict(k_weight=torch.ones(128, device="cuda", dtype=torch.bfloat16)), TypeError)):
        with pytest.raises(error):
            a.cache.append_rotated(**{**good, **bad})
    positions = ints([0, 1, 2])
    good = dict(q=a.q, k=a.k, positions=positions, turns=turns, q_out=a.q_out, k_out=torch.empty_like(a.k))
    for bad, error in ((dict(q=a.q.half()), TypeError), (dict(positions=positions.long()), TypeError),
                       (dict(positions=positions[:2]), ValueError), (dict(k=None), ValueError),
                       (dict(k=a.k.float()), TypeError), (dict(k_out=a.k.cpu()), ValueError)):
        with pytest.raises(error):
            ckv.rotate(**{**good, **bad})
    p = Plan([3, 4], [1, 1])
    with pytest.raises(TypeError):
        p.run(start=p.dev["start"].long())
    with pytest.raises(ValueError):
        p.run(shared=p.dev["shared"][:1])
    with pytest.raises(ckv.CKVError):  # granted is held_out
        p.run(held_out=p.granted)
