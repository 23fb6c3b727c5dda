"""The paged step's oracle (plans, rotary positions, groups) against hand
examples, torch and complex arithmetic; the frequencies' helper; and the
refusals of the entry points on the host (every error is found before a launch,
so no GPU is touched)."""
import ctypes
import fractions
import math

import numpy as np
import pytest
import torch

import oracle.batch as ob
from recallable_kv_cache_gb300 import build, ckv
from test_paged_oracle import ALIGN, ARG, BAD_CACHES, CAPACITY, DTYPE, P, i64, struct


# ---------------------------------------------------------------- oracle pins
def test_plan_by_hand():
    """Pages of 16: sequence 0 grows into a second page, 1 was cut to 5 rows and
    hands two pages back, 2 has ended but keeps its prefix's page, 3 wants more
    pages than are left, 4 fits its last page."""
    table = [[7, -1, -1, -1], [3, 4, 5, -1], [9, 8, -1, -1], [1, -1, -1, -1], [2, -1, -1, -1]]
    got = ob.plan(table, [2, 1, 0, 40, 1], [15, 5, 0, 10, 15], [100, 50, 0, 10, 15], [0, 0, 1, 0, 0], [1, 3, 2, 1, 1],
                  [-1, 20, 21, -1, -1, -1], [1, 2], 16, 46, 30)
    assert got["table"][0] == [7, 20, -1, -1] and got["table"][3] == [1, -1, -1, -1]
    assert got["held"] == [2, 1, 1, 1, 1] and got["granted"] == [2, 1, 0, 0, 1]
    assert got["span"] == [2, 4] and got["ring"] == [-1, 20, 21, 4, 5, 8]
    assert got["lens"] == [17, 6, 0, 10, 16] and got["seen"] == [102, 51, 0, 10, 16]
    assert got["starts"] == [0, 2, 3, 3, 43, 44]
    assert got["slots"][0] == [7 * 16 + 15, 0, 15, 100] and got["slots"][1] == [20 * 16, 0, 16, 101]
    assert got["slots"][2] == [3 * 16 + 5, 1, 5, 50] and got["slots"][43] == [2 * 16 + 15, 4, 15, 15]
    assert all(x == [-1] * 4 for x in got["slots"][3:43] + got["slots"][44:]) and not got["errors"]


def test_plan_conserves_pages():
    rng = np.random.default_rng(0)
    for _ in range(30):
        S, page, width, n = 7, 16, 6, 40
        perm = list(rng.permutation(n))
        held = rng.integers(0, width + 1, S)
        table, at = [], 0
        for h in held:
            table.append([int(x) for x in perm[at:at + h]] + [-1] * (width - h))
            at += h
        head, free = int(rng.integers(0, n)), n - at
        ring = [-1] * n
        for i, p in enumerate(perm[at:]):
            ring[(head + i) % n] = int(p)
        start = [int(rng.integers(0, h * page + 1)) for h in held]
        counts = [int(rng.integers(0, width * page - a + 1)) for a in start]
        got = ob.plan(table, counts, start, start, [0] * S, held, ring, [head, free], page, sum(counts), n)
        now = [p for row, h in zip(got["table"], got["held"]) for p in row[:h]]
        left = [got["ring"][(got["span"][0] + i) % n] for i in range(got["span"][1])]
        assert sorted(now + left) == list(range(n))
        slots = [x[0] for x in got["slots"] if x[0] >= 0]
        assert len(set(slots)) == len(slots) == sum(got["granted"])


def test_rotary_is_a_complex_product():
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=128), [10000.0 ** (-2 * i / 64) for i in range(32)]
    turns = [int(t) % 2 ** 64 for t in ckv.rotary_turns(w)]
    for p in (0, 1, -3, 517, 2 ** 31 - 1):
        z = np.exp(1j * np.array([math.fmod(float(fractions.Fraction(v) * p % (2 * ckv._PI)), 7) for v in w]))
        got = ob.rotary(x, p, turns, 64, True)
        want = (x[0:64:2] + 1j * x[1:64:2]) * z
        assert np.allclose(got[0:64:2] + 1j * got[1:64:2], want, atol=1e-9)
        assert np.array_equal(got[64:], x[64:])
        got = ob.rotary(x, p, turns, 64, False, amplitude=1.5)
        want = (x[:32] + 1j * x[32:64]) * z * 1.5
        assert np.allclose(got[:32] + 1j * got[32:64], want, atol=1e-9)


def test_rotary_norm_equals_torch():
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=128), rng.normal(size=128)
    want = torch.nn.functional.rms_norm(torch.tensor(x), (128,), torch.tensor(w), eps=1e-3)
    assert np.allclose(ob.rotary(x, 5, [], 0, False, w, 1e-3), want.numpy(), rtol=1e-12)


def test_groups_by_hand():
    assert ob.groups([0, 3, 4, 9], [100, 50, 40], [37, 0, 0, 0, 60, 0, 0, 0, 0], 9, 64) == [(0, 3, 32), (3, 4, 0), (4, 9, 32)]
    # a start below an earlier one, one past the end
    assert ob.groups([2, 5, 3, 99], [16, 16, 16], [16] * 6, 6, 64) == [(2, 5, 16), (5, 5, 0), (5, 6, 0)]


# ---------------------------------------------------------------- frequencies
def test_turns_are_exact():
    w = [1.0, 0.1, 1e-6, 2 * math.pi, 0.0, -0.5, 7.0]
    got = [int(x) for x in ckv.rotary_turns(w)]
    for t, x in zip(got, w):
        exact = fractions.Fraction(x) / (2 * ckv._PI) * 2 ** 64
        assert abs((t - exact + 2 ** 63) % 2 ** 64 - 2 ** 63) <= 1
    for bad in (math.nan, math.inf):
        with pytest.raises((ValueError, OverflowError)):
            ckv.rotary_turns([bad])


def test_frequency_scalings():
    plain, one = ckv.rotary_frequencies(128, 10000.0)
    assert one == 1.0 and plain[0] == 1.0 and abs(plain[32] - 0.01) < 1e-15
    linear, _ = ckv.rotary_frequencies(128, 10000.0, "linear", 4.0)
    assert all(abs(a - b / 4) < 1e-18 for a, b in zip(linear, plain))
    base, _ = ckv.rotary_frequencies(128, 10000.0, "base", 4.0)
    assert base[0] == 1.0 and abs(base[-1] / (plain[-1] / 4) - 1) < 1e-12
    bands, one = ckv.rotary_frequencies(128, 500000.0, "bands", 8.0, 8192, 1.0, 4.0)
    p5, _ = ckv.rotary_frequencies(128, 500000.0)
    for a, b in zip(bands, p5):
        turned = 8192 * b / (2 * math.pi)
        if turned > 4:
            assert a == b
        elif turned < 1:
            assert abs(a - b / 8) < 1e-18
        else:
            assert b / 8 < a < b
    assert one == 1.0
    ramp, amplitude = ckv.rotary_frequencies(128, 10000.0, "ramp", 16.0, 4096)
    assert abs(amplitude - (0.1 * math.log(16) + 1)) < 1e-15
    assert ramp[0] == plain[0] and abs(ramp[-1] - plain[-1] / 16) < 1e-18
    assert all(a >= b for a, b in zip(ramp, ramp[1:]))
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="x"),
                dict(rot=8, scaling="ramp", low=2.0, high=1.0)):
        with pytest.raises(ValueError):
            ckv.rotary_frequencies(**bad)


@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
@pytest.mark.parametrize("rot,base,original,low,high", [
    (128, 10000.0, 4096, 1.0, 32.0), (64, 10000.0, 32768, 1.0, 4.0), (128, 500000.0, 8192, 1.0, 4.0),
    (16, 1e6, 4096, 1.0, 32.0), (128, 1e6, 64, 0.25, 7.5),  # borders in front of the first pair
    (128, 10000.0, 10 ** 6, 1.0, 32.0), (128, 10000.0, 10 ** 6, 0.001, 32.0), (64, 10.0, 10 ** 6, 1.0, 32.0),  # behind the last
])
def test_every_pair_of_the_scalings(rot, base, factor, original, low, high):
    """Both published formulas: by wavelengths, and by the pair whose wavelength fits
    the original length a number of times."""
    theta = np.float64(base) ** (-np.arange(0, rot, 2) / rot)
    wavelength = 2 * np.pi / theta

    # bands: wavelengths below original / high stay, above original / low are divided
    smooth = (original / wavelength - low) / (high - low)
    want = np.where(wavelength < original / high, theta,
                    np.where(wavelength > original / low, theta / factor, (1 - smooth) * theta / factor + smooth * theta))
    got, amplitude = ckv.rotary_frequencies(rot, base, "bands", factor, original, low, high)
    assert amplitude == 1.0 and np.allclose(got, want, rtol=1e-12, atol=0)

    # ramp: d ln(L / (2 pi n)) / (2 ln base) for the borders, whole and inside [0, d - 1]
    border = lambda n: rot * np.log(original / (n * 2 * np.pi)) / (2 * np.log(base))
    first, last = max(np.floor(border(high)), 0), min(np.ceil(border(low)), rot - 1)
    if first == last:
        last += 0.001
    extrapolated = 1 - np.clip((np.arange(rot // 2) - first) / (last - first), 0, 1)
    if first > last:  # the formula has no ramp here: every pair turns more than `high` times, and stays
        assert (original / wavelength > high).all()
        extrapolated = 1.0
    want = theta / factor * (1 - extrapolated) + theta * extrapolated
    got, amplitude = ckv.rotary_frequencies(rot, base, "ramp", factor, original, low, high)
    assert abs(amplitude - (0.1 * np.log(factor) + 1)) < 1e-12 and np.allclose(got, want, rtol=1e-12, atol=0)


def test_usual_borders_of_the_scalings():
    """A ramp ends at 32 turns where nothing is said, bands at 4."""
    for scaling, high in (("ramp", 32.0), ("bands", 4.0)):
        args = (128, 500000.0, scaling, 8.0, 8192)
        assert ckv.rotary_frequencies(*args) == ckv.rotary_frequencies(*args, low=1.0, high=high)
        assert ckv.rotary_frequencies(*args) != ckv.rotary_frequencies(*args, low=1.0, high=36.0 - high)
    with pytest.raises(ValueError):
        ckv.rotary_frequencies(128, scaling="bands", factor=8.0, low=4.0)


# ---------------------------------------------------------------- refusals of the C ABI
@pytest.fixture(scope="module")
def lib():
    build.build()
    return ckv.lib()


STEP = 1 << 24  # between the addresses of the arrays, none of which is read


def rot(**kw):
    base = dict(turns=P, q_weight=None, k_weight=P, eps=1e-6, amplitude=1.0, rot=128, interleaved=0)
    base.update(kw)
    return ckv.Rotary(*[base[n] for n, _ in ckv.Rotary._fields_])


def plan(lib, c, **kw):
    names = ["counts", "start", "first", "shared", "held_in", "held_out", "ring", "cap", "span_in", "span_out", "granted",
             "starts", "slots", "n_slots"]
    base = {n: P + (20 + i) * STEP for i, n in enumerate(names)}
    base.update(start=None, first=None, shared=None, cap=64, n_slots=8)
    base.update(kw)
    return lib.ckv_paged_plan(ctypes.addressof(c), *[base[n] for n in names], None)


def apart(**kw):
    """A cache whose arrays are apart from one another."""
    return struct(**{**dict(table=P + STEP, lens=P + 2 * STEP, seen=P + 3 * STEP, mass=P + 4 * STEP, pos=P + 5 * STEP), **kw})


def rotate(lib, r, **kw):
    names = ["q", "q_stride", "q_out", "q_out_stride", "heads_q", "k", "k_stride", "k_out", "k_out_stride", "heads_k",
             "positions", "tokens", "d", "dtype"]
    st = i64(1024, 128)
    base = dict(q=P, q_stride=st, q_out=P, q_out_stride=st, heads_q=8, k=P, k_stride=st, k_out=P, k_out_stride=st,
                heads_k=8, positions=P, tokens=5, d=128, dtype=ckv.BF16)
    base.update(kw)
    return lib.ckv_rotate(None if r is None else ctypes.addressof(r), *[base[n] for n in names], None)


def append(lib, c, r, **kw):
    names = ["q", "q_stride", "g", "q_out", "q_out_stride", "k", "k_stride", "v", "v_stride", "slots", "tokens"]
    st = i64(1024, 128)
    base = dict(q=P, q_stride=st, g=4, q_out=P, q_out_stride=st, k=P, k_stride=st, v=P, v_stride=st, slots=P, tokens=5)
    base.update(kw)
    return lib.ckv_paged_append_rotated(ctypes.addressof(c), None if r is None else ctypes.addressof(r),
                                        *[base[n] for n in names], None)


def shared(lib, c, **kw):
    names = ["q", "q_dtype", "q_stride", "g", "scale", "group_starts", "prefix", "groups", "out", "lse", "workspace", "bytes"]
    base = dict(q=P, q_dtype=c.kv_dtype, q_stride=i64(1024, 128), g=4, scale=0.1, group_starts=P, prefix=P, groups=2, out=P,
                lse=P, workspace=P, bytes=1 << 40)
    base.update(kw)
    return lib.ckv_paged_shared_attn(ctypes.addressof(c), *[base[n] for n in names], None)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad, code):
    c = struct(**bad)
    n = ctypes.c_int64()
    assert plan(lib, c) == code
    assert append(lib, c, rot()) == code
    assert shared(lib, c) == code
    assert lib.ckv_paged_shared_workspace(ctypes.addressof(c), 4, ctypes.byref(n)) == code


@pytest.mark.parametrize("bad,code", [
    (dict(counts=None), ARG), (dict(held_in=None), ARG), (dict(held_out=None), ARG), (dict(ring=None), ARG),
    (dict(span_in=None), ARG), (dict(span_out=None), ARG), (dict(granted=None), ARG), (dict(starts=None), ARG),
    (dict(slots=None), ARG), (dict(cap=0), ARG), (dict(n_slots=0), ARG), (dict(n_slots=2 ** 31 - 1), ARG),
    (dict(slots=P + 8), ALIGN),
    # overlaps: an output with another output, with an input that is not its own pair, or in part
    (dict(granted=P + 2 * STEP), ARG), (dict(starts=P + 3 * STEP + 8), ARG), (dict(held_out=P + 2 * STEP), ARG),
    (dict(start=P + 2 * STEP + 4), ARG), (dict(first=P + 3 * STEP - 4), ARG), (dict(ring=P + STEP), ARG),
    (dict(shared=P + 25 * STEP), ARG), (dict(held_in=P + 25 * STEP + 4), ARG), (dict(span_in=P + 29 * STEP + 4), ARG),
])
def test_bad_plans_are_refused(lib, bad, code):
    assert plan(lib, apart(), **bad) == code


def test_plan_from_the_longest_ring_is_refused(lib):
    assert plan(lib, apart(), cap=2 ** 31 - 1, ring=P + 64 * STEP) == ARG


def test_plan_of_too_many_slots_is_refused(lib):
    assert plan(lib, apart(n_pages=1 << 26)) == ARG
    assert append(lib, apart(n_pages=1 << 26), rot()) == ARG


BAD_ROTARY = [dict(turns=None), dict(rot=8), dict(rot=-16), dict(rot=144), dict(rot=120), dict(eps=-1.0),
              dict(eps=math.inf), dict(eps=math.nan), dict(amplitude=math.inf), dict(amplitude=math.nan),
              dict(interleaved=2)]


@pytest.mark.parametrize("bad", BAD_ROTARY)
def test_bad_rotaries_are_refused(lib, bad):
    assert rotate(lib, rot(**bad)) == ARG
    assert append(lib, apart(), rot(**bad)) == ARG


@pytest.mark.parametrize("bad", [dict(turns=P + 8), dict(q_weight=P + 4), dict(k_weight=P + 8)])
def test_misaligned_rotaries_are_refused(lib, bad):
    assert rotate(lib, rot(**bad)) == ALIGN
    assert append(lib, apart(), rot(**bad)) == ALIGN


def test_null_rotary_is_refused(lib):
    assert rotate(lib, None) == ARG and append(lib, apart(), None) == ARG


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), ARG), (dict(k_out=None), ARG), (dict(q_stride=None), ARG), (dict(positions=None), ARG),
    (dict(tokens=0), ARG), (dict(d=64), ARG), (dict(dtype=2), DTYPE), (dict(heads_q=-1), ARG),
    (dict(heads_q=0, heads_k=0), ARG), (dict(tokens=1 << 28), ARG), (dict(q=P + 8), ALIGN), (dict(k_out=P + 4), ALIGN),
    (dict(q_stride=i64(-1024, 128)), ARG), (dict(q_out_stride=i64(1024, 64)), ARG), (dict(q_out_stride=i64(0, 128)), ARG),
    (dict(k_stride=i64(1028, 128)), ALIGN), (dict(k_stride=i64(1 << 38, 128)), ARG),
    (dict(q_stride=i64(2048, 128)), ARG),  # in place with other strides
])
def test_bad_rotations_are_refused(lib, bad, code):
    assert rotate(lib, rot(), **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), ARG), (dict(q_out=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG),
    (dict(tokens=0), ARG), (dict(g=-1), ARG), (dict(g=1 << 30), ARG), (dict(tokens=1 << 28), ARG),
    (dict(slots=P + 4), ALIGN), (dict(k=P + 8), ALIGN), (dict(v_stride=i64(1, 128)), ALIGN),
    (dict(q_out_stride=i64(1024, 0)), ARG), (dict(q_stride=i64(2048, 128)), ARG),
])
def test_bad_appends_are_refused(lib, bad, code):
    assert append(lib, apart(), rot(), **bad) == code


FAR = dict(q=P, k=P + STEP, q_out=P + 2 * STEP, k_out=P + 3 * STEP, positions=P + 4 * STEP)
ROW = 256  # bytes of a bf16 row


@pytest.mark.parametrize("bad", [
    # rows of an output on one another: equal strides, a token's rows into the next one's, a lattice that meets
    dict(q_out_stride=i64(128, 128)), dict(k_out_stride=i64(256, 128)), dict(q_out_stride=i64(128, 256)),
    dict(q_out_stride=i64(384, 256)), dict(q_out_stride=i64(1000, 128)), dict(q_out_stride=i64(128, 632)),
    # one output on the other, or on an input in part or of the other kind
    dict(k_out=P + 2 * STEP), dict(k_out=P + 2 * STEP + 7 * ROW), dict(q_out=P + 16), dict(q_out=P - 16), dict(q_out=P + ROW),
    dict(q_out=P + STEP), dict(k_out=P + STEP + 1024 * 2), dict(k_out=P), dict(q=P + STEP, q_out=P + STEP),
    dict(q_out=P, q_out_stride=i64(1024, 128), heads_q=9, q_stride=i64(1024, 128)),
    # an output on the positions, the turns or a weight
    dict(positions=P + 2 * STEP + 1024 * 2 - 4), dict(positions=P + 3 * STEP + 512), dict(q_out=P + 6 * STEP - 16),
    dict(k_out=P + 7 * STEP + 496),
])
def test_rotations_onto_themselves_are_refused(lib, bad):
    assert rotate(lib, rot(turns=P + 6 * STEP, k_weight=P + 7 * STEP), **{**FAR, **bad}) == ARG


@pytest.mark.parametrize("bad", [
    dict(q_out_stride=i64(128, 128)), dict(q_out_stride=i64(1024, 1024)), dict(q_out=P + 16), dict(q_out=P + STEP),
    dict(q_out=P + 2 * STEP + ROW), dict(slots=P + 3 * STEP + 7 * ROW), dict(q_out=P + 6 * STEP),
])
def test_appends_onto_their_inputs_are_refused(lib, bad):
    good = dict(q=P, k=P + STEP, v=P + 2 * STEP, q_out=P + 3 * STEP, slots=P + 4 * STEP)
    assert append(lib, apart(), rot(turns=P + 6 * STEP), **{**good, **bad}) == ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up, and what is not refused is launched")
def test_overlaps_equal_row_by_row(lib):
    """Small layouts of every kind, refused just where two rows, taken byte by byte, overlap."""
    rng = np.random.default_rng(0)
    seen = {True: 0, False: 0}
    for i in range(6000):
        tokens, hq, hk = (int(x) for x in rng.integers(1, 5, 3))
        step = lambda lo: 8 * int(rng.choice([16, 17, 24, 32, 33, 40, 48, 64, 80, 96, 112, 128, 160, 200, 256, 320, 384]
                                             + ([0, 1, 8] if lo == 0 else [])))
        pick = lambda lo: (step(lo), step(lo))
        if i % 3 == 0:  # parts of one tensor, as a projection leaves them
            all_heads = 2 * (hq + hk)
            st = {n: (128 * all_heads, 128) for n in ("q", "k", "q_out", "k_out")}
            at = {n: 256 * int(rng.integers(0, all_heads)) for n in st}
        else:
            st = {n: pick(0 if n in "qk" else 1) for n in ("q", "k", "q_out", "k_out")}
            at = {n: 16 * int(rng.integers(0, 400)) for n in st}
        for n in "qk":
            if rng.random() < 0.4:
                at[n + "_out"], st[n + "_out"] = at[n], st[n]
        heads = dict(q=hq, k=hk, q_out=hq, k_out=hk)
        rows = {n: [at[n] + 2 * (t * st[n][0] * (tokens > 1) + h * st[n][1] * (heads[n] > 1))
                    for t in range(tokens) for h in range(heads[n])] for n in st}
        legal = all(st[n][d] >= 128 or e == 1 for n in ("q_out", "k_out") for d, e in ((0, tokens), (1, heads[n])))
        meet = lambda x, y, same=False: any(abs(a - b) < 256 for i, a in enumerate(rows[x]) for j, b in enumerate(rows[y])
                                            if not (same and i == j))
        bad = not legal
        for n, other in (("q", "k"), ("k", "q")):
            bad |= meet(n + "_out", n + "_out", True) or meet(n + "_out", other + "_out") or meet(n + "_out", other)
            bad |= rows[n] != rows[n + "_out"] and meet(n, n + "_out")
        code = rotate(lib, rot(turns=P + 6 * STEP, k_weight=P + 7 * STEP), heads_q=hq, heads_k=hk, tokens=tokens,
                      positions=P + 8 * STEP, **{n: P + at[n] for n in st}, **{n + "_stride": i64(*st[n]) for n in st})
        assert (code == ARG) == bad, (tokens, heads, st, at, code)
        seen[bad] += 1
    assert min(seen.values()) > 500


@pytest.mark.parametrize("dtype", [ckv.BF16, ckv.F32])
@pytest.mark.parametrize("bad,code", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(q_stride=None), ARG), (dict(workspace=None), ARG),
    (dict(g=0), ARG), (dict(g=17), ARG), (dict(groups=-1), ARG), (dict(groups=4), ARG), (dict(group_starts=None), ARG),
    (dict(prefix=None), ARG), (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG), (dict(scale=3e38), ARG),
    (dict(bytes=1000), CAPACITY), (dict(q_dtype=2), DTYPE), (dict(q=P + 4), ALIGN), (dict(out=P + 4), ALIGN),
    (dict(workspace=P + 16), ALIGN), (dict(q_stride=i64(-1, 128)), ARG), (dict(q_stride=i64(1026, 128)), ALIGN),
])
def test_bad_shared_attention_is_refused(lib, bad, code, dtype):
    c = apart(kv_dtype=dtype)
    if "q_dtype" in bad:
        bad = dict(q_dtype=1 - dtype)
    assert shared(lib, c, **bad) == code


def test_shared_workspace(lib):
    c = apart()
    r, n, m = ctypes.addressof(c), ctypes.c_int64(), ctypes.c_int64()
    for g, code in ((0, ARG), (17, ARG), (4, 0)):
        assert lib.ckv_paged_shared_workspace(r, g, ctypes.byref(n)) == code
    assert lib.ckv_paged_shared_workspace(r, 4, None) == ARG
    assert lib.ckv_paged_attn_workspace(r, 4, 0, ctypes.byref(m)) == 0 and n.value > m.value
    assert shared(lib, c, bytes=n.value - 1) == CAPACITY


def test_rows_off_the_gpu_are_refused():
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        ckv.rotate(x, x, torch.zeros(4, dtype=torch.int32), None, x, x)
    with pytest.raises(ValueError, match="must be given"):
        ckv.rotate(None, None, None, None, None, None)
