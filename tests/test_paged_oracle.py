"""The paged cache's oracle against hand examples and torch, and the refusals
of its entry points on the host (no GPU is touched: every error below is found
before a launch)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import oracle.paged as po
from recallable_kv_cache_gb300 import build, ckv

ARG, DTYPE, CAPACITY, ALIGN = -1, -2, -3, -8


# ---------------------------------------------------------------- oracle pins
def test_rows_follow_the_page_table():
    pool = np.arange(4 * 2 * 16 * 3, dtype=np.float64).reshape(4, 2, 16, 3)
    got, ok = po.rows(pool, np.array([2, 0, 9]), 1, 40, 4)
    assert ok.tolist() == [True] * 32 + [False] * 8
    assert np.array_equal(got[:16], pool[2, 1]) and np.array_equal(got[16:32], pool[0, 1])
    assert not got[32:].any()


def test_attention_equals_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 8)), rng.normal(size=(20, 8)), rng.normal(size=(20, 8))
    ok = np.ones(20, dtype=bool)
    ok[5] = False
    out, lse, w = po.attend(q, k, v, ok, 0.3)
    t = [torch.tensor(x) for x in (q, k[ok], v[ok])]
    want = torch.nn.functional.scaled_dot_product_attention(t[0], t[1], t[2], scale=0.3)
    assert np.allclose(out, want.numpy(), rtol=1e-12)
    assert np.allclose(lse, torch.logsumexp(0.3 * t[0] @ t[1].T, dim=1).numpy(), rtol=1e-12)
    assert w[5] == 0 and abs(w.sum() - 3) < 1e-12


def test_attention_of_no_rows():
    out, lse, w = po.attend(np.ones((2, 4)), np.zeros((0, 4)), np.zeros((0, 4)), np.zeros(0, dtype=bool), 1.0)
    assert not out.any() and np.isneginf(lse).all() and len(w) == 0


def test_eviction_by_hand():
    #       sink  0.5  0.9  0.5  nan  0.1 recent
    mass = np.array([0.0, 0.5, 0.9, 0.5, np.nan, 0.1, 0.0])
    pos = np.array([0, 1, 2, 3, 4, 5, 6])
    kept = po.keep(mass, pos, 7, 4, 1, 1)
    assert kept.tolist() == [True, True, True, False, False, False, True]
    assert po.moves(kept, 4).tolist() == [[6, 3]]
    assert po.keep(mass, pos, 7, 7, 1, 1).all()
    assert po.moves(po.keep(mass, pos, 7, 7, 1, 1), 7).shape == (0, 2)


def test_eviction_is_the_best_set_of_its_size():
    rng = np.random.default_rng(1)
    for _ in range(20):
        n, budget = 7, 4
        mass, pos = rng.integers(0, 4, n).astype(float), rng.permutation(n)
        kept = po.keep(mass, pos, n, budget, 1, 1)
        safe = (pos < 1) | (pos >= n - 1)
        assert kept.sum() == budget and kept[safe].all()
        best = max(sum(mass[list(c)]) for c in itertools.combinations(range(n), budget)
                   if set(np.flatnonzero(safe)) <= set(c))
        assert mass[kept].sum() == best


# ---------------------------------------------------------------- refusals of the C ABI
@pytest.fixture(scope="module")
def lib():
    build.build()
    return ckv.lib()


P = 1 << 20  # an aligned address that is never read: the calls below end on the host


def struct(**kw):
    base = dict(K=P, V=P, k_stride=(2 * 64 * 128, 64 * 128, 128), v_stride=(2 * 64 * 128, 64 * 128, 128), table=P,
                lens=P, mass=P, pos=P, seen=P, dev_err=None, n_pages=5, heads=2, page_size=64, seqs=3, max_pages=4,
                d=128, kv_dtype=ckv.BF16)
    base.update(kw)
    base["k_stride"] = (ctypes.c_int64 * 3)(*base["k_stride"])
    base["v_stride"] = (ctypes.c_int64 * 3)(*base["v_stride"])
    return ckv.PagedCacheStruct(*[base[n] for n, _ in ckv.PagedCacheStruct._fields_])


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


BAD_CACHES = [
    (dict(K=None), ARG), (dict(V=None), ARG), (dict(table=None), ARG), (dict(lens=None), ARG), (dict(d=64), ARG),
    (dict(kv_dtype=2), DTYPE), (dict(n_pages=0), ARG), (dict(heads=0), ARG), (dict(seqs=0), ARG),
    (dict(max_pages=0), ARG), (dict(page_size=0), ARG), (dict(page_size=24), ARG), (dict(page_size=-16), ARG),
    (dict(max_pages=1 << 25), ARG), (dict(seqs=1 << 30, heads=2), ARG), (dict(K=P + 8), ALIGN), (dict(V=P + 2), ALIGN),
    (dict(k_stride=(16384, 8192, 127)), ARG), (dict(k_stride=(0, 8192, 128)), ARG),
    (dict(v_stride=(16384, -8192, 128)), ARG), (dict(k_stride=(16384, 8192, 132)), ALIGN),
    (dict(v_stride=(16388, 8192, 128)), ALIGN), (dict(seen=None), ARG), (dict(mass=P + 4), ALIGN),
    (dict(pos=P + 8), ALIGN),
]


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad, code):
    c = struct(**bad)
    r = ctypes.addressof(c)
    n = ctypes.c_int64()
    assert lib.ckv_paged_attn_workspace(r, 4, 0, ctypes.byref(n)) == code
    assert lib.ckv_paged_append(r, P, P, i64(128, 128, 128), i64(128, 128, 128), 1, None, None, None, None) == code
    assert lib.ckv_paged_decode_attn(r, P, c.kv_dtype, i64(1024, 128), 4, 0.1, P, P, None, None, P, 1 << 40,
                                     None) == code
    assert lib.ckv_paged_evict_select(r, 64, 16, 16, 64, P, P, None) == code
    assert lib.ckv_paged_evict_apply(r, 64, 64, P, P, None) == code


def test_strides_of_single_extents_do_not_matter(lib):
    c = struct(n_pages=1, heads=1, k_stride=(0, 0, 128), v_stride=(3, -5, 128))
    n = ctypes.c_int64()
    assert lib.ckv_paged_attn_workspace(ctypes.addressof(c), 4, 0, ctypes.byref(n)) == 0 and n.value > 0


def test_append_refusals(lib):
    c = struct()
    r = ctypes.addressof(c)
    st = i64(128, 128, 128)

    def call(k=P, v=P, ks=st, vs=st, n=1):
        return lib.ckv_paged_append(r, k, v, ks, vs, n, None, None, None, None)

    assert call(k=None) == ARG and call(v=None) == ARG and call(ks=None) == ARG and call(vs=None) == ARG
    assert call(n=0) == ARG and call(n=-1) == ARG
    assert call(ks=i64(-128, 128, 128)) == ARG and call(vs=i64(128, 128, 1 << 40)) == ARG
    assert call(k=P + 4) == ALIGN and call(vs=i64(128, 130, 128)) == ALIGN
    assert lib.ckv_paged_append(None, P, P, st, st, 1, None, None, None, None) == ARG


def test_append_refuses_arrays_that_overlap_in_part(lib):
    """counts, start and first against lens and seen, and these two: the blocks
    of other sequences would read what one of them writes."""
    far = 1 << 24
    for at in (4, 8, -4, -8):  # three sequences: twelve bytes
        c = struct(lens=far, seen=2 * far)
        r = ctypes.addressof(c)
        for x in (far + at, 2 * far + at):
            for args in ((x, None, None), (None, x, None), (None, None, x), (x, 4 * far, 5 * far)):
                assert lib.ckv_paged_append(r, P, P, i64(128, 128, 128), i64(128, 128, 128), 1, *args, None) == ARG
        c = struct(lens=far, seen=far + at)
        assert lib.ckv_paged_append(ctypes.addressof(c), P, P, i64(128, 128, 128), i64(128, 128, 128), 1, None, None,
                                    None, None) == ARG


def test_attention_refusals(lib):
    c = struct()
    r = ctypes.addressof(c)

    def call(q=P, dtype=ckv.BF16, qs=i64(1024, 128), g=4, scale=0.1, out=P, mass_in=None, mass_out=None, ws=P,
             nbytes=1 << 40):
        return lib.ckv_paged_decode_attn(r, q, dtype, qs, g, scale, out, P, mass_in, mass_out, ws, nbytes, None)

    assert call(q=None) == ARG and call(qs=None) == ARG and call(out=None) == ARG and call(ws=None) == ARG
    assert call(dtype=ckv.F32) == DTYPE and call(dtype=9) == DTYPE
    assert call(g=0) == ARG and call(g=17) == ARG and call(g=-1) == ARG
    assert call(scale=float("nan")) == ARG and call(scale=float("inf")) == ARG
    assert call(mass_in=P) == ARG and call(mass_out=P + 4) == ALIGN and call(mass_in=P + 8, mass_out=P) == ALIGN
    assert call(qs=i64(-8, 128)) == ARG and call(qs=i64(1024, 129)) == ALIGN
    assert call(q=P + 2) == ALIGN and call(out=P + 4) == ALIGN and call(ws=P + 128) == ALIGN
    n, m = ctypes.c_int64(), ctypes.c_int64()
    assert lib.ckv_paged_attn_workspace(r, 4, 0, ctypes.byref(n)) == 0
    assert lib.ckv_paged_attn_workspace(r, 4, 1, ctypes.byref(m)) == 0
    assert m.value > n.value
    assert call(nbytes=n.value - 1) == CAPACITY
    assert call(mass_out=P, nbytes=m.value - 1) == CAPACITY
    for g in (0, 17):
        assert lib.ckv_paged_attn_workspace(r, g, 0, ctypes.byref(n)) == ARG
    assert lib.ckv_paged_attn_workspace(r, 4, 0, None) == ARG


def test_eviction_refusals(lib):
    c = struct()  # R = 256
    r = ctypes.addressof(c)

    def select(budget=64, sinks=16, recent=16, most=64, moves=P, n=P, ref=r):
        return lib.ckv_paged_evict_select(ref, budget, sinks, recent, most, moves, n, None)

    def apply(budget=64, most=64, moves=P, n=P, ref=r):
        return lib.ckv_paged_evict_apply(ref, budget, most, moves, n, None)

    for call in (select, apply):
        assert call(budget=0) == ARG and call(budget=-1) == ARG and call(moves=None) == ARG and call(n=None) == ARG
        assert call(most=-1) == ARG and call(most=63) == CAPACITY and call(budget=200, most=55) == CAPACITY
        assert call(moves=P + 4) == ALIGN
    assert select(sinks=-1) == ARG and select(recent=-1) == ARG and select(sinks=40, recent=25) == ARG
    assert select(sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == ARG
    for missing in ("mass", "pos"):
        c2 = struct(**{missing: None})
        assert select(ref=ctypes.addressof(c2)) == ARG


@pytest.mark.parametrize("most", [2 ** 30 + 1, 2 ** 31 - 1])
def test_eviction_refuses_more_moves_than_words_are_counted(lib, most):
    c = struct()
    r = ctypes.addressof(c)
    assert lib.ckv_paged_evict_select(r, 64, 16, 16, most, P, P, None) == ARG
    assert lib.ckv_paged_evict_apply(r, 64, most, P, P, None) == ARG


@pytest.mark.parametrize("scale", [3e38, -2.4e38])
def test_attention_refuses_scales_whose_base_2_form_is_infinite(lib, scale):
    c = struct()
    assert lib.ckv_paged_decode_attn(ctypes.addressof(c), P, ckv.BF16, i64(1024, 128), 4, scale, P, P, None, None, P,
                                     1 << 40, None) == ARG


def test_attention_refuses_weights_that_overlap_in_part(lib):
    """A row's old weight would be read after another row's new one is written."""
    c = struct()  # 3 * 2 * 256 weights
    far = 1 << 24
    for at in (16, 1024, 4 * 1536 - 16):
        for x, y in ((far, far + at), (far + at, far)):
            assert lib.ckv_paged_decode_attn(ctypes.addressof(c), P, ckv.BF16, i64(1024, 128), 4, 0.1, P, P, x, y, P,
                                             1 << 40, None) == ARG


def test_wait_limit_refusals(lib):
    for cycles, stall in ((0, 0), (-1, 0), (4_000_000_001, 0), (1000, 2), (1000, -1)):
        assert lib.ckv_paged_set_wait_limit(cycles, stall) == ARG
    assert lib.ckv_paged_set_wait_limit(2_000_000_000, 0) == 0


def test_struct_matches_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ckv.h")).read()
    body = [b for b in re.findall(r"typedef struct \{(.*?)\} (\w+);", src, flags=re.S) if b[1] == "ckv_paged_cache"]
    fields = re.findall(r"[\s*](\w+)(?:\[3\])?;", body[0][0])
    assert fields == [f for f, _ in ckv.PagedCacheStruct._fields_]


# ---------------------------------------------------------------- refusals of the binding
def tensors(**kw):
    K = torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16)
    t = dict(K=K, V=K.clone(), table=torch.zeros(3, 4, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32),
             g=4, mass=torch.zeros(3, 2, 64), pos=torch.zeros(3, 2, 64, dtype=torch.int32),
             seen=torch.zeros(3, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("bad,exc", [
    (dict(K=torch.zeros(5, 16, 128, dtype=torch.bfloat16)), ValueError),
    (dict(V=torch.zeros(5, 2, 16, 128)), ValueError),
    (dict(K=torch.zeros(5, 2, 16, 128, dtype=torch.float16), V=torch.zeros(5, 2, 16, 128, dtype=torch.float16)), TypeError),
    (dict(K=torch.zeros(5, 2, 128, 16, dtype=torch.bfloat16).transpose(2, 3)), ValueError),
    (dict(table=torch.zeros(3, 4, dtype=torch.int64)), TypeError),
    (dict(table=torch.zeros(12, dtype=torch.int32)), ValueError),
    (dict(lens=torch.zeros(4, dtype=torch.int32)), ValueError),
    (dict(lens=torch.zeros(6, dtype=torch.int32)[::2]), ValueError),
    (dict(mass=torch.zeros(3, 2, 63)), ValueError),
    (dict(mass=torch.zeros(3, 2, 64, dtype=torch.float64)), TypeError),
    (dict(pos=torch.zeros(3, 2, 64)), TypeError),
    (dict(seen=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(dev_err=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(), ValueError),  # everything right, but not on a GPU
])
def test_handle_refuses_wrong_tensors(bad, exc):
    with pytest.raises(exc):
        ckv.PagedCache(**tensors(**bad))


def test_workspace_is_recorded_once_on_every_other_stream():
    """The allocator learns of each stream the workspace is used on, before the
    launch, but not of one that is capturing (nothing runs there)."""
    import contextlib
    log, capturing = [], []

    class Cuda:
        ExternalStream = staticmethod(lambda raw, device: raw)

        @staticmethod
        @contextlib.contextmanager
        def stream(raw):
            log.append(("on", raw))
            yield

        is_current_stream_capturing = staticmethod(lambda: log[-1][1] in capturing)

    class Workspace:
        record_stream = staticmethod(lambda raw: log.append(("record", raw)))

    h = ckv.PagedCache.__new__(ckv.PagedCache)
    h.device, h._index, h._ref, h._cuda, h.workspace, h._streams = "cuda:0", 0, None, Cuda, Workspace, {5}
    h._raw_stream, h._current = (lambda i: 5), (lambda: 0)
    h._attn, h._append = (lambda *a: log.append(("attn", a[-1])) or 0), (lambda *a: 0)
    h._call(h._attn, None)
    assert log == [("attn", 5)]
    h._call(h._append, 9)
    assert log == [("attn", 5)]  # it does not use the workspace
    h._call(h._attn, 9)
    h._call(h._attn, 9)
    assert log[1:] == [("on", 9), ("record", 9), ("attn", 9), ("attn", 9)]
    capturing.append(7)
    h._call(h._attn, 7)
    assert log[5:] == [("on", 7), ("attn", 7)]
    capturing.clear()
    h._call(h._attn, 7)
    assert log[7:] == [("on", 7), ("record", 7), ("attn", 7)]


def test_workspace_is_recorded_on_the_default_stream():
    """Its address is 0, for which torch would make a stream of its own."""
    import contextlib
    log = []

    class Cuda:
        default_stream = staticmethod(lambda device: ("default", device))
        stream = staticmethod(lambda st: contextlib.nullcontext())
        is_current_stream_capturing = staticmethod(lambda: False)

        @staticmethod
        def ExternalStream(raw, device):
            assert raw

    class Workspace:
        record_stream = staticmethod(log.append)

    h = ckv.PagedCache.__new__(ckv.PagedCache)
    h.device, h._cuda, h.workspace, h._streams = "cuda:0", Cuda, Workspace, {5}
    h._note_stream(0)
    assert log == [("default", "cuda:0")] and h._streams == {0, 5}


def test_raw_calls_have_public_stand_ins():
    from types import SimpleNamespace as NS
    cuda = NS(current_stream=lambda i: NS(cuda_stream=100 + i), current_device=lambda: 2)
    stream, device = ckv._raw_calls(NS(_C=NS(), cuda=cuda))
    assert stream(1) == 101 and device() == 2
    own = NS(_cuda_getCurrentRawStream=lambda i: 7, _cuda_getDevice=lambda: 3)
    stream, device = ckv._raw_calls(NS(_C=own, cuda=cuda))
    assert stream(1) == 7 and device() == 3
