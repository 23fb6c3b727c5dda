"""Thin ctypes binding of libckv.so (the C ABI declared in include/ckv.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the cudaStream_t, and a non-zero ckv_status becomes CKVError.
Every step of the path runs in the library's CUDA kernels; there is no CPU
fallback, and the library is loaded on first use (RuntimeError if it has not
been built).
"""
from __future__ import annotations

import ctypes
import fractions
import math
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libckv.so")

F32, BF16 = 0, 1
# pi to 50 decimals
_PI = fractions.Fraction("3.14159265358979323846264338327950288419716939937511")
DEV_ERRORS = {0: "ok", 1: "timeout", 2: "bad index", 3: "bad count", 4: "bad label", 5: "bad csr"}

# Every entry point of include/ckv.h with its argument types.
_P, _I, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
SIGNATURES = {
    "ckv_status_str": ([_I], ctypes.c_char_p),
    "ckv_version": ([], _I),
    "ckv_create": ([_P, ctypes.POINTER(_P)], _I),
    "ckv_destroy": ([_P], _I),
    "ckv_cluster_prefill": ([_P, _P, _I, _I, _P], _I),
    "ckv_cluster_incremental": ([_P, _P, _I, _I, _I, _P], _I),
    "ckv_kmeans_assign": ([_P, _P, _I, _P, _P], _I),
    "ckv_kmeans_update": ([_P, _P, _I, _P, _P], _I),
    "ckv_score": ([_P, _P, _I, _P, _P], _I),
    "ckv_select_scored": ([_P, _P, _I, _P, _P, _P], _I),
    "ckv_select": ([_P, _P, _I, _I, _P, _P, _P], _I),
    "ckv_sparse_decode_attn": ([_P, _P, _I, _P, _P, _P, _P, _I, _I, _P, _P], _I),
    "ckv_decode_step": ([_P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P], _I),
    "ckv_quest_pages": ([_P, _I, _I, _I, _I, _I, _P, _P, _P], _I),
    "ckv_quest_score": ([_P, _I, _P, _P, _I, _I, _I, _P, _P], _I),
    "ckv_selection_overlap": ([_I, _I, _I, _P, _P, _I, _P, _P, _I, _P, _P], _I),
    "ckv_centroid_channels": ([_P, _P, _P, _P], _I),
    "ckv_append_kv": ([_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P], _I),
    "ckv_channel_prescore": ([_P, _P, _I, _P, _P, _I, _P, _P, _P], _I),
    "ckv_cluster_incremental_begin": ([_P, _P, _I, _I, _I, _P], _I),
    "ckv_cluster_incremental_commit": ([_P, _P], _I),
    "ckv_get_info": ([_P, _P], _I),
    "ckv_export_clusters": ([_P, _P, _P, _P, _P, _P, _P], _I),
    "ckv_import_clusters": ([_P, _I, _I, _P, _P, _P, _P, _P], _I),
    "ckv_get_device_error": ([_P, ctypes.POINTER(_I)], _I),
    "ckv_set_wait_limit": ([_P, ctypes.c_int64, _I], _I),
    "ckv_set_l2_persistence": ([_P, ctypes.c_int64], _I),
    "ckv_paged_append": ([_P, _P, _P, _P, _P, _I, _P, _P, _P, _P], _I),
    "ckv_paged_attn_workspace": ([_P, _I, _I, ctypes.POINTER(ctypes.c_int64)], _I),
    "ckv_paged_decode_attn": ([_P, _P, _I, _P, _I, _F, _P, _P, _P, _P, _P, ctypes.c_int64, _P], _I),
    "ckv_paged_set_wait_limit": ([ctypes.c_int64, _I], _I),
    "ckv_paged_evict_select": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "ckv_paged_evict_apply": ([_P, _I, _I, _P, _P, _P], _I),
    "ckv_paged_plan": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P], _I),
    "ckv_rotate": ([_P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P], _I),
    "ckv_paged_append_rotated": ([_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P], _I),
    "ckv_paged_shared_workspace": ([_P, _I, ctypes.POINTER(ctypes.c_int64)], _I),
    "ckv_paged_shared_attn": ([_P, _P, _I, _P, _I, _F, _P, _P, _I, _P, _P, _P, ctypes.c_int64, _P], _I),
    "ckv_sparse_decode_attn_noalloc": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P], _I),
}


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "units", "d", "g", "sinks", "ratio", "m", "c_plus", "iters", "max_len",
        "max_clusters", "max_budget", "kv_dtype")]


class Info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_clusters", "prefill_clusters", "prefill_len", "clustered_end")]


class PagedCacheStruct(ctypes.Structure):
    """ckv_paged_cache."""
    _fields_ = ([(n, _P) for n in ("K", "V")]
                + [(n, ctypes.c_int64 * 3) for n in ("k_stride", "v_stride")]
                + [(n, _P) for n in ("table", "lens", "mass", "pos", "seen", "dev_err")]
                + [(n, ctypes.c_int32) for n in ("n_pages", "heads", "page_size", "seqs", "max_pages", "d",
                                                 "kv_dtype")])


class Rotary(ctypes.Structure):
    """ckv_rotary."""
    _fields_ = ([(n, _P) for n in ("turns", "q_weight", "k_weight")] + [("eps", _F), ("amplitude", _F)]
                + [("rot", _I), ("interleaved", _I)])


_ROTARY = struct.Struct("PPPffii").pack  # its bytes, in a third of the time


class CKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().ckv_status_str(status).decode()}")


_LIB = None


def lib():
    """The loaded libckv.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "recallable_kv_cache_gb300.build.build(); there is no CPU fallback")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = handle
    return _LIB


def _check(status: int, where: str):
    if status != 0:
        raise CKVError(status, where)


def ptr(t) -> int | None:
    """Device pointer of a tensor (or None)."""
    if t is None:
        return None
    return t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _is_tensor(t) -> bool:
    return hasattr(t, "shape") and hasattr(t, "data_ptr")


class Context:
    """One library context: the cluster state of `units` (sequence, layer, KV
    head) triples, allocated on the current CUDA device.

    Tensor arguments are checked against the context's layout before the call
    (the C ABI takes plain pointers and cannot see extents): K and V must be
    contiguous [units, max_len, d], q contiguous [units, g, d], idx [units, >= B]
    and count [units] int32, out [units, g, d]; a mismatch raises ValueError
    and nothing is launched."""

    def __init__(self, units: int, g: int, max_len: int, max_clusters: int, max_budget: int,
                 kv_dtype: str = "bf16", d: int = 128, sinks: int = 16, ratio: int = 80,
                 m: int = 320, c_plus: int = 4, iters: int = 10):
        self.cfg = Config(units, d, g, sinks, ratio, m, c_plus, iters, max_len, max_clusters,
                          max_budget, BF16 if kv_dtype == "bf16" else F32)
        h = ctypes.c_void_p()
        _check(lib().ckv_create(ctypes.byref(self.cfg), ctypes.byref(h)), "ckv_create")
        self.handle = h

    def _kv(self, *ts):
        for t in ts:
            if _is_tensor(t) and (tuple(t.shape) != (self.cfg.units, self.cfg.max_len, self.cfg.d)
                                  or not t.is_contiguous()):
                raise ValueError(f"K/V must be contiguous [{self.cfg.units}, {self.cfg.max_len}, {self.cfg.d}], "
                                 f"got {tuple(t.shape)}")

    def _q(self, q):
        if _is_tensor(q) and (tuple(q.shape) != (self.cfg.units, self.cfg.g, self.cfg.d) or not q.is_contiguous()):
            raise ValueError(f"q must be contiguous [{self.cfg.units}, {self.cfg.g}, {self.cfg.d}], got {tuple(q.shape)}")

    def _sel(self, B, idx, count):
        if _is_tensor(idx) and (idx.dim() != 2 or idx.shape[0] != self.cfg.units or idx.shape[1] < max(B, 1)
                                or not idx.is_contiguous() or idx.stride(0) != B and B > 0):
            raise ValueError(f"idx must be contiguous [{self.cfg.units}, B={B}], got {tuple(idx.shape)}")
        if _is_tensor(count) and tuple(count.shape) != (self.cfg.units,):
            raise ValueError(f"count must be [{self.cfg.units}], got {tuple(count.shape)}")

    def _out(self, out):
        if _is_tensor(out) and (tuple(out.shape) != (self.cfg.units, self.cfg.g, self.cfg.d) or not out.is_contiguous()):
            raise ValueError(f"out must be contiguous [{self.cfg.units}, {self.cfg.g}, {self.cfg.d}], "
                             f"got {tuple(out.shape)}")

    def close(self):
        if getattr(self, "handle", None):
            _check(lib().ckv_destroy(self.handle), "ckv_destroy")
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- clustering ------------------------------------------------------------
    def cluster_prefill(self, K, L: int, n_clusters: int = 0, stream=None):
        self._kv(K)
        _check(lib().ckv_cluster_prefill(self.handle, ptr(K), L, n_clusters, _stream(stream)),
               "ckv_cluster_prefill")

    def cluster_incremental(self, K, start: int, m: int | None = None, c_plus: int | None = None,
                            stream=None):
        m = self.cfg.m if m is None else m
        c_plus = self.cfg.c_plus if c_plus is None else c_plus
        self._kv(K)
        _check(lib().ckv_cluster_incremental(self.handle, ptr(K), start, m, c_plus, _stream(stream)),
               "ckv_cluster_incremental")

    def cluster_incremental_begin(self, K, start: int, m: int | None = None, c_plus: int | None = None,
                                  stream=None):
        m = self.cfg.m if m is None else m
        c_plus = self.cfg.c_plus if c_plus is None else c_plus
        self._kv(K)
        _check(lib().ckv_cluster_incremental_begin(self.handle, ptr(K), start, m, c_plus, _stream(stream)),
               "ckv_cluster_incremental_begin")

    def cluster_incremental_commit(self, stream=None):
        _check(lib().ckv_cluster_incremental_commit(self.handle, _stream(stream)),
               "ckv_cluster_incremental_commit")

    def kmeans_assign(self, K, L: int, labels, stream=None):
        self._kv(K)
        _check(lib().ckv_kmeans_assign(self.handle, ptr(K), L, ptr(labels), _stream(stream)),
               "ckv_kmeans_assign")

    def kmeans_update(self, K, L: int, labels, stream=None):
        self._kv(K)
        _check(lib().ckv_kmeans_update(self.handle, ptr(K), L, ptr(labels), _stream(stream)),
               "ckv_kmeans_update")

    # -- decode ----------------------------------------------------------------
    def score(self, q, scores, stream=None):
        self._q(q)
        _check(lib().ckv_score(self.handle, ptr(q), _dtype_code(q), ptr(scores), _stream(stream)),
               "ckv_score")

    def centroid_channels(self, muT, chmax, stream=None):
        """Channel-major scoring centroids and per-channel maxima (see ckv_centroid_channels)."""
        _check(lib().ckv_centroid_channels(self.handle, ptr(muT), ptr(chmax), _stream(stream)),
               "ckv_centroid_channels")

    def channel_prescore(self, q, muT, chmax, r: int, scores, channels=None, stream=None):
        """Scores over the r critical channels (see ckv_channel_prescore)."""
        _check(lib().ckv_channel_prescore(self.handle, ptr(q), _dtype_code(q), ptr(muT), ptr(chmax), r,
                                          ptr(scores), ptr(channels), _stream(stream)), "ckv_channel_prescore")

    def select_scored(self, scores, B: int, idx, count, stream=None):
        _check(lib().ckv_select_scored(self.handle, ptr(scores), B, ptr(idx), ptr(count),
                                       _stream(stream)), "ckv_select_scored")

    def select(self, q, B: int, idx, count, stream=None):
        self._q(q)
        self._sel(B, idx, count)
        _check(lib().ckv_select(self.handle, ptr(q), _dtype_code(q), B, ptr(idx), ptr(count),
                                _stream(stream)), "ckv_select")

    def sparse_decode_attn(self, q, K, V, idx, count, B: int, cur_len: int, out, stream=None):
        self._q(q)
        self._kv(K, V)
        self._sel(B, idx, count)
        self._out(out)
        _check(lib().ckv_sparse_decode_attn(self.handle, ptr(q), _dtype_code(q), ptr(K), ptr(V),
                                            ptr(idx), ptr(count), B, cur_len, ptr(out),
                                            _stream(stream)), "ckv_sparse_decode_attn")

    def decode_step(self, q, K, V, B: int, cur_len: int, idx, count, out, stream=None):
        self._q(q)
        self._kv(K, V)
        self._sel(B, idx, count)
        self._out(out)
        _check(lib().ckv_decode_step(self.handle, ptr(q), _dtype_code(q), ptr(K), ptr(V), B, cur_len, ptr(idx),
                                     ptr(count), ptr(out), _stream(stream)), "ckv_decode_step")

    # -- state -----------------------------------------------------------------
    def info(self) -> Info:
        inf = Info()
        _check(lib().ckv_get_info(self.handle, ctypes.byref(inf)), "ckv_get_info")
        return inf

    def export_clusters(self, mu=None, mu_hat=None, sizes=None, offsets=None, perm=None, stream=None):
        _check(lib().ckv_export_clusters(self.handle, ptr(mu), ptr(mu_hat), ptr(sizes), ptr(offsets),
                                         ptr(perm), _stream(stream)), "ckv_export_clusters")

    def import_clusters(self, n_clusters: int, clustered_end: int, mu, sizes=None, offsets=None,
                        perm=None, stream=None):
        _check(lib().ckv_import_clusters(self.handle, n_clusters, clustered_end, ptr(mu), ptr(sizes),
                                         ptr(offsets), ptr(perm), _stream(stream)),
               "ckv_import_clusters")

    def set_wait_limit(self, cycles: int = 2_000_000_000, stall: bool = False):
        """Bounded-wait limit of this context's kernels, and the failure
        detection test switch (see ckv_set_wait_limit)."""
        _check(lib().ckv_set_wait_limit(self.handle, int(cycles), 1 if stall else 0), "ckv_set_wait_limit")

    def set_l2_persistence(self, nbytes: int = -1):
        """L2 set-aside for the centroid scoring copy and perm, which every
        decode step re-reads (see ckv_set_l2_persistence): -1 = what the
        context needs, 0 = off."""
        _check(lib().ckv_set_l2_persistence(self.handle, int(nbytes)), "ckv_set_l2_persistence")

    def device_error(self) -> int:
        v = ctypes.c_int32()
        _check(lib().ckv_get_device_error(self.handle, ctypes.byref(v)), "ckv_get_device_error")
        return v.value


def sparse_decode_attn_noalloc(q, K, V, idx, count, units: int, g: int, max_len: int, sinks: int,
                               clustered_end: int, cur_len: int, B: int, out, dev_err=None, stream=None):
    """Sparse decode attention without a context and without any allocation:
    for callers that may not allocate device memory (inside graph capture, or
    under an engine that owns all device memory).  Its scratch is a fixed
    8 MiB array inside the library; calls that overlap on the GPU race.  The
    first call on a device must come before any stream capture."""
    _check(lib().ckv_sparse_decode_attn_noalloc(ptr(q), _dtype_code(q), ptr(K), ptr(V), ptr(idx),
                                                ptr(count), units, g, max_len, sinks, clustered_end,
                                                cur_len, B, ptr(out), ptr(dev_err), _stream(stream)),
           "ckv_sparse_decode_attn_noalloc")


def quest_pages(K, L: int, page_max, page_min, sinks: int = 16, stream=None):
    """Page metadata of the page-granular comparator (see ckv_quest_pages)."""
    units, max_len = K.shape[0], K.shape[1]
    _check(lib().ckv_quest_pages(ptr(K), _dtype_code(K), units, max_len, sinks, L, ptr(page_max), ptr(page_min),
                                 _stream(stream)), "ckv_quest_pages")


def quest_score(q, page_max, page_min, scores, stream=None):
    """Page weights of the page-granular comparator (see ckv_quest_score)."""
    units, g = q.shape[0], q.shape[1]
    _check(lib().ckv_quest_score(ptr(q), _dtype_code(q), ptr(page_max), ptr(page_min), units, g,
                                 page_max.shape[1], ptr(scores), _stream(stream)), "ckv_quest_score")


def selection_overlap(prev, idx, count, hits, max_len: int, stream=None):
    """hits[u] = tokens of the selection (idx, count) that appear in any of the
    earlier selections ``prev`` = [(idx_r, count_r), ...] (see
    ckv_selection_overlap).  All idx_r share one shape [units, B_prev]."""
    units, B = idx.shape
    R = len(prev)
    B_prev = prev[0][0].shape[1] if R else 0
    ip = (ctypes.c_void_p * max(R, 1))(*[ptr(p[0]) for p in prev])
    cp = (ctypes.c_void_p * max(R, 1))(*[ptr(p[1]) for p in prev])
    _check(lib().ckv_selection_overlap(units, max_len, R, ip, cp, B_prev, ptr(idx), ptr(count), B, ptr(hits),
                                       _stream(stream)), "ckv_selection_overlap")


def append_kv(k_src, v_src, K, V, pos: int, n: int | None = None, stream=None):
    """Rows [pos, pos + n) of every unit of K and V := rows [0, n) of k_src /
    v_src (see ckv_append_kv).  k_src / v_src are [units, d] (one row, n = 1)
    or [units, src_len, d] (a view with a unit stride is taken as src_len =
    that stride / d); they may live in pinned host memory the device maps."""
    units, max_len, d = K.shape
    if k_src.dim() == 2:
        src_len, n = 1, 1
    else:
        src_len = k_src.stride(0) // d
        n = k_src.shape[1] if n is None else n
    _check(lib().ckv_append_kv(ptr(k_src), ptr(v_src), src_len, _dtype_code(K), units, max_len, pos, n, ptr(K),
                               ptr(V), _stream(stream)), "ckv_append_kv")


def _raw_calls(torch):
    """(raw current stream of a device, current device): torch's own raw calls,
    as making a Stream object takes longer than a launch (3 us a call), or the
    public ones in a build that lacks those."""
    return (getattr(torch._C, "_cuda_getCurrentRawStream", None)
            or (lambda index: torch.cuda.current_stream(index).cuda_stream),
            getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device)


_TORCH = None


def _torch():
    """(torch, int32, int64, float32, *_raw_calls), looked up once."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = (torch, torch.int32, torch.int64, torch.float32, *_raw_calls(torch))
    return _TORCH


def rotary_turns(frequencies):
    """The pairs' angular frequencies (radians per position, floats) as the 64-bit
    fractions of a turn that the rotary calls take: int64 [rot / 2], on the CPU,
    holding the bits of round(w / (2 pi) * 2^64) mod 2^64."""
    import torch
    tau = 2 * _PI
    turns = []
    for w in frequencies:
        exact = fractions.Fraction(float(w)) / tau * 2 ** 64  # refuses infinities and NaN
        bits = round(exact) % 2 ** 64
        turns.append(bits - 2 ** 64 if bits >= 2 ** 63 else bits)
    return torch.tensor(turns, dtype=torch.int64)


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original: int = 8192, low: float = 1.0, high: float | None = None):
    """(frequencies [rot / 2] in radians per position, amplitude) of rotary
    positions, w_i = base^(-2 i / rot), scaled for contexts ``factor`` times the
    ``original`` length by one of
      "linear"  positions interpolated: w_i / factor;
      "base"    the base raised so that the slowest pair is interpolated and the
                fastest stays: base * factor^(rot / (rot - 2));
      "ramp"    pairs that turn more than ``high`` times over the original length
                stay, those that turn less than ``low`` times are interpolated,
                and in between the share goes with their number i; the amplitude
                is 0.1 ln(factor) + 1 (YaRN, arXiv 2309.00071);
      "bands"   the same borders, the share going with the number of turns, and
                an amplitude of 1.
    ``high`` is 32 for a ramp and 4 for bands if None, as is usual."""
    if rot < 2 or rot % 2 or not base > 0 or not factor >= 1:
        raise ValueError(f"rot must be even and positive, base > 0 and factor >= 1, got {rot}, {base}, {factor}")
    if scaling not in (None, "linear", "base", "ramp", "bands"):
        raise ValueError(f"scaling must be None, linear, base, ramp or bands, got {scaling!r}")
    half, amplitude = rot // 2, 1.0
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    w = [base ** (-i / half) for i in range(half)]
    if scaling == "linear":
        w = [x / factor for x in w]
    elif scaling in ("ramp", "bands"):
        if high is None:
            high = 32.0 if scaling == "ramp" else 4.0
        if not 0 < low < high or original < 1:
            raise ValueError(f"0 < low < high and original >= 1 are needed, got {low}, {high}, {original}")
        if scaling == "ramp":
            # the (fractional) pair that turns n times over the original length
            pair = [half * math.log(original / (2 * math.pi * n)) / math.log(base) for n in (high, low)]
            first, last = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
            share = [min(1.0, max(0.0, (i - first) / max(last - first, 1e-3))) for i in range(half)]
            amplitude = 0.1 * math.log(factor) + 1.0
        else:
            turned = [original * x / (2 * math.pi) for x in w]
            share = [min(1.0, max(0.0, (high - n) / (high - low))) for n in turned]
        w = [x * (1 - s) + x / factor * s for x, s in zip(w, share)]
    return w, amplitude


_STRIDES = {}  # stride arrays, made once for equal strides


def _rotary(turns, q_weight, k_weight, eps, amplitude, interleaved, device):
    """ckv_rotary of a call, as bytes, after the checks."""
    _, _, i64, f32, _, _ = _torch()
    rot = at = 0
    if turns is not None:
        if turns.dtype is not i64:
            raise TypeError(f"turns must be int64 (see rotary_turns), got {turns.dtype}")
        if turns.dim() != 1 or not turns.is_contiguous() or turns.device != device:
            raise ValueError(f"turns must be contiguous [rot / 2] on {device}, got {list(turns.shape)} on {turns.device}")
        rot, at = 2 * turns.shape[0], turns.data_ptr()
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if w.dtype is not f32:
                raise TypeError(f"{name} must be float32, got {w.dtype}")
            if w.shape != (128,) or not w.is_contiguous() or w.device != device:
                raise ValueError(f"{name} must be contiguous [128] on {device}, got {list(w.shape)} on {w.device}")
    return _ROTARY(at, 0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(), eps,
                   amplitude, rot, 1 if interleaved else 0)


def _heads(name, t, tokens, heads, dtype, device):
    """(address, strides as a C array) of t [tokens, heads, 128] after the checks."""
    shape, st = t.shape, t.stride()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape != (tokens, heads, 128):
        raise ValueError(f"{name} must be [{tokens}, {heads}, 128], got {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if st[2] != 1:
        raise ValueError(f"the channels of {name} must be contiguous, got strides {list(st)}")
    got = _STRIDES.get(st)
    if got is None:
        if len(_STRIDES) > 256:
            _STRIDES.clear()
        got = _STRIDES[st] = (ctypes.c_int64 * 2)(st[0], st[1])
    return t.data_ptr(), got


def rotate(q, k, positions, turns, q_out, k_out, interleaved: bool = False, q_weight=None, k_weight=None,
           eps: float = 1e-6, amplitude: float = 1.0, stream=None):
    """Norms (with q_weight, k_weight [128] float32) and rotary positions of q
    [tokens, heads_q, 128] and k [tokens, heads_k, 128] into q_out and k_out, which
    may be q and k (see ckv_rotate).  positions [tokens] int32; turns [rot / 2]
    int64 (see rotary_turns), or None for norms alone; either of q and k may be
    None, with its output."""
    torch, i32, _, _, raw_stream, current = _torch()
    x = k if q is None else q
    if x is None or x.dim() != 3:
        raise ValueError("q or k must be given, as [tokens, heads, 128]")
    tokens, device, dtype, code = x.shape[0], x.device, x.dtype, _dtype_code(x)
    if not x.is_cuda:
        raise ValueError(f"the rows must be on a CUDA device, got {device}")
    if positions.dtype is not i32:
        raise TypeError(f"positions must be int32, got {positions.dtype}")
    if positions.shape != (tokens,) or not positions.is_contiguous() or positions.device != device:
        raise ValueError(f"positions must be contiguous [{tokens}] on {device}, got {list(positions.shape)} on "
                         f"{positions.device}")
    args = []
    for name, t, o in (("q", q, q_out), ("k", k, k_out)):
        if (t is None) != (o is None):
            raise ValueError(f"{name} and {name}_out go together")
        if t is None:
            args += (None, None, None, None, 0)
        else:
            heads = t.shape[1] if t.dim() == 3 else 0
            args += _heads(name, t, tokens, heads, dtype, device)
            args += _heads(name + "_out", o, tokens, heads, dtype, device)
            args.append(heads)
    rotary = _rotary(turns, q_weight, k_weight, eps, amplitude, interleaved, device)
    index, fn = device.index, lib().ckv_rotate
    stream = raw_stream(index) if stream is None else getattr(stream, "cuda_stream", stream)
    if index == current():
        status = fn(rotary, *args, positions.data_ptr(), tokens, 128, code, stream)
    else:
        with torch.cuda.device(index):
            status = fn(rotary, *args, positions.data_ptr(), tokens, 128, code, stream)
    if status:
        raise CKVError(status, "ckv_rotate")


def paged_set_wait_limit(cycles: int = 2_000_000_000, stall: bool = False):
    """Bounded-wait limit of the paged attention in this process, and its
    failure detection test switch (see ckv_paged_set_wait_limit)."""
    _check(lib().ckv_paged_set_wait_limit(int(cycles), 1 if stall else 0), "ckv_paged_set_wait_limit")


def _address(name, t, shape, dtype, device, contiguous=True):
    """Address of a paged cache's tensor after the checks."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name} must be {'contiguous ' if contiguous else ''}{list(shape)}, got "
                         f"{list(t.shape)} with strides {list(t.stride())}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    return t.data_ptr()


def _addresses(dtype, device):
    """_address of contiguous tensors of one dtype and device, in one look where all
    is well: the calls of a step have a dozen of them."""
    index = device.index

    def address(name, t, shape):
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
            return t.data_ptr()
        return _address(name, t, shape, dtype, device)
    return address


class PagedCache:
    """A paged K/V cache over the caller's tensors (see the paged cache section
    of ckv.h): ``K``, ``V`` [n_pages, heads, page_size, 128] bf16 or float32, any
    strides with contiguous channels; ``table`` [seqs, max_pages] and ``lens``
    [seqs] int32; optionally ``mass`` (float32) and ``pos`` (int32) [seqs, heads,
    max_pages * page_size], ``seen`` [seqs] int32 and ``dev_err`` [1] int32.

    ``g`` is the number of query heads per KV head.  With ``shared`` the handle has
    the workspace of shared_attn too.  ``mass`` and ``pos`` are
    sized by the capacity, 8 bytes for each of seqs * heads * rows, and with
    ``mass`` so is the workspace, 4 g bytes for each (0.27 g MB without; a handle
    made without ``mass`` takes no ``mass_out``).  The handle keeps the
    tensors alive and owns the attention's workspace, allocated here (so that
    every call may be captured into a CUDA graph; the handle itself is made
    outside a capture).  Like a Context, one handle
    must not be used from two streams at the same time; another handle over the
    same tensors has a workspace of its own.  Calls run on the tensors' device,
    on ``stream`` or that device's current stream.  The handle may be dropped
    while calls are under way: the workspace's memory is used again only after
    them.  A graph captured from its calls keeps nothing alive, so the handle
    has to outlive it, and a raw stream (not torch's) has to outlive the handle.
    A tensor of another shape, dtype, device or layout raises ValueError
    (TypeError for dtypes) and nothing is launched."""

    _shared_attn = None

    def __init__(self, K, V, table, lens, g: int = 1, mass=None, pos=None, seen=None, dev_err=None,
                 shared: bool = False):
        import torch
        self.device = K.device
        if K.dim() != 4 or K.shape != V.shape or K.dtype != V.dtype:
            raise ValueError("K and V must be [n_pages, heads, page_size, 128] of one dtype, got "
                             f"{tuple(K.shape)} {K.dtype}, {tuple(V.shape)} {V.dtype}")
        if K.stride(3) != 1 or V.stride(3) != 1:
            raise ValueError("the channels of K and V must be contiguous")
        code = _dtype_code(K)
        n_pages, heads, page, d = K.shape
        if table.dim() != 2:
            raise ValueError(f"table must be [seqs, max_pages], got {tuple(table.shape)}")
        seqs, width = table.shape
        self.seqs, self.heads, self.g, self.rows = seqs, heads, g, width * page
        self.dtype, self._code = K.dtype, code
        self._i32, self._f32 = torch.int32, torch.float32
        self._per_seq, self._per_unit, self._per_row = (seqs,), (seqs, heads), (seqs, heads, self.rows)
        self._q_shape, self._lse_shape = (seqs, heads * g, 128), (seqs, heads * g)
        for name, t, shape, dtype in (
                ("V", V, tuple(K.shape), K.dtype), ("table", table, (seqs, width), self._i32),
                ("lens", lens, self._per_seq, self._i32), ("mass", mass, self._per_row, self._f32),
                ("pos", pos, self._per_row, self._i32), ("seen", seen, self._per_seq, self._i32),
                ("dev_err", dev_err, (1,), self._i32)):
            self._tensor(name, t, shape, dtype, contiguous=name != "V")
        if self.device.type != "cuda":
            raise ValueError(f"the cache must be on a CUDA device, got {self.device}")
        self.K, self.V, self.table, self.lens = K, V, table, lens
        self.mass, self.pos, self.seen, self.dev_err = mass, pos, seen, dev_err
        self._struct = PagedCacheStruct(
            ptr(K), ptr(V), (ctypes.c_int64 * 3)(*K.stride()[:3]), (ctypes.c_int64 * 3)(*V.stride()[:3]), ptr(table),
            ptr(lens), ptr(mass), ptr(pos), ptr(seen), ptr(dev_err), n_pages, heads, page, seqs, width, d, code)
        self._ref = ctypes.addressof(self._struct)
        so = lib()
        self._append, self._attn = so.ckv_paged_append, so.ckv_paged_decode_attn
        self._select, self._apply = so.ckv_paged_evict_select, so.ckv_paged_evict_apply
        self._cuda, self._index = torch.cuda, self.device.index
        self._raw_stream, self._current = _torch()[4:]
        self._ints, self._floats = _addresses(torch.int32, self.device), _addresses(torch.float32, self.device)
        self._stride_arrays = {}
        self._plan, self._append_rotated = so.ckv_paged_plan, so.ckv_paged_append_rotated
        self._shared_attn = so.ckv_paged_shared_attn
        need = ctypes.c_int64()
        _check(so.ckv_paged_attn_workspace(self._ref, g, 0 if mass is None else 1, ctypes.byref(need)),
               "ckv_paged_attn_workspace")
        if shared:
            more = ctypes.c_int64()
            _check(so.ckv_paged_shared_workspace(self._ref, g, ctypes.byref(more)), "ckv_paged_shared_workspace")
            need.value = max(need.value, more.value)
        self.shared = shared
        self.workspace = torch.empty(need.value, dtype=torch.uint8, device=self.device)
        self.workspace[:4096].zero_()  # the counters; calls leave them zero
        torch.cuda.current_stream(self.device).synchronize()  # whatever stream the first call is on
        self._streams = {self._raw_stream(self._index)}  # on which the allocator knows the workspace is used
        self._workspace = (ptr(self.workspace), need.value)

    def _tensor(self, name, t, shape, dtype, contiguous=True):
        """Address of t after the checks; None is passed on (the C call says
        which arguments it needs)."""
        return None if t is None else _address(name, t, shape, dtype, self.device, contiguous)

    def _strides(self, t, n):
        """The first n strides of t as a C array (made once for equal strides)."""
        key = t.stride()
        got = self._stride_arrays.get(key)
        if got is None:
            if len(self._stride_arrays) > 256:
                self._stride_arrays.clear()
            if key[n] != 1:
                raise ValueError(f"the channels must be contiguous, got strides {list(key)}")
            got = self._stride_arrays[key] = (ctypes.c_int64 * n)(*key[:n])
        return got

    def _note_stream(self, raw):
        """Tells the allocator that the workspace is in use on a stream, once for
        each: memory that is freed goes to the stream it was allocated on, after
        what is then queued on the others.  Not while the stream is capturing:
        nothing runs, and the graph's replays are its owner's."""
        # 0 is the default stream, which is no address for ExternalStream
        stream = (self._cuda.ExternalStream(raw, device=self.device) if raw
                  else self._cuda.default_stream(self.device))
        with self._cuda.stream(stream):
            if self._cuda.is_current_stream_capturing():
                return
        self.workspace.record_stream(stream)
        self._streams.add(raw)

    def _call(self, fn, stream, *args):
        stream = self._raw_stream(self._index) if stream is None else getattr(stream, "cuda_stream", stream)
        if stream not in self._streams and (fn is self._attn or fn is self._shared_attn):
            self._note_stream(stream)
        if self._index == self._current():
            status = fn(self._ref, *args, stream)
        else:
            with self._cuda.device(self._index):
                status = fn(self._ref, *args, stream)
        if status:
            raise CKVError(status, fn.__name__)

    def append(self, k, v, counts=None, start=None, first=None, stream=None):
        """counts[s] rows of k, v [seqs, heads, n, 128] (any strides with
        contiguous channels) to every sequence (see ckv_paged_append); k and v
        may live in pinned host memory the device maps."""
        shape, device, i32, tensor = k.shape, self.device, self._i32, self._tensor
        if len(shape) != 4 or shape[0] != self.seqs or shape[1] != self.heads or shape[3] != 128 or v.shape != shape:
            raise ValueError(f"k and v must be [{self.seqs}, {self.heads}, n, 128], got {tuple(shape)}, "
                             f"{tuple(v.shape)}")
        if k.dtype != self.dtype or v.dtype != self.dtype:
            raise TypeError(f"k and v must be {self.dtype}, got {k.dtype}, {v.dtype}")
        if k.device != device or v.device != device:
            for t in (k, v):
                if t.device != device and not (t.device.type == "cpu" and t.is_pinned()):
                    raise ValueError(f"k and v must be on {device} or pinned, got {t.device}")
        self._call(self._append, stream, k.data_ptr(), v.data_ptr(), self._strides(k, 3), self._strides(v, 3), shape[2],
                   None if counts is None else tensor("counts", counts, self._per_seq, i32),
                   None if start is None else tensor("start", start, self._per_seq, i32),
                   None if first is None else tensor("first", first, self._per_seq, i32))

    def decode_attn(self, q, out, lse=None, mass_in=None, mass_out=None, scale=None, stream=None):
        """Attention of q [seqs, heads * g, 128] over the rows held into out
        [seqs, heads * g, 128] float32 (see ckv_paged_decode_attn).  With
        ``mass_out`` (for instance the cache's own mass, given as mass_in too)
        each row's weight is added to mass_in.  scale: 1 / sqrt(128) if None."""
        if q.shape != self._q_shape:
            raise ValueError(f"q must be {list(self._q_shape)}, got {tuple(q.shape)}")
        if q.dtype != self.dtype:
            raise TypeError(f"q must be {self.dtype}, got {q.dtype}")
        if q.device != self.device:
            raise ValueError(f"q is on {q.device}, the cache on {self.device}")
        f32, tensor = self._f32, self._tensor
        self._call(self._attn, stream, q.data_ptr(), self._code, self._strides(q, 2), self.g,
                   128 ** -0.5 if scale is None else scale, tensor("out", out, self._q_shape, f32),
                   None if lse is None else tensor("lse", lse, self._lse_shape, f32),
                   None if mass_in is None else tensor("mass_in", mass_in, self._per_row, f32),
                   None if mass_out is None else tensor("mass_out", mass_out, self._per_row, f32),
                   *self._workspace)

    def _moves(self, moves, n_moves):
        shape = moves.shape
        if len(shape) != 4:
            raise ValueError(f"moves must be [seqs, heads, max_moves, 2], got {tuple(shape)}")
        return (shape[2], self._tensor("moves", moves, (self.seqs, self.heads, shape[2], 2), self._i32),
                self._tensor("n_moves", n_moves, self._per_unit, self._i32))

    def evict_select(self, budget: int, sinks: int, recent: int, moves, n_moves, stream=None):
        """The rows to move when every KV head keeps ``budget`` of its rows (see
        ckv_paged_evict_select): moves [seqs, heads, max_moves, 2], n_moves
        [seqs, heads] int32."""
        self._call(self._select, stream, budget, sinks, recent, *self._moves(moves, n_moves))

    def evict_apply(self, budget: int, moves, n_moves, stream=None):
        """Carries the moves out and shortens lens (see ckv_paged_evict_apply)."""
        self._call(self._apply, stream, budget, *self._moves(moves, n_moves))

    def evict(self, budget: int, sinks: int, recent: int, moves, n_moves, stream=None):
        """evict_select, then evict_apply."""
        self.evict_select(budget, sinks, recent, moves, n_moves, stream)
        self.evict_apply(budget, moves, n_moves, stream)

    # -- a step's tokens ---------------------------------------------------------
    def plan(self, counts, held, free, span, slots, starts, granted, shared=None, start=None, first=None,
             held_out=None, span_out=None, stream=None):
        """Pages for counts[s] more tokens of every sequence, and where each token
        goes (see ckv_paged_plan): counts, held, granted, shared, start, first,
        held_out [seqs], span, span_out [2], starts [seqs + 1], slots [tokens, 4]
        and the ring of free pages ``free``, all int32.  held_out and span_out are
        held and span themselves if None; table, lens and seen change."""
        ints, per_seq = self._ints, self._per_seq
        if free.dim() != 1 or slots.dim() != 2:
            raise ValueError(f"free must be [pages] and slots [tokens, 4], got {list(free.shape)}, {list(slots.shape)}")
        n_slots, cap = slots.shape[0], free.shape[0]
        h, sp = ints("held", held, per_seq), ints("span", span, (2,))
        self._call(self._plan, stream, ints("counts", counts, per_seq),
                   None if start is None else ints("start", start, per_seq),
                   None if first is None else ints("first", first, per_seq),
                   None if shared is None else ints("shared", shared, per_seq), h,
                   h if held_out is None else ints("held_out", held_out, per_seq), ints("free", free, (cap,)), cap, sp,
                   sp if span_out is None else ints("span_out", span_out, (2,)), ints("granted", granted, per_seq),
                   ints("starts", starts, (self.seqs + 1,)), ints("slots", slots, (n_slots, 4)), n_slots)

    def append_rotated(self, q, k, v, slots, turns, q_out, interleaved: bool = False, q_weight=None, k_weight=None,
                       eps: float = 1e-6, amplitude: float = 1.0, stream=None):
        """q, k normed and rotated (see rotate), q into q_out, k and v into the rows
        that slots [tokens, 4] of a plan gives them (see ckv_paged_append_rotated):
        q, q_out [tokens, heads * g, 128] (both None: no queries), k, v [tokens,
        heads, 128], any strides with contiguous channels."""
        device, heads, dtype = self.device, self.heads, self.dtype
        if k.dim() != 3:
            raise ValueError(f"k must be [tokens, {heads}, 128], got {list(k.shape)}")
        tokens, g = k.shape[0], self.g
        rotary = _rotary(turns, q_weight, k_weight, eps, amplitude, interleaved, device)
        if q is None and q_out is None:
            g = 0
            queries = rotated = (None, None)
        elif q is None or q_out is None:
            raise ValueError("q and q_out go together")
        else:
            queries = _heads("q", q, tokens, heads * g, dtype, device)
            rotated = _heads("q_out", q_out, tokens, heads * g, dtype, device)
        self._call(self._append_rotated, stream, rotary, *queries, g, *rotated,
                   *_heads("k", k, tokens, heads, dtype, device), *_heads("v", v, tokens, heads, dtype, device),
                   self._ints("slots", slots, (tokens, 4)), tokens)

    def shared_attn(self, q, out, group_starts, prefix, lse=None, scale=None, stream=None):
        """decode_attn (without weights) where sequences group_starts[i] ..
        group_starts[i + 1] - 1 have their first prefix[i] rows in common, which
        are then read once for all of them (see ckv_paged_shared_attn; those of a
        float32 cache are read once for each): group_starts [groups + 1] and prefix
        [groups] int32.  The handle must have been made with shared=True."""
        if not self.shared:
            raise ValueError("the handle was made without shared=True and has no workspace for this call")
        if q.shape != self._q_shape:
            raise ValueError(f"q must be {list(self._q_shape)}, got {tuple(q.shape)}")
        if q.dtype != self.dtype:
            raise TypeError(f"q must be {self.dtype}, got {q.dtype}")
        if q.device != self.device:
            raise ValueError(f"q is on {q.device}, the cache on {self.device}")
        if prefix.dim() != 1:
            raise ValueError(f"prefix must be [groups], got {list(prefix.shape)}")
        groups, ints, floats = prefix.shape[0], self._ints, self._floats
        self._call(self._shared_attn, stream, q.data_ptr(), self._code, self._strides(q, 2), self.g,
                   128 ** -0.5 if scale is None else scale, ints("group_starts", group_starts, (groups + 1,)),
                   ints("prefix", prefix, (groups,)), groups, floats("out", out, self._q_shape),
                   None if lse is None else floats("lse", lse, self._lse_shape), *self._workspace)
