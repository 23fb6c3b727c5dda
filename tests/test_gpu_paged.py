"""GPU parity of the paged cache (append, decode attention with the accumulated
weights, eviction) against its float64 oracle, through the public handle.

Tolerances of the attention.  Let S = max_r scale * sum_i |q_i k_ri|, n the rows.
  * a score sums 128 products in fp32, each step off by at most one unit in the
    last place of the running sum (a tensor core may truncate): es = 2^-16 S
    covers 128 * 2^-23 S and the rounding of the scale and of log2(e);
  * a weight's numerator and denominator each inherit es: 2 es, doubled for the
    second order; the exponential and a weight carried as two or more bf16 terms
    add at most 2^-17 together, doubled for the denominator: 2^-16;
  * sums over rows take at most n / 16 + 200 sequential steps (a tile of 16
    rows is one tensor-core step, partial sums are joined), each off by 2^-23.
So |out - exact| <= (4 es + 2^-16 + 2 * 2^-23 (n / 16 + 200)) sum_r w_r |v_r|,
the weights by the same factor, and lse by 2 es + 2^-19 + 2^-23 (n / 16 + 200 +
|lse|).  Copies and choices are exact."""
import math

import numpy as np
import pytest
import torch

import oracle.paged as po
from recallable_kv_cache_gb300 import ckv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
D = 128


def pools(n_pages, heads, page, dtype, layout, gen):
    """K, V [n_pages, heads, page, 128] of normal values in one of four layouts."""
    if layout == "hpd":
        shape, view = (2, n_pages, heads, page, D), lambda x: (x[0], x[1])
    elif layout == "phd":
        shape, view = (2, n_pages, page, heads, D), lambda x: (x[0].transpose(1, 2), x[1].transpose(1, 2))
    elif layout == "kv_in_page":
        shape, view = (n_pages, 2, heads, page, D), lambda x: (x[:, 0], x[:, 1])
    else:  # "wide": rows 160 channels apart, a slice of a wider pool
        shape, view = (2, n_pages, heads, page, 160), lambda x: (x[0][..., 8:136], x[1][..., 16:144])
    x = torch.randn(shape, generator=gen).to(DT[dtype]).cuda()
    return view(x)


class Case:
    """A cache of random contents: every row and page that is not held is NaN."""

    def __init__(self, lens, heads=2, g=4, page=16, dtype="bf16", layout="hpd", spare=3, width=None, seed=0,
                 q_scale=1.5, garbage=float("nan")):
        gen = torch.Generator().manual_seed(seed)
        S = len(lens)
        need = [-(-n // page) for n in lens]
        width = width or max(1, max(need))
        n_pages = sum(need) + spare
        self.K, self.V = pools(n_pages, heads, page, dtype, layout, gen)
        perm = torch.randperm(n_pages, generator=gen).to(torch.int32)
        table = torch.full((S, width), 2 ** 31 - 1, dtype=torch.int32)
        held = torch.zeros(n_pages, page, dtype=torch.bool)
        at = 0
        for s, n in enumerate(lens):
            table[s, :need[s]] = perm[at:at + need[s]]
            for i in range(need[s]):
                held[perm[at + i].long(), :min(page, n - i * page)] = True
            at += need[s]
        mask = ~held.cuda()[:, None, :, None].expand(n_pages, heads, page, D)
        self.K.masked_fill_(mask, garbage)
        self.V.masked_fill_(mask, garbage)
        R = width * page
        self.S, self.heads, self.g, self.page, self.R, self.n_pages, self.dtype = S, heads, g, page, R, n_pages, dtype
        self.lens_list = list(lens)
        self.table, self.lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.mass = torch.rand(S, heads, R, generator=gen).cuda()
        self.pos = torch.arange(R, dtype=torch.int32).expand(S, heads, R).contiguous().cuda()
        self.seen = self.lens.clone()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q = (q_scale * torch.randn(S, heads * g, D, generator=gen)).to(DT[dtype]).cuda()
        self.out = torch.full((S, heads * g, D), float("nan"), device="cuda")
        self.lse = torch.full((S, heads * g), float("nan"), device="cuda")
        self.handle = self.make()

    def make(self):
        return ckv.PagedCache(self.K, self.V, self.table, self.lens, g=self.g, mass=self.mass, pos=self.pos,
                              seen=self.seen, dev_err=self.err)

    def rows(self, s, h, n=None):
        n = self.lens_list[s] if n is None else n
        t = self.table[s].cpu().numpy()
        k, ok = po.rows(self.host("K"), t, h, n, self.n_pages)
        v, _ = po.rows(self.host("V"), t, h, n, self.n_pages)
        return k, v, ok

    def host(self, name):
        key = "_host_" + name
        if not hasattr(self, key):
            setattr(self, key, getattr(self, name).double().cpu().numpy())
        return getattr(self, key)

    def check_attention(self, scale=None, mass_in=None, mass_out=None, mass_before=None):
        """out, lse (and mass_out) against the oracle within the derived bounds."""
        scale = D ** -0.5 if scale is None else scale
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        mo = None if mass_out is None else mass_out.double().cpu().numpy()
        for s in range(self.S):
            for h in range(self.heads):
                k, v, ok = self.rows(s, h)
                qs = q[s, h * self.g:(h + 1) * self.g]
                o, z, w = po.attend(qs, k, v, ok, scale)
                got, gl = out[s, h * self.g:(h + 1) * self.g], lse[s, h * self.g:(h + 1) * self.g]
                n = self.lens_list[s]
                es = 2.0 ** -16 * abs(scale) * max([np.abs(qs) @ np.abs(x) for x in k[ok]], key=np.max).max() if ok.any() else 0.0
                sums = 2.0 ** -23 * (n / 16 + 200)
                eps = 4 * es + 2.0 ** -16 + 2 * sums
                for j in range(self.g):
                    if not ok.any():
                        assert not got[j].any() and gl[j] == -math.inf
                        continue
                    p = np.exp(scale * (k[ok] @ qs[j]) - z[j])
                    bound = eps * (p @ np.abs(v[ok])) + 1e-30
                    assert (np.abs(got[j] - o[j]) <= bound).all(), (s, h, j, np.abs(got[j] - o[j]).max(), bound.min())
                    assert abs(gl[j] - z[j]) <= 2 * es + 2.0 ** -19 + sums + 2.0 ** -23 * abs(z[j])
                if mo is not None:
                    base = np.zeros(n) if mass_in is None else mass_in[s, h, :n]
                    want = base + w
                    assert (np.abs(mo[s, h, :n] - want) <= eps * w + 2.0 ** -23 * np.abs(want) + 1e-30).all()
                    assert np.array_equal(mo[s, h, n:], mass_before[s, h, n:])


ATTEND = [
    # lens, heads, g, page, dtype, layout
    ([1], 1, 1, 16, "bf16", "hpd"),
    ([1], 1, 1, 16, "f32", "hpd"),
    ([0], 1, 4, 16, "bf16", "hpd"),
    ([0, 0, 0], 3, 2, 16, "f32", "hpd"),
    ([15, 16, 17, 31, 32, 33], 2, 4, 16, "bf16", "hpd"),
    ([15, 16, 17, 31, 32, 33], 2, 4, 16, "f32", "phd"),
    ([0, 7, 0, 129, 1, 0], 3, 8, 48, "bf16", "phd"),
    ([0, 7, 0, 129, 1, 0], 3, 8, 48, "f32", "kv_in_page"),
    ([63, 64, 65, 2], 8, 3, 64, "bf16", "kv_in_page"),
    ([500, 3], 5, 5, 32, "f32", "wide"),
    ([500, 3], 5, 7, 32, "bf16", "wide"),
    ([700, 255, 256, 257], 2, 9, 128, "bf16", "phd"),
    ([700, 255, 256, 257], 2, 12, 128, "f32", "hpd"),
    ([333, 1000], 1, 16, 16, "bf16", "hpd"),
    ([333, 1000], 1, 16, 16, "f32", "phd"),
    ([4097], 1, 2, 2048, "bf16", "hpd"),
    ([4097], 2, 6, 16, "f32", "hpd"),
    ([5000, 1, 77], 4, 1, 64, "bf16", "phd"),
    ([3] * 70, 7, 4, 16, "bf16", "hpd"),
    ([3, 0, 20] * 60, 11, 2, 16, "f32", "hpd"),
    # more sequences than a CTA has threads, and shares of units across CTAs
    ([1, 0, 0, 37] * 200, 1, 4, 16, "bf16", "hpd"),
    ([0, 2, 19] * 250, 1, 1, 16, "f32", "phd"),
    ([2000, 1900, 1000], 3, 4, 16, "bf16", "hpd"),
    ([2000, 5, 1000], 3, 16, 48, "f32", "hpd"),
]


@pytest.mark.parametrize("lens,heads,g,page,dtype,layout", ATTEND)
@pytest.mark.parametrize("mass", [False, True])
def test_attention(lens, heads, g, page, dtype, layout, mass):
    c = Case(lens, heads, g, page, dtype, layout, seed=len(lens) + g)
    mass_out = torch.full_like(c.mass, 7.0) if mass else None
    before = None if mass_out is None else mass_out.double().cpu().numpy()
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_in=c.mass if mass else None, mass_out=mass_out)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check_attention(mass_in=c.mass.double().cpu().numpy(), mass_out=mass_out, mass_before=before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_in_place_and_from_zero(dtype):
    c = Case([40, 0, 113], 2, 4, 16, dtype)
    before = c.mass.double().cpu().numpy()
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_in=c.mass, mass_out=c.mass)
    torch.cuda.synchronize()
    c.check_attention(mass_in=before, mass_out=c.mass, mass_before=before)
    fresh = torch.full_like(c.mass, -3.0)
    c.handle.decode_attn(c.q, c.out, mass_out=fresh)
    torch.cuda.synchronize()
    c.check_attention(mass_in=None, mass_out=fresh, mass_before=fresh.double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.11, 0.5])
def test_scale_and_strided_queries(dtype, scale):
    c = Case([90, 17], 2, 3, 32, dtype)
    wide = torch.zeros(2, 2 * 6 + 5, 136 * 2, dtype=DT[dtype], device="cuda")
    q = wide[:, 1:12:2, 8:136]
    q.copy_(c.q)
    c.handle.decode_attn(q, c.out, lse=c.lse, scale=scale)
    torch.cuda.synchronize()
    c.check_attention(scale=scale)


@pytest.mark.parametrize("dtype,S,heads,g", [("bf16", 1, 2, 3), ("f32", 1, 1, 1), ("bf16", 4, 1, 1), ("f32", 1, 1, 12)])
def test_strides_of_single_extents_are_free(dtype, S, heads, g):
    """One sequence, head or row: torch gives such an extent any stride."""
    c = Case([40] * S, heads, g, 16, dtype, width=3)
    h = heads * g
    q = torch.empty_strided(c.q.shape, (3 if S == 1 else h * 136, 5 if h == 1 else 136, 1), dtype=DT[dtype], device="cuda")
    q.copy_(c.q)
    c.handle.decode_attn(q, c.out, lse=c.lse)
    torch.cuda.synchronize()
    c.check_attention()
    k = torch.empty_strided((S, heads, 1, D), (7 if S == 1 else heads * 136, 9 if heads == 1 else 136, 1, 1),
                            dtype=DT[dtype], device="cuda")
    k.normal_()
    c.handle.append(k, k)
    for s in range(S):
        assert torch.equal(c.K[int(c.table[s, 2]), :, 8], k[s, :, 0])
    assert int(c.err) == 0 and c.lens.tolist() == [41] * S


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_and_far_scores(dtype):
    """Scores up to several hundred: the running maximum carries the sum."""
    c = Case([1000, 33], 2, 4, 16, dtype, q_scale=40.0)
    c.handle.decode_attn(c.q, c.out, lse=c.lse)
    torch.cuda.synchronize()
    c.check_attention()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("garbage", [float("inf"), float("-inf"), 3e38])
def test_rows_not_held_are_never_used(dtype, garbage):
    c = Case([5, 0, 47], 2, 8, 48, dtype, "phd", garbage=garbage)
    out = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=out)
    torch.cuda.synchronize()
    c.check_attention(mass_out=out, mass_before=np.zeros(out.shape))


RANGES = ["small V", "V by channel", "V by row", "large V", "V with zeros", "K against q", "K large", "q large", "scale"]


@pytest.mark.parametrize("kind", RANGES)
@pytest.mark.parametrize("dtype,g", [("f32", 2), ("f32", 8), ("f32", 9), ("f32", 16), ("bf16", 4), ("bf16", 16)])
def test_operands_over_the_whole_range(dtype, g, kind):
    """Operands from the smallest subnormal to the largest finite value, at the
    bounds at the top of this file; below 2^-126 a step of a sum is off by half
    a unit of 2^-149: one for each row and, where the running maximum grows, one
    more, and some for what is joined at the end."""
    c = Case([1, 7, 130, 61, 3000], 2, g, 16, dtype, "hpd", seed=g)
    gen = torch.Generator(device="cuda").manual_seed(7)
    scale, rows, channels = D ** -0.5, c.K.shape[:3] + (1,), torch.arange(D, device="cuda")
    if kind == "small V":
        c.V *= 1e-38
    elif kind == "V by channel":  # 2^-145 to 2^109
        c.V.copy_(torch.ldexp(c.V.float(), 2 * channels - 145))
    elif kind == "V by row":  # 2^-140 to 2^-90, so that only some tiles are small
        c.V.copy_(torch.ldexp(c.V.float(), torch.randint(-140, -90, rows, generator=gen, device="cuda")))
    elif kind == "large V":  # rows of the largest value, with weights that all but vanish
        top = torch.finfo(DT[dtype]).max
        c.q.copy_(torch.full_like(c.q, 1.0))
        pick = (torch.rand(rows, generator=gen, device="cuda") < 0.2) & c.K.isfinite()
        c.V.copy_(torch.where(pick, torch.sign(c.V) * top, c.V))
        c.K.copy_(torch.where(pick, torch.full_like(c.K, -4.0), c.K))
    elif kind == "V with zeros":
        c.V.copy_(torch.where((channels >= 96) & c.V.isfinite(), torch.zeros_like(c.V), c.V))
    elif kind == "K against q":  # products near 1 of factors from 2^-120 to 2^120
        e = (channels * 53) % 241 - 120
        c.K.copy_(torch.ldexp(c.K.float(), e))
        c.q.copy_(torch.ldexp(c.q.float(), -e))
    elif kind == "K large":  # the largest values against zeros and tiny ones
        c.K.copy_(torch.where((channels % 3 == 0) & c.K.isfinite(), torch.full_like(c.K, torch.finfo(DT[dtype]).max), c.K))
        c.q.copy_(torch.where(channels % 3 == 0, torch.where(channels % 2 == 0, 0.0, 2.0 ** -126), c.q.float()))
    elif kind == "q large":
        c.q.copy_(torch.where(channels % 3 == 0, torch.full_like(c.q, torch.finfo(DT[dtype]).max), c.q))
        c.K.copy_(torch.where((channels % 3 == 0) & c.K.isfinite(), c.K.float() * 2.0 ** -127, c.K.float()))
    else:  # a large scale over small operands
        c.K.copy_(torch.ldexp(c.K.float(), torch.tensor(-40, device="cuda")))
        c.q.copy_(torch.ldexp(c.q.float(), torch.tensor(-60, device="cuda")))
        scale = 2.0 ** 97
    mass = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=mass, scale=scale)
    torch.cuda.synchronize()
    out, lse, q = (x.double().cpu().numpy() for x in (c.out, c.lse, c.q))
    for s, n in enumerate(c.lens_list):
        for h in range(c.heads):
            k, v, ok = c.rows(s, h)
            at = slice(h * g, (h + 1) * g)
            o, z, w = po.attend(q[s, at], k, v, ok, scale)
            es = 2.0 ** -16 * scale * (np.abs(q[s, at]) @ np.abs(k).T).max()
            sums = 2.0 ** -23 * (n / 16 + 200)
            eps = 4 * es + 2.0 ** -16 + 2 * sums
            p = np.exp(scale * (q[s, at] @ k.T) - z[:, None])
            bound = eps * (p @ np.abs(v)) + (2 * n + 16) * 2.0 ** -149
            assert (np.abs(out[s, at] - o) <= bound).all()
            assert (np.abs(lse[s, at] - z) <= 2 * es + 2.0 ** -19 + sums + 2.0 ** -23 * np.abs(z)).all()
            assert (np.abs(mass[s, h, :n].double().cpu().numpy() - w) <= eps * w + 2.0 ** -23 * w + 1e-30).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_and_lengths_are_reported(dtype):
    """A bad page id drops its rows, a bad length is clamped; both are reported,
    and the other sequences' results stand."""
    c = Case([100, 64, 40], 2, 4, 16, dtype, width=7)
    c.table[0, 2], c.table[0, 5] = -1, c.n_pages
    c.handle.decode_attn(c.q, c.out, lse=c.lse)
    torch.cuda.synchronize()
    assert int(c.err) == 2  # bad index
    c.check_attention()
    c = Case([112, 64, 40], 2, 4, 16, dtype, width=7)
    c.lens[0], c.lens[2] = 5000, -3
    c.lens_list = [112, 64, 0]
    c.handle.decode_attn(c.q, c.out, lse=c.lse)
    torch.cuda.synchronize()
    assert int(c.err) == 3  # bad count
    c.check_attention()


@pytest.mark.parametrize("lens,width", [([100, 64, 300], 24), ([5000, 64, 7000], 440)])
@pytest.mark.parametrize("dtype,g", [("bf16", 4), ("bf16", 16), ("f32", 2), ("f32", 7), ("f32", 12)])
@pytest.mark.parametrize("bad", ["some", "all of one", "all"])
def test_bad_pages_with_weights(lens, width, dtype, g, bad):
    """Rows of bad pages weigh nothing, and a unit that has no others leaves its
    weights as they were: in the attention kernel (short capacity), in the kernel
    behind it and through the merge across CTAs, on a workspace that still has
    the scores of a call with good pages."""
    c = Case(lens, 2, g, 16, dtype, width=width)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=torch.zeros_like(c.mass))
    pages = [-(-n // 16) for n in lens]
    if bad == "some":
        for s, n in enumerate(pages):
            c.table[s, :n:3] = -1
            c.table[s, n // 2] = c.n_pages
    else:
        for s in [0] if bad == "all of one" else [0, 1, 2]:
            c.table[s, :pages[s]] = -7
    before = c.mass.clone()
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_in=c.mass, mass_out=c.mass)
    torch.cuda.synchronize()
    assert int(c.err) == 2
    host = before.double().cpu().numpy()
    c.check_attention(mass_in=host, mass_out=c.mass, mass_before=host)
    for s, n in enumerate(lens):
        ok = torch.tensor(c.rows(s, 0)[2])
        assert torch.equal(c.mass[s, :, :n].cpu()[:, ~ok], before[s, :, :n].cpu()[:, ~ok])
        assert ok.any() == (bad == "some" or (bad == "all of one" and s != 0))


@pytest.mark.parametrize("dtype,n,heads,g,page", [("bf16", 70001, 2, 4, 64), ("f32", 30011, 1, 7, 16),
                                                  ("bf16", 131071, 1, 16, 128), ("f32", 20003, 2, 12, 32)])
def test_long_sequences(dtype, n, heads, g, page):
    """Against torch in float64 on the GPU; besides the bounds, the relative
    2-norm of the error: the rounding of a score (|s| below 8, some hundred
    roundings of 2^-24 relative each, random) is the largest part, about 5e-6."""
    c = Case([n, 13], heads, g, page, dtype, "phd")
    mass = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=mass)
    torch.cuda.synchronize()
    pages = c.table[0, :-(-n // page)].long()
    for h in range(heads):
        k = c.K[pages, h].reshape(-1, D)[:n].double()
        v = c.V[pages, h].reshape(-1, D)[:n].double()
        s = c.q[0, h * g:(h + 1) * g].double() @ k.T / math.sqrt(D)
        p = torch.softmax(s, dim=1)
        want, got = p @ v, c.out[0, h * g:(h + 1) * g].double()
        assert float((got - want).norm() / want.norm()) <= 1e-5
        assert float((mass[0, h, :n].double() - p.sum(0)).norm() / p.sum(0).norm()) <= 1e-5
        assert torch.allclose(c.lse[0, h * g:(h + 1) * g].double(), torch.logsumexp(s, 1), rtol=0, atol=1e-5)
    assert not mass[0, :, n:].any() and not mass[1, :, 13:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """Pages more than 2^32 bytes and 2^31 elements into their pools."""
    heads, page, n_pages = 8, 128, 20000  # 2.6e9 elements
    K = torch.empty(n_pages, heads, page, D, dtype=DT[dtype], device="cuda")
    V = torch.empty_like(K)
    ids = torch.tensor([[19999, 3, 19998, 16500]], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    for p in ids[0].tolist():
        K[p] = torch.randn(heads, page, D, generator=gen, device="cuda").to(DT[dtype])
        V[p] = torch.randn(heads, page, D, generator=gen, device="cuda").to(DT[dtype])
    lens = torch.tensor([400], dtype=torch.int32, device="cuda")
    R = 512
    mass = torch.rand(1, heads, R, generator=gen, device="cuda")
    pos = torch.arange(R, dtype=torch.int32, device="cuda").expand(1, heads, R).contiguous()
    seen = lens.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = ckv.PagedCache(K, V, ids, lens, g=4, mass=mass, pos=pos, seen=seen, dev_err=err)
    q = torch.randn(1, heads * 4, D, generator=gen, device="cuda").to(DT[dtype])
    out = torch.empty(1, heads * 4, D, device="cuda")

    def want(n):
        k = K[ids[0].long()].transpose(0, 1).reshape(heads, R, D)[:, :n].double()
        v = V[ids[0].long()].transpose(0, 1).reshape(heads, R, D)[:, :n].double()
        s = torch.matmul(q.view(heads, 4, D).double(), k.transpose(1, 2)) / math.sqrt(D)
        return torch.matmul(torch.softmax(s, -1), v).view(1, heads * 4, D)

    cache.decode_attn(q, out)
    assert float((out.double() - want(400)).norm() / want(400).norm()) <= 1e-5
    new = torch.randn(1, heads, 100, D, generator=gen, device="cuda").to(DT[dtype])
    cache.append(new, new)
    assert int(lens) == 500 and torch.equal(K[19998, :, 127], K[19998, :, 127])
    assert torch.equal(K[16500, :, 16:116], new[0]) and torch.equal(V[16500, :, 16:116], new[0])
    moves = torch.zeros(1, heads, 300, 2, dtype=torch.int32, device="cuda")
    n_moves = torch.zeros(1, heads, dtype=torch.int32, device="cuda")
    before = K[ids[0].long()].transpose(0, 1).reshape(heads, R, D).clone()
    cache.evict(300, 4, 100, moves, n_moves)
    after = K[ids[0].long()].transpose(0, 1).reshape(heads, R, D)
    for h in range(heads):
        m = moves[0, h, :int(n_moves[0, h])].long()
        assert len(m) >= 100 and torch.equal(after[h, m[:, 1]], before[h, m[:, 0]])
    cache.decode_attn(q, out)
    assert float((out.double() - want(300)).norm() / want(300).norm()) <= 1e-5
    assert int(err) == 0


@pytest.mark.parametrize("lens,heads", [([900, 64, 2500, 0, 33], 4), ([20, 300, 0, 129], 2), ([9000], 1), ([8], 1)])
@pytest.mark.parametrize("dtype,g", [("bf16", 4), ("bf16", 16), ("f32", 2), ("f32", 8), ("f32", 12)])
def test_a_wait_that_runs_out_is_reported(lens, heads, dtype, g):
    """Every other warp leaves out its first copy and gives up waiting for it
    after about a millisecond, in units of a CTA's own and in units that CTAs
    share: the error word says so, the arrival counters are zero again, and the
    next call on the handle is right."""
    c = Case(lens, heads, g, 16, dtype)
    mass = torch.zeros_like(c.mass)
    ckv.paged_set_wait_limit(2_000_000, stall=True)
    try:
        c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=mass)
        torch.cuda.synchronize()
    finally:
        ckv.paged_set_wait_limit()
    stalled = max(lens) * heads * len(lens) > 16  # one tile: one warp, and it is not an odd one
    assert int(c.err) == (1 if stalled else 0)
    assert not c.handle.workspace[:1024].any()
    c.err.zero_()
    mass.zero_()
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=mass)
    torch.cuda.synchronize()
    assert int(c.err) == 0 and not c.handle.workspace[:1024].any()
    c.check_attention(mass_out=mass, mass_before=np.zeros(mass.shape))


def test_results_do_not_change_from_run_to_run():
    c = Case([3000, 1, 0, 777, 2048], 3, 5, 16, "bf16")
    first = None
    for _ in range(5):
        mass = torch.zeros_like(c.mass)
        c.out.fill_(float("nan"))
        c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=mass)
        got = (c.out.clone(), c.lse.clone(), mass)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_two_handles_and_graphs_at_once():
    """Two captured graphs over one cache, each with its own handle, replayed on
    two streams at the same time, and new lengths written between replays."""
    c = Case([900, 64, 2500, 0], 4, 4, 16, "bf16", width=200)
    other = c.make()
    out2, lse2 = torch.empty_like(c.out), torch.empty_like(c.lse)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    torch.cuda.synchronize()
    for st, (handle, out, lse) in zip(streams, ((c.handle, c.out, c.lse), (other, out2, lse2))):
        with torch.cuda.stream(st):
            handle.decode_attn(c.q, out, lse=lse)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            handle.decode_attn(c.q, out, lse=lse)
        graphs.append(graph)
    for lens in ([900, 64, 2500, 0], [1, 63, 2499, 0], [0, 0, 16, 0]):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.lens_list = lens
        torch.cuda.synchronize()
        for _ in range(20):
            for st, graph in zip(streams, graphs):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        c.check_attention()
        assert torch.equal(c.out, out2) and torch.equal(c.lse, lse2)


@pytest.mark.parametrize("lens", [[900, 64, 2500, 0], [300, 1, 0, 384]])
def test_weights_in_two_graphs_at_once(lens):
    """Weights from two handles' graphs on two streams at the same time, added
    in place replay after replay, in the attention kernel (short capacity) and
    behind it."""
    c = Case(lens, 2, 3, 16, "bf16")
    mass = [torch.zeros_like(c.mass), torch.zeros_like(c.mass)]
    outs = [torch.empty_like(c.out), torch.empty_like(c.out)]
    one = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=one)
    torch.cuda.synchronize()
    c.check_attention(mass_out=one, mass_before=np.zeros(one.shape))
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, m, o in zip(streams, mass, outs):
        handle = c.make()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            handle.decode_attn(c.q, o, mass_in=m, mass_out=m)
        graphs.append((graph, handle))
    torch.cuda.synchronize()
    for _ in range(16):
        for st, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    # 16 additions of the same value, each rounded to half a unit in the last place
    assert torch.equal(mass[0], mass[1]) and torch.equal(outs[0], c.out) and torch.equal(outs[1], c.out)
    assert ((mass[0].double() - 16 * one.double()).abs() <= 16 * 2.0 ** -24 * 16 * one.double()).all()


def test_shared_pages():
    """Sequences that share a prefix's pages: each has its own weights."""
    c = Case([64, 80, 33], 2, 4, 16, "bf16", width=5)
    c.table[1, :4] = c.table[0, :4]
    c.table[2, :2] = c.table[0, :2]
    c.table[2, 2] = c.table[0, 2]
    mass = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=mass)
    torch.cuda.synchronize()
    c.check_attention(mass_out=mass, mass_before=np.zeros(mass.shape))


@pytest.mark.parametrize("dtype,g", [("bf16", 4), ("f32", 2)])
def test_a_slab_is_a_paged_cache(dtype, g):
    """The recallable path's [units][max_len][d] slabs under an identity table:
    the paged attention equals the sparse attention whose budget covers all."""
    from parity import ATTN_TOL, make_ctx
    units, max_len, L = 5, 640, 601
    gen = torch.Generator().manual_seed(2)
    K, V = (torch.randn(units, max_len, D, generator=gen).to(DT[dtype]).cuda() for _ in range(2))
    q = torch.randn(units, g, D, generator=gen).to(DT[dtype]).cuda()
    ctx = make_ctx(units, g, max_len, 8, max_len, dtype)
    ctx.cluster_prefill(K, L - 3, 7)
    idx = torch.zeros(units, max_len, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(units, dtype=torch.int32, device="cuda")
    want, got = (torch.zeros(units, g, D, device="cuda") for _ in range(2))
    ctx.decode_step(q, K, V, max_len, L, idx, cnt, want)
    cache = ckv.PagedCache(K.view(-1, 1, 64, D), V.view(-1, 1, 64, D),
                           torch.arange(units * 10, dtype=torch.int32, device="cuda").view(units, 10),
                           torch.full((units,), L, dtype=torch.int32, device="cuda"), g=g)
    cache.decode_attn(q, got)
    torch.cuda.synchronize()
    assert ctx.device_error() == 0
    assert (got - want).abs().max().item() <= ATTN_TOL[dtype]
    ctx.close()


def test_raw_calls_and_public_ones_agree():
    from types import SimpleNamespace as NS
    raw, public = ckv._raw_calls(torch), ckv._raw_calls(NS(_C=NS(), cuda=torch.cuda))
    for st in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(st):
            assert raw[0](0) == public[0](0) == st.cuda_stream and raw[1]() == public[1]() == 0


def test_side_stream_argument():
    c = Case([100, 20], 2, 4, 16, "bf16")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.handle.decode_attn(c.q, c.out, lse=c.lse, stream=st)
    st.synchronize()
    c.check_attention()


@pytest.mark.parametrize("how", ["argument", "current", "in a pool"])
def test_handle_dropped_with_work_queued_on_another_stream(how):
    """The workspace of a handle that dies while a side stream has yet to use it
    is not handed out on the stream that the handle was made on."""
    c = Case([900, 64, 2500, 0], 4, 4, 16, "bf16", width=200)
    want = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=want)
    mass, out = torch.zeros_like(c.mass), torch.zeros_like(c.out)
    handle, side = c.make(), torch.cuda.Stream()
    if how == "in a pool":  # the first call on the stream is captured, the second is not
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            handle.decode_attn(c.q, out, mass_out=mass)
    torch.cuda.synchronize()
    at, nbytes = handle.workspace.data_ptr(), handle.workspace.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some 0.2 s
    if how == "argument":
        handle.decode_attn(c.q, out, mass_out=mass, stream=side)
    else:
        with torch.cuda.stream(side):
            handle.decode_attn(c.q, out, mass_out=mass)
    del handle
    others = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()
    for t in others:
        assert not t.data_ptr() <= at < t.data_ptr() + nbytes
        t.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and torch.equal(mass, want)


def test_handle_made_on_a_side_stream_and_dropped_with_work_on_the_default_one():
    c = Case([900, 64, 2500, 0], 4, 4, 16, "bf16", width=200)
    want = torch.zeros_like(c.mass)
    c.handle.decode_attn(c.q, c.out, lse=c.lse, mass_out=want)
    mass, out, side = torch.zeros_like(c.mass), torch.zeros_like(c.out), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        handle = c.make()
    at, nbytes = handle.workspace.data_ptr(), handle.workspace.numel()
    torch.cuda._sleep(400_000_000)  # some 0.2 s
    handle.decode_attn(c.q, out, mass_out=mass)
    del handle
    with torch.cuda.stream(side):
        others = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert not torch.cuda.default_stream().query()
        for t in others:
            assert not t.data_ptr() <= at < t.data_ptr() + nbytes
            t.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and torch.equal(mass, want)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,layout,page,heads,n", [
    ("bf16", "hpd", 16, 2, 1), ("f32", "phd", 16, 3, 1), ("bf16", "kv_in_page", 48, 8, 37), ("f32", "wide", 32, 1, 70),
    ("bf16", "phd", 64, 5, 500), ("f32", "hpd", 16, 2, 300)])
@pytest.mark.parametrize("given", [False, True])
def test_append(dtype, layout, page, heads, n, given):
    """Rows, positions and weights of the appended rows; nothing else changes,
    bit for bit, and a sequence that would overflow is left as it is."""
    lens = [0, 5, page, 2 * page + 1, 7]
    width = 3 + -(-n // page)
    c = Case([width * page] * 5, heads, 1, page, dtype, layout, garbage=0.0)
    c.lens.copy_(torch.tensor(lens))
    c.seen.copy_(torch.tensor([0, 105, page, 1000, 7]))
    counts = torch.tensor([n, max(0, n - 1), 0, n, n], dtype=torch.int32, device="cuda")
    start, first = c.lens.clone(), c.seen.clone()
    bad = 4
    if given:
        start = torch.tensor([3, 0, 1, page, width * page - n + 1], dtype=torch.int32, device="cuda")
        first = torch.tensor([9, 8, 7, 6, 5], dtype=torch.int32, device="cuda")
    else:
        start[bad] = c.lens[bad] = width * page - n + 1
    src = torch.randn(2, 5, n, heads, D).to(DT[dtype]).cuda()
    k, v = src[0].transpose(1, 2), src[1].transpose(1, 2)
    want = {x: getattr(c, x).clone() for x in ("K", "V", "mass", "pos", "lens", "seen")}
    for s in range(4):
        for j in range(int(counts[s])):
            r = int(start[s]) + j
            pg = int(c.table[s, r // page])
            want["K"][pg, :, r % page], want["V"][pg, :, r % page] = k[s, :, j], v[s, :, j]
            want["pos"][s, :, r], want["mass"][s, :, r] = int(first[s]) + j, 0.0
        want["lens"][s], want["seen"][s] = start[s] + counts[s], first[s] + counts[s]
    c.handle.append(k, v, counts=counts, start=start if given else None, first=first if given else None)
    torch.cuda.synchronize()
    for x, t in want.items():
        assert torch.equal(getattr(c, x), t), x
    assert int(c.err) == 3
    c.err.zero_()
    c.handle.append(k[:, :, :0].new_zeros(5, heads, 1, D), v[:, :, :1], counts=torch.zeros_like(counts))
    assert int(c.err) == 0 and torch.equal(c.lens, want["lens"]) and torch.equal(c.K, want["K"])


@pytest.mark.parametrize("dtype,n,heads", [("bf16", 1, 2), ("bf16", 300, 4), ("f32", 90, 8), ("bf16", 2000, 8)])
@pytest.mark.parametrize("start,first,counts", [("seen", "own", None), ("own", "lens", None), ("seen", "lens", None),
                                                ("lens", "own", "lens"), ("own", "own", "seen"), ("own", "own", "lens")])
def test_append_with_lens_and_seen_as_other_arguments(dtype, n, heads, start, first, counts):
    """start = seen, first = lens and counts = either: every block of a sequence
    takes the values from before the call, however many blocks it has."""
    page, S = 64, 6
    width = 2 + -(-2 * n // page)
    c = Case([width * page] * S, heads, 1, page, dtype, "hpd", garbage=0.0)
    c.lens.copy_(torch.tensor([0, 1, n, 5 % n, n // 2, n]))
    c.seen.copy_(torch.tensor([n, 0, 3 % n, 1, n, n // 3]))
    vec = {"lens": c.lens, "seen": c.seen, "own": torch.arange(S, dtype=torch.int32, device="cuda") % n, None: None}
    old = {k: None if t is None else t.cpu().clone() for k, t in vec.items()}
    src = torch.randn(2, S, heads, n, D).to(DT[dtype]).cuda()
    want = {x: getattr(c, x).clone() for x in ("K", "V", "mass", "pos")}
    cnt = [n] * S if counts is None else old[counts].tolist()
    for s in range(S):
        j = torch.arange(cnt[s], device="cuda")
        r = j + int(old[start][s])
        pg = c.table[s].long()[r // page]
        want["K"][pg, :, r % page], want["V"][pg, :, r % page] = (x[s, :, j].transpose(0, 1) for x in src)
        want["pos"][s][:, r], want["mass"][s][:, r] = (j + int(old[first][s])).int(), 0.0
    c.handle.append(src[0], src[1], counts=vec[counts], start=vec[start], first=vec[first])
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for x, t in want.items():
        assert torch.equal(getattr(c, x), t), x
    assert c.lens.tolist() == [int(a) + b for a, b in zip(old[start], cnt)]
    assert c.seen.tolist() == [int(a) + b for a, b in zip(old[first], cnt)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_far_into_the_pools_leaves_the_rest_alone(dtype):
    """Rows past 2^32 bytes into the pools: every other row of the page written,
    of its neighbours and of the sequence's other pages stays as it was."""
    heads, page, n_pages = 8, 128, 20000
    K = torch.empty(n_pages, heads, page, D, dtype=DT[dtype], device="cuda")
    V = torch.empty_like(K)
    ids = torch.tensor([[19999, 3, 19998, 16500]], dtype=torch.int32, device="cuda")
    near = [0, 1, 2, 3, 4, 16499, 16500, 16501, 19997, 19998, 19999]
    for pool in (K, V):
        for p in near:
            pool[p].normal_()
    lens = torch.tensor([400], dtype=torch.int32, device="cuda")
    want = [pool[near].clone() for pool in (K, V)]
    new = torch.randn(2, 1, heads, 100, D, device="cuda").to(DT[dtype])
    for w, x in zip(want, new):
        w[near.index(16500), :, 16:116] = x[0]
    ckv.PagedCache(K, V, ids, lens).append(new[0], new[1])
    assert int(lens) == 500
    assert all(torch.equal(pool[near], w) for pool, w in zip((K, V), want))


def test_append_bad_counts_and_pages():
    c = Case([64] * 4, 2, 1, 16, "bf16", garbage=0.0)
    c.lens.copy_(torch.tensor([-1, 0, 0, 8]))
    c.table[3, 1] = -5
    before = c.K.clone()
    k = torch.ones(4, 2, 12, D, dtype=torch.bfloat16, device="cuda")
    c.handle.append(k, k, counts=torch.tensor([1, -1, 13, 12], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(c.err) in (2, 3) and c.lens.tolist() == [-1, 0, 0, 20]
    pg = int(c.table[3, 0])
    before[pg, :, 8:] = 1
    assert torch.equal(c.K, before)


@pytest.mark.parametrize("given", [False, True])
def test_append_of_positions_past_the_largest(given):
    """A sequence whose positions would pass 2^31 - 1, or that starts below 0,
    is left as it is; one that ends there is not."""
    c = Case([64] * 4, 2, 1, 16, "bf16", garbage=0.0)
    c.lens.zero_()
    first = torch.tensor([2 ** 31 - 1, 2 ** 31 - 11, 2 ** 31 - 13, -1], dtype=torch.int32, device="cuda")
    if not given:
        c.seen.copy_(first)
    before = {x: getattr(c, x).clone() for x in ("K", "mass", "pos", "seen")}
    k = torch.ones(4, 2, 12, D, dtype=torch.bfloat16, device="cuda")
    c.handle.append(k, k, first=first if given else None)
    torch.cuda.synchronize()
    assert int(c.err) == 3 and c.lens.tolist() == [0, 0, 12, 0]
    before["K"][int(c.table[2, 0]), :, :12] = 1
    before["mass"][2, :, :12] = 0
    before["pos"][2, :, :12] = torch.arange(2 ** 31 - 13, 2 ** 31 - 1, device="cuda").int()
    before["seen"][2] = 2 ** 31 - 1
    for x, t in before.items():
        assert torch.equal(getattr(c, x), t), x


def test_append_without_row_state_and_from_pinned_memory():
    c = Case([32, 32], 2, 1, 16, "bf16", garbage=0.0)
    c.lens.zero_()
    plain = ckv.PagedCache(c.K, c.V, c.table, c.lens)
    k = torch.randn(2, 2, 20, D).to(torch.bfloat16).pin_memory()
    plain.append(k, k)
    torch.cuda.synchronize()
    assert c.lens.tolist() == [20, 20]
    for s in range(2):
        got = torch.cat([c.K[p] for p in c.table[s, :2].tolist()], dim=1)[:, :20]
        assert torch.equal(got.cpu(), k[s])


def test_append_broadcast_source():
    c = Case([32, 32], 4, 1, 16, "f32", garbage=0.0)
    c.lens.zero_()
    k = torch.randn(1, 1, 9, D, device="cuda").expand(2, 4, 9, D)
    c.handle.append(k, k)
    for s in range(2):
        assert torch.equal(c.K[int(c.table[s, 0]), :, :9], k[s])


# ---------------------------------------------------------------- eviction
def weights(kind, S, heads, R, gen):
    m = torch.exp(2 * torch.randn(S, heads, R, generator=gen))
    if kind == "equal":
        m.fill_(0.25)
    elif kind == "few":
        m = torch.randint(0, 3, m.shape, generator=gen).float()
    elif kind == "odd":
        pick = torch.randint(0, 8, m.shape, generator=gen)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-42, -1.5)):
            m[pick == i] = x
    elif kind == "close":  # differ in the lowest bits only
        m = (torch.full(m.shape, 1.5).view(torch.int32) + torch.randint(0, 40, m.shape, generator=gen)).int().view(torch.float32)
    return m


SELECT = [
    # lens, heads, page, budget, sinks, recent
    ([1344, 1025, 1024, 3], 2, 16, 1024, 16, 256),
    ([1, 2, 48, 96], 3, 48, 1, 0, 0),
    ([100, 97, 0], 1, 16, 96, 0, 96),
    ([100, 97, 0], 2, 16, 96, 96, 0),
    ([5000, 300, 4999], 2, 64, 257, 16, 100),
    ([2049, 1023], 1, 16, 40, 4, 4),
    ([70000], 1, 16, 30000, 16, 500),
    ([9001, 8000], 1, 48, 3001, 16, 500),
    ([400001], 1, 16, 1000, 16, 500),
    ([40000, 20000, 33, 39999], 2, 64, 5000, 16, 100),
    # the largest slices whose keys stay in shared memory: of a cluster of eight, of a CTA alone
    ([327001], 1, 16, 1000, 16, 500),
    ([40950] + [50] * 79, 1, 16, 3000, 16, 100),
    ([6000, 5999] * 20, 2, 16, 700, 16, 100),
]


@pytest.mark.parametrize("kind", ["plain", "equal", "few", "odd", "close"])
@pytest.mark.parametrize("lens,heads,page,budget,sinks,recent", SELECT)
def test_evict_select(lens, heads, page, budget, sinks, recent, kind):
    gen = torch.Generator().manual_seed(budget)
    S, width = len(lens), max(1, -(-max(lens) // page))
    R = width * page
    K = torch.zeros(1, heads, page, D, dtype=torch.bfloat16, device="cuda")
    mass = weights(kind, S, heads, R, gen)
    # as after earlier evictions: every row's position is its own, in no order
    pos = torch.stack([torch.stack([torch.randperm(R, generator=gen) for _ in range(heads)]) for _ in range(S)]).int()
    seen = torch.full((S,), R, dtype=torch.int32)
    most = max(0, min(budget, R - budget))
    moves = torch.full((S, heads, most, 2), -7, dtype=torch.int32, device="cuda")
    n_moves = torch.full((S, heads), -7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = ckv.PagedCache(K, K.clone(), torch.zeros(S, width, dtype=torch.int32, device="cuda"),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"), mass=mass.cuda(), pos=pos.cuda(),
                           seen=seen.cuda(), dev_err=err)
    cache.evict_select(budget, sinks, recent, moves, n_moves)
    got, n_got = moves.cpu().numpy(), n_moves.cpu().numpy()
    assert int(err) == 0
    for s, n in enumerate(lens):
        for h in range(heads):
            kept = po.keep(mass[s, h, :n].numpy(), pos[s, h, :n].numpy(), R, budget, sinks, recent)
            want = po.moves(kept, budget)
            assert n_got[s, h] == len(want)
            assert np.array_equal(got[s, h, :len(want)], want)
            assert (got[s, h, len(want):] == -7).all()


@pytest.mark.parametrize("kind", ["plain", "equal", "odd"])
@pytest.mark.parametrize("lens,heads,page,budget,sinks,recent,rows", [
    ([1344, 1025, 1024, 3], 2, 16, 1024, 16, 256, 33792),
    ([1344, 1025, 1024, 3], 2, 16, 1024, 16, 256, 131072),
    ([1344] * 40, 8, 16, 1024, 16, 256, 33792),
    ([70, 5000, 0, 41], 1, 64, 40, 4, 8, 131072),
    ([129, 128, 4097], 3, 48, 127, 0, 3, 48 * 1000),
    ([1344, 20000, 60], 1, 16, 50, 16, 20, 400000),
])
def test_evict_select_in_caches_wider_than_their_sequences(lens, heads, page, budget, sinks, recent, rows, kind):
    """Capacities that give a unit more CTAs, and longer ones, than its rows
    need; what is not held is NaN and must not count."""
    gen = torch.Generator().manual_seed(budget)
    S, width, most = len(lens), rows // page, min(budget, rows - budget)
    K = torch.zeros(1, heads, page, D, dtype=torch.bfloat16, device="cuda")
    longest = max(lens)
    few = weights(kind, S, heads, longest, gen)
    mass = torch.full((S, heads, rows), float("nan"), device="cuda")
    pos = torch.zeros(S, heads, rows, dtype=torch.int32, device="cuda")  # of rows not held: protected, if they counted
    held_pos = torch.stack([torch.randperm(longest, generator=gen).int() for _ in range(S * heads)]).view(S, heads, -1)
    mass[:, :, :longest], pos[:, :, :longest] = few.cuda(), held_pos.cuda()
    for s, n in enumerate(lens):
        mass[s, :, n:], pos[s, :, n:] = float("nan"), 0
    moves = torch.full((S, heads, most, 2), -7, dtype=torch.int32, device="cuda")
    n_moves = torch.full((S, heads), -7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = ckv.PagedCache(K, K.clone(), torch.zeros(S, width, dtype=torch.int32, device="cuda"),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"), mass=mass, pos=pos,
                           seen=torch.full((S,), longest, dtype=torch.int32, device="cuda"), dev_err=err)
    cache.evict_select(budget, sinks, recent, moves, n_moves)
    got, n_got = moves.cpu().numpy(), n_moves.cpu().numpy()
    assert int(err) == 0
    for s, n in enumerate(lens):
        for h in range(heads):
            kept = po.keep(few[s, h, :n].numpy(), held_pos[s, h, :n].numpy(), longest, budget, sinks, recent)
            want = po.moves(kept, budget)
            assert n_got[s, h] == len(want) and np.array_equal(got[s, h, :len(want)], want)
            assert (got[s, h, len(want):] == -7).all()


LONGEST = (43696, 49146)  # page size and pages of 2^31 - 32 rows, the last multiple of 16 that a cache takes


def longest_cache(rows_held, mass, pos, **kw):
    """One unit of 2^31 - 32 rows, every page of which is the same one."""
    page, width = LONGEST
    gen = torch.Generator(device="cuda").manual_seed(1)
    K, V = torch.randn(2, 1, 1, page, D, generator=gen, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([rows_held], dtype=torch.int32, device="cuda")
    return ckv.PagedCache(K, V, torch.zeros(1, width, dtype=torch.int32, device="cuda"), lens, mass=mass, pos=pos,
                          seen=lens.clone(), dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"), **kw)


@pytest.mark.parametrize("short", [0, 1, 900])
def test_evict_select_of_the_longest_cache(short):
    """2^31 - 32 rows, the last CTA's slice of which ends within 2^10 of 2^31:
    planted rows, protected rows and, all others being equal, the lowest."""
    R, budget, sinks, recent = LONGEST[0] * LONGEST[1], 1000, 16, 50
    assert R == 2 ** 31 - 32
    n = R - short
    rng = np.random.default_rng(short)
    planted = np.unique(np.concatenate([rng.integers(0, n, 600), n - 1 - rng.integers(0, 4000, 150),
                                        rng.integers(0, 1500, 100)]))
    mass = torch.full((1, 1, R), 0.5, device="cuda")
    mass[0, 0, torch.tensor(planted, device="cuda")] = 1 + torch.rand(len(planted), device="cuda")
    mass[0, 0, n:] = 9.0  # not held
    pos = torch.arange(R, dtype=torch.int32, device="cuda").view(1, 1, R)
    cache = longest_cache(n, mass, pos)
    moves = torch.full((1, 1, budget, 2), -7, dtype=torch.int32, device="cuda")
    n_moves = torch.full((1, 1), -7, dtype=torch.int32, device="cuda")
    cache.evict_select(budget, sinks, recent, moves, n_moves)
    kept = set(planted.tolist()) | set(range(sinks)) | set(range(n - recent, n))
    row = 0
    while len(kept) < budget:
        kept.add(row)
        row += 1
    movers = sorted(r for r in kept if r >= budget)
    holes = [r for r in range(budget) if r not in kept]
    assert int(cache.dev_err) == 0 and int(n_moves) == len(movers) == len(holes)
    assert moves[0, 0, :len(movers)].tolist() == [list(x) for x in zip(movers, holes)]
    assert (moves[0, 0, len(movers):] == -7).all()


@pytest.mark.parametrize("short", [0, 5])
def test_attention_and_weights_of_the_longest_cache(short):
    """2^31 - 32 rows in 49146 pages that are all the same one: a row's weight
    is that of its slot, and the output that of one page, but for the last rows
    (relative bounds as above: n / 16 + 200 steps, of which a warp takes 2^17
    and the joining some hundred, |s| below 8)."""
    page, width = LONGEST
    R = page * width
    n = R - short
    mass = torch.full((1, 1, R), 2.0 ** -31, device="cuda")
    cache = longest_cache(n, mass, None, g=2)
    q = torch.randn(1, 2, D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros(1, 2, D, device="cuda"), torch.zeros(1, 2, device="cuda")
    cache.decode_attn(q, out, lse=lse, mass_in=mass, mass_out=mass)
    torch.cuda.synchronize()
    assert int(cache.dev_err) == 0
    k, v = cache.K[0, 0].double(), cache.V[0, 0].double()
    s = q[0].double() @ k.T / math.sqrt(D)
    times = torch.full((page,), float(width), dtype=torch.float64, device="cuda")
    times[page - short:] -= 1
    e = torch.exp(s) * times
    z = torch.log(e.sum(1))
    eps = 2.0 ** -23 * (2 ** 17 + 1000) + 2.0 ** -14
    assert ((lse[0].double() - z).abs() <= eps).all()
    p = e / e.sum(1, keepdim=True)
    assert ((out[0].double() - p @ v).abs() <= 2 * eps * (p @ v.abs())).all()
    want = 2.0 ** -31 + torch.exp(s - z[:, None]).sum(0)
    got = mass[0, 0].view(width, page)
    for i in range(0, width, 4096):
        held = torch.ones(min(4096, width - i), page, dtype=torch.bool, device="cuda")
        if i + 4096 >= width and short:
            held[-1, page - short:] = False
        part = got[i:i + 4096].double()
        assert ((part - want).abs() <= 2 * eps * want)[held].all()
        assert (part[~held] == 2.0 ** -31).all()


@pytest.mark.parametrize("dtype,layout,page,heads", [("bf16", "hpd", 16, 2), ("f32", "phd", 48, 3),
                                                     ("bf16", "kv_in_page", 64, 1), ("f32", "wide", 16, 2)])
def test_evict_apply(dtype, layout, page, heads):
    lens, budget = [200, 130, 100, 0, 131], 130
    c = Case(lens, heads, 1, page, dtype, layout, width=-(-200 // page), garbage=0.0)
    R = c.R
    most = min(budget, R - budget)
    moves = torch.zeros(5, heads, most, 2, dtype=torch.int32)
    n_moves = torch.zeros(5, heads, dtype=torch.int32)
    rng = np.random.default_rng(0)
    want = {x: getattr(c, x).clone() for x in ("K", "V", "mass", "pos")}
    for s, n in enumerate(lens):
        for h in range(heads):
            m = min(max(0, n - budget), most, 1 + 30 * h + 40 * (s == 0))
            src = np.sort(rng.choice(np.arange(budget, max(n, budget)), m, replace=False)) if m else np.zeros(0, int)
            dst = np.sort(rng.choice(budget, m, replace=False))
            n_moves[s, h] = m
            for i, (a, b) in enumerate(zip(src, dst)):
                moves[s, h, i, 0], moves[s, h, i, 1] = int(a), int(b)
                pa, pb = int(c.table[s, a // page]), int(c.table[s, b // page])
                want["K"][pb, h, b % page], want["V"][pb, h, b % page] = c.K[pa, h, a % page], c.V[pa, h, a % page]
                want["mass"][s, h, b], want["pos"][s, h, b] = c.mass[s, h, a], c.pos[s, h, a]
    for _ in range(2):  # repeating the call changes nothing
        c.handle.evict_apply(budget, moves.cuda(), n_moves.cuda())
        torch.cuda.synchronize()
        for x, t in want.items():
            assert torch.equal(getattr(c, x), t), x
        assert c.lens.tolist() == [130, 130, 100, 0, 130] and int(c.err) == 0


def test_eviction_of_nothing():
    """A budget that the whole capacity fits: no moves, and no room for any needed."""
    c = Case([64, 10], 2, 1, 16, "bf16", garbage=0.0)
    moves = torch.zeros(2, 2, 0, 2, dtype=torch.int32, device="cuda")
    n_moves = torch.full((2, 2), 9, dtype=torch.int32, device="cuda")
    before = c.K.clone()
    c.handle.evict(64, 8, 8, moves, n_moves)
    assert not n_moves.any() and torch.equal(c.K, before) and c.lens.tolist() == [64, 10] and int(c.err) == 0


def test_evict_apply_skips_bad_moves():
    c = Case([64, 64], 1, 1, 16, "bf16", garbage=0.0)
    budget = 40
    bad = [(39, 3), (64, 3), (-1, 3), (50, 40), (50, -1), (60, 5)]
    moves = torch.zeros(2, 1, 24, 2, dtype=torch.int32)
    moves[0, 0, :6] = torch.tensor(bad)
    want = c.K.clone()
    t = c.table[0].tolist()
    want[t[0], 0, 5] = c.K[t[3], 0, 12]
    c.handle.evict_apply(budget, moves.cuda(), torch.tensor([[6], [-4]], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(c.K, want) and int(c.err) in (2, 3) and c.lens.tolist() == [40, 40]


# ---------------------------------------------------------------- a run together
@pytest.mark.parametrize("dtype,heads,g,page", [("bf16", 2, 4, 16), ("f32", 3, 2, 32)])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_loop_with_eviction(dtype, heads, g, page, captured):
    """Prompts, then decode steps of append, attention with weights and, every
    few steps, eviction to a budget, eager and as replayed graphs.  The rows
    held are followed on the host by their token positions: every step's
    attention is compared with the oracle's over exactly those tokens, and the
    rows evicted must be the oracle's choice from the weights on the GPU."""
    gen = torch.Generator().manual_seed(5)
    S, budget, every, steps, sinks, recent = 3, 40, 8, 33, 4, 8
    prompt = [45, 1, 70]
    width = -(-(80 + every) // page)
    R = width * page
    tokens = 70 + steps
    tk, tv = (torch.randn(S, tokens, heads, D, generator=gen).to(DT[dtype]) for _ in range(2))
    qs = (1.5 * torch.randn(steps, S, heads * g, D, generator=gen)).to(DT[dtype])
    dev = "cuda"
    K = torch.full((S * width, heads, page, D), float("nan"), dtype=DT[dtype], device=dev)
    V = K.clone()
    table = torch.randperm(S * width, generator=gen).to(torch.int32).view(S, width).to(dev)
    lens, seen = (torch.zeros(S, dtype=torch.int32, device=dev) for _ in range(2))
    mass, pos = torch.zeros(S, heads, R, device=dev), torch.zeros(S, heads, R, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    cache = ckv.PagedCache(K, V, table, lens, g=g, mass=mass, pos=pos, seen=seen, dev_err=err)
    moves = torch.zeros(S, heads, budget, 2, dtype=torch.int32, device=dev)
    n_moves = torch.zeros(S, heads, dtype=torch.int32, device=dev)
    q, out, lse = qs[0].to(dev), torch.zeros(S, heads * g, D, device=dev), torch.zeros(S, heads * g, device=dev)
    k1, v1 = (torch.zeros(S, heads, 1, D, dtype=DT[dtype], device=dev) for _ in range(2))

    def step():
        cache.append(k1, v1)
        cache.decode_attn(q, out, lse=lse, mass_in=mass, mass_out=mass)

    def evict():
        cache.evict(budget, sinks, recent, moves, n_moves)

    longest = max(prompt)
    pk, pv = tk[:, :longest].transpose(1, 2).to(dev), tv[:, :longest].transpose(1, 2).to(dev)
    counts = torch.tensor(prompt, dtype=torch.int32, device=dev)
    run_step, run_evict = step, evict
    if captured:
        saved = [t.clone() for t in (K, V, lens, seen, mass, pos)]
        cache.append(pk, pv, counts=counts)
        graphs = []
        for fn in (step, evict):
            fn()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                fn()
            graphs.append(graph)
        run_step, run_evict = graphs[0].replay, graphs[1].replay
        for t, x in zip((K, V, lens, seen, mass, pos), saved):
            t.copy_(x)
        torch.cuda.synchronize()
    cache.append(pk, pv, counts=counts)
    held = [[list(range(n)) for _ in range(heads)] for n in prompt]  # token in each row
    for i in range(steps):
        tok = [n + i for n in prompt]
        k1.copy_(torch.stack([tk[s, tok[s]] for s in range(S)]).unsqueeze(2))
        v1.copy_(torch.stack([tv[s, tok[s]] for s in range(S)]).unsqueeze(2))
        q.copy_(qs[i])
        run_step()
        torch.cuda.synchronize()
        m_before = mass.cpu()
        for s in range(S):
            for h in range(heads):
                rows = held[s][h]
                rows.append(tok[s])
                assert int(lens[s]) == len(rows) and pos[s, h, :len(rows)].tolist() == rows
                kk, vv = tk[s, rows, h].double().numpy(), tv[s, rows, h].double().numpy()
                qq = qs[i, s, h * g:(h + 1) * g].double().numpy()
                o, z, _ = po.attend(qq, kk, vv, np.ones(len(rows), dtype=bool), D ** -0.5)
                got = out[s, h * g:(h + 1) * g].double().cpu().numpy()
                assert np.abs(got - o).max() <= 2e-3 * np.abs(vv).max()
                assert np.linalg.norm(got - o) <= 1e-5 * np.linalg.norm(o)
                assert np.abs(lse[s, h * g:(h + 1) * g].double().cpu().numpy() - z).max() <= 1e-5
        if i % every == every - 1:
            run_evict()
            torch.cuda.synchronize()
            for s in range(S):
                for h in range(heads):
                    rows = held[s][h]
                    kept = po.keep(m_before[s, h, :len(rows)].numpy(), np.array(rows), tok[s] + 1, budget, sinks, recent)
                    for a, b in po.moves(kept, budget):
                        rows[b] = rows[a]
                    del rows[budget:]
                    assert int(lens[s]) == len(rows)
    assert int(err) == 0
    # the weights of a row sum to g per step over the rows held
    assert (mass >= 0).all()


@pytest.mark.parametrize("dtype,heads,g,page,prompt,budget,rows", [
    ("bf16", 2, 4, 16, [45, 1, 70], 40, 96), ("f32", 3, 2, 32, [45, 1, 70], 40, 96), ("f32", 1, 12, 16, [45, 1, 70], 40, 96),
    ("bf16", 2, 4, 16, [700, 300, 1], 250, 1024), ("f32", 1, 8, 64, [700, 300, 1], 250, 1024)])
@pytest.mark.parametrize("captured", [False, True])
def test_accumulated_weights_follow_their_tokens(dtype, heads, g, page, prompt, budget, rows, captured):
    """The weight of every token held, added up on the host from the oracle's
    weights step by step, against the cache's: over appends (a new row starts
    from zero, also in a slot that an evicted row had), attention in place, in
    the attention kernel and behind it, and evictions (a weight moves with its
    row).  A step is off by eps times what it adds (the bounds at the top of
    this file) and rounds the sum to half a unit in the last place."""
    gen = torch.Generator().manual_seed(11)
    S, every, steps, sinks, recent, dev = len(prompt), 6, 20, 4, 8, "cuda"
    width = rows // page
    tokens = max(prompt) + steps
    tk, tv = (torch.randn(S, tokens, heads, D, generator=gen).to(DT[dtype]) for _ in range(2))
    qs = (1.5 * torch.randn(steps, S, heads * g, D, generator=gen)).to(DT[dtype])
    K = torch.full((S * width, heads, page, D), float("nan"), dtype=DT[dtype], device=dev)
    V = K.clone()
    table = torch.randperm(S * width, generator=gen).to(torch.int32).view(S, width).to(dev)
    lens, seen = (torch.zeros(S, dtype=torch.int32, device=dev) for _ in range(2))
    mass = torch.full((S, heads, rows), 99.0, device=dev)
    pos, err = torch.zeros(S, heads, rows, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    cache = ckv.PagedCache(K, V, table, lens, g=g, mass=mass, pos=pos, seen=seen, dev_err=err)
    moves = torch.zeros(S, heads, budget, 2, dtype=torch.int32, device=dev)
    n_moves = torch.zeros(S, heads, dtype=torch.int32, device=dev)
    q, out = qs[0].to(dev), torch.zeros(S, heads * g, D, device=dev)
    k1, v1 = (torch.zeros(S, heads, 1, D, dtype=DT[dtype], device=dev) for _ in range(2))

    def step():
        cache.append(k1, v1)
        cache.decode_attn(q, out, mass_in=mass, mass_out=mass)

    def evict():
        cache.evict(budget, sinks, recent, moves, n_moves)

    run_step, run_evict = step, evict
    if captured:  # nothing runs while it is captured
        graphs = []
        for fn in (step, evict):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                fn()
            graphs.append(graph)
        run_step, run_evict = graphs[0].replay, graphs[1].replay
    longest = max(prompt)
    cache.append(tk[:, :longest].transpose(1, 2).to(dev), tv[:, :longest].transpose(1, 2).to(dev),
                 counts=torch.tensor(prompt, dtype=torch.int32, device=dev))
    held = [[list(range(n)) for _ in range(heads)] for n in prompt]  # token in each row
    want, off = np.zeros((S, heads, tokens)), np.zeros((S, heads, tokens))  # weight of a token, and its bound
    for i in range(steps):
        k1.copy_(torch.stack([tk[s, n + i] for s, n in enumerate(prompt)]).unsqueeze(2))
        v1.copy_(torch.stack([tv[s, n + i] for s, n in enumerate(prompt)]).unsqueeze(2))
        q.copy_(qs[i])
        run_step()
        got = mass.double().cpu().numpy()
        for s in range(S):
            for h in range(heads):
                at = held[s][h]
                at.append(prompt[s] + i)
                kk, vv = tk[s, at, h].double().numpy(), tv[s, at, h].double().numpy()
                qq = qs[i, s, h * g:(h + 1) * g].double().numpy()
                _, _, w = po.attend(qq, kk, vv, np.ones(len(at), dtype=bool), D ** -0.5)
                es = 2.0 ** -16 * D ** -0.5 * (np.abs(qq) @ np.abs(kk).T).max()
                eps = 4 * es + 2.0 ** -16 + 2 * 2.0 ** -23 * (len(at) / 16 + 200)
                want[s, h, at] += w
                off[s, h, at] += eps * w + 2.0 ** -24 * want[s, h, at] * (1 + eps)
                assert abs(got[s, h, :len(at)].sum() - want[s, h, at].sum()) <= off[s, h, at].sum()
                assert (np.abs(got[s, h, :len(at)] - want[s, h, at]) <= off[s, h, at] + 1e-30).all(), (i, s, h)
                assert (got[s, h, max(len(at), max(prompt) + steps):] == 99.0).all()
        if i % every == every - 1:
            before = mass.cpu()
            run_evict()
            for s in range(S):
                for h in range(heads):
                    at = held[s][h]
                    kept = po.keep(before[s, h, :len(at)].numpy(), np.array(at), prompt[s] + i + 1, budget, sinks, recent)
                    for a, b in po.moves(kept, budget):
                        at[b] = at[a]
                    del at[budget:]
                    assert int(lens[s]) == len(at) and pos[s, h, :len(at)].tolist() == at
    assert int(err) == 0


def test_weights_added_call_after_call_on_one_stream():
    """Sixteen calls in a row that add in place, with nothing between them: each
    reads what the one before has written, also where it looks ahead."""
    for lens in ([900, 64, 2500, 0], [300, 1, 0, 384], [5000]):
        c = Case(lens, 2, 3, 16, "bf16")
        one, mass = torch.zeros_like(c.mass), torch.zeros_like(c.mass)
        c.handle.decode_attn(c.q, c.out, mass_out=one)
        torch.cuda.synchronize()
        for _ in range(16):
            c.handle.decode_attn(c.q, c.out, mass_in=mass, mass_out=mass)
        torch.cuda.synchronize()
        assert ((mass.double() - 16 * one.double()).abs() <= 16 * 2.0 ** -24 * 16 * one.double()).all()


# ---------------------------------------------------------------- refusals of the binding
def test_calls_refuse_wrong_tensors():
    c = Case([20, 3], 2, 4, 16, "bf16")
    h, i32 = c.handle, torch.int32
    with pytest.raises(ValueError):
        h.decode_attn(c.q[:, :4], c.out)
    with pytest.raises(TypeError):
        h.decode_attn(c.q.float(), c.out)
    with pytest.raises(ValueError):
        h.decode_attn(c.q.cpu(), c.out)
    with pytest.raises(TypeError):
        h.decode_attn(c.q, c.out.bfloat16())
    with pytest.raises(ValueError):
        h.decode_attn(c.q, c.out[:, :, :64])
    with pytest.raises(ValueError):
        h.decode_attn(c.q, c.out, lse=c.lse[:1])
    with pytest.raises(ValueError):
        h.decode_attn(c.q, c.out, mass_out=c.mass[:, :1])
    with pytest.raises(ckv.CKVError, match="ARG"):
        h.decode_attn(c.q, c.out, mass_in=c.mass)
    with pytest.raises(ckv.CKVError, match="ARG"):
        h.decode_attn(c.q, c.out, scale=float("nan"))
    with pytest.raises(ckv.CKVError, match="ARG"):
        h.decode_attn(c.q, None)
    bare = ckv.PagedCache(c.K, c.V, c.table, c.lens, g=4)
    with pytest.raises(ckv.CKVError, match="CAPACITY"):
        bare.decode_attn(c.q, c.out, mass_out=c.mass)
    with pytest.raises(ckv.CKVError, match="ARG"):
        ckv.PagedCache(c.K, c.V, c.table, c.lens, g=17)
    k = torch.zeros(2, 2, 3, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        h.append(k, k[:, :, :2])
    with pytest.raises(TypeError):
        h.append(k, k.float())
    with pytest.raises(ValueError):
        h.append(k, k.cpu())
    with pytest.raises(TypeError):
        h.append(k, k, counts=torch.ones(2, device="cuda"))
    with pytest.raises(ckv.CKVError, match="ARG"):
        h.append(k[:, :, :0], k[:, :, :0])
    moves, n = torch.zeros(2, 2, 8, 2, dtype=i32, device="cuda"), torch.zeros(2, 2, dtype=i32, device="cuda")
    with pytest.raises(ckv.CKVError, match="CAPACITY"):
        h.evict_select(16, 4, 4, moves, n)
    with pytest.raises(ckv.CKVError, match="ARG"):
        h.evict_select(24, 20, 8, moves, n)
    with pytest.raises(ValueError):
        h.evict_apply(24, moves[..., 0], n)
    with pytest.raises(TypeError):
        h.evict_apply(24, moves.long(), n)
    with pytest.raises(ckv.CKVError, match="ARG"):
        bare.evict_select(24, 4, 4, moves, n)
    torch.cuda.synchronize()
    assert torch.isnan(c.out).all()
