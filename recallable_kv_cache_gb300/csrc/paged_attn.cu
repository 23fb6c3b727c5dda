// Decode attention of one new token per sequence over a paged cache.
//
//   s_jr = scale q_j . K_r,  lse_j = ln sum_r e^{s_jr},  o_j = sum_r e^{s_jr - lse_j} V_r
//
// for the g query heads j that share a KV head, over its rows r < lens[s].
//
// Every held row is read once for all g heads, so the call is bound by HBM:
// 512 bytes a row (bf16) for 4 g 128 operations.  The rows of every (sequence,
// KV head), a unit, are cut into tiles; all tiles of the call, unit after
// unit, are dealt out evenly to the warps of a persistent grid (lens lives on
// the device, so every CTA derives the deal from it by a scan).  A warp streams
// its tiles through a ring of its own: one tensor-map copy (TMA) for the K
// rows of a tile and one for the V rows, a stage's mbarrier telling when both
// have landed; it keeps the running maximum and sum of the softmax and the
// unnormalised output in registers.  A tile never crosses a page (pages are
// multiples of 16 rows).  Where a unit ends inside the warp's share its result
// is final; the parts of a unit that several warps share are merged in tile
// order, first inside the CTA, then across CTAs by the one that finishes its
// part last, so the result does not depend on timing.  Where the accumulated
// weights are wanted the scores are left in the workspace, and
// paged_weights_kernel adds e^{s - lse}.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "mma_sync.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace ckv {
namespace paged {
namespace {

using namespace mmas;

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// A stage holds the K rows, then the V rows of one tile.  Eight warps with two
// stages each have 128 KB of an SM under way.  More of it lowers the rate (12
// warps of two stages: 90 instead of 87 us for one sequence of 128k rows and 8
// KV heads, 642 instead of 627 us for 32 of 32k rows), less does too (four of
// three: 104 and 744 us).
constexpr int STAGE = 8192;
constexpr int WARPS = 8, NST = 2;

// A cache of whose sequences the first skip[s] rows (a multiple of 16) are left
// out: they are attended elsewhere, together with those of other sequences.
struct OwnRows : Cache {
    const int32_t* skip;
    const int32_t* ctas;  // how many CTAs of the grid work: the others' SMs are taken
    // [seqs * heads] what the kernel behind finds of each unit with rows: n << 16 |
    // c, parts of CTAs c .. c + n - 1; n = 0: the result, in out and lse2
    int32_t* left;
};
// A cache in whose sequences a group's leading rows stand, which each attends by
// itself.  Its own or the group's rows, whichever are more, are looked up by every
// CTA into shared memory (0.5 us; by a kernel in front of this one 2).
struct GroupRows : Cache {
    Groups groups;
};
__device__ __forceinline__ int* rows_here() {
    __shared__ int rows[FEW_SEQS];
    return rows;
}
__device__ __forceinline__ int rows_held(const GroupRows&, int s) { return rows_here()[s]; }
template <int NT>
__device__ __forceinline__ void look_up_rows(const GroupRows& c) {
    __shared__ int first[FEW_GROUPS], end[FEW_GROUPS], shared[FEW_GROUPS];
    int* rows = rows_here();
    const int tid = threadIdx.x, n = c.groups.n;
    const bool reports = blockIdx.x == 0;
    int start = c.seqs, next = c.seqs, prefix = 0;
    if (tid < n) {
        start = c.groups.starts[tid];
        next = c.groups.starts[tid + 1];
        prefix = c.groups.prefix[tid];
        if (reports && (start < 0 || next > c.seqs || start > next || prefix < 0)) report(c.dev_err, CKV_DEV_BAD_COUNT);
    }
    for (int s = tid; s < c.seqs; s += NT) rows[s] = rows_held(static_cast<const Cache&>(c), s);
    __syncthreads();
    if (tid < 32) {
        // starts ascend: each is at least the largest before it
        int x = max(0, min(start, c.seqs));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, x, o);
            if (tid >= o) x = max(x, y);
        }
        const int e = max(x, min(next, c.seqs));
        first[tid] = x;
        end[tid] = e;
        shared[tid] = e - x > 1 ? min(max(prefix, 0), rows[x]) & ~(TILE - 1) : 0;
    }
    __syncthreads();
    for (int s = tid; s < c.seqs; s += NT) {
        int i = -1;  // the last group that begins at s or before
        for (int k = 0; k < n; ++k)
            if (first[k] <= s) i = k;
        if (i >= 0 && s < end[i] && shared[i] > rows[s]) {
            if (reports) report(c.dev_err, CKV_DEV_BAD_COUNT);
            rows[s] = shared[i];
        }
    }
    __syncthreads();
}
__device__ __forceinline__ int working_ctas(const Cache&) { return gridDim.x; }
__device__ __forceinline__ int working_ctas(const OwnRows& c) { return min((int)gridDim.x, max(1, *c.ctas)); }
__device__ __forceinline__ int first_row(const Cache&, int) { return 0; }
__device__ __forceinline__ int first_row(const OwnRows& c, int s) { return c.skip[s]; }
// rows to attend: those held from the first on
template <typename C>
__device__ __forceinline__ int rows_attended(const C& c, int s) {
    return max(0, rows_held(c, s) - first_row(c, s));
}

template <typename C>
struct AttnArgsOf {
    C c;
    const void* q;
    long long qst[2];  // element strides: sequence, query head
    int g;
    float qscale;  // scale * log2(e): scores are kept in base 2
    float* out;
    float* lse;
    const float* mass_in;
    float* mass_out;
    unsigned* arrived;  // [grid] CTAs that have left their part of the unit that begins in CTA i; zero between calls
    float* part;        // [grid][2] partials of units that several CTAs share
    float* lse2;        // [units][g], base 2
    float* scores;      // [units][g][rows], base 2
    int fuse;           // every unit has a CTA to itself, which adds its weights
    long long wait_limit;
    int stall;  // failure detection test: odd warps do not ask for their first tile
};

using AttnArgs = AttnArgsOf<Cache>;

// A partial: O [g][D], then the maxima [g], then the sums [g]; a multiple of
// 16 bytes, as O is read and written 16 bytes at a time.

// ---------------------------------------------------------------- the deal
template <int TR, typename C>
__device__ __forceinline__ int tiles_of(const C& c, int s) {
    return (rows_attended(c, s) + TR - 1) / TR;
}
struct Pos {
    int s, h, k, nt;  // nt = 0: past the last tile
};
// l tiles further on
template <int TR, typename C>
__device__ __forceinline__ Pos advance(const C& c, Pos p, int l) {
    p.k += l;
    while (p.nt && p.k >= p.nt) {
        p.k -= p.nt;
        if (++p.h == c.heads) {
            p.h = 0;
            do {
                ++p.s;
                p.nt = p.s < c.seqs ? tiles_of<TR>(c, p.s) : 0;
            } while (p.nt == 0 && p.s < c.seqs);
        }
    }
    return p;
}
// Merging across CTAs takes some 3 us, as long as two or three tiles of a warp.
// So where every unit can have a CTA to itself and the largest then has at most
// OWN_EXTRA tiles a warp more than in an even deal, it gets one: 128 units of
// 300 to 640 rows 11.1 instead of 14.2 us, 8 units of 200 rows 7.1 instead of
// 9.6, of 384 rows 8.2 instead of 8.5; of 512 rows 9.3 instead of 8.7, which
// the rule leaves to the even deal.
constexpr int OWN_EXTRA = 2;
// The deal of this call, and where the shares of CTA `cta`'s warps begin.  Every
// thread adds up a chunk of the sequences' tiles; a scan gives the total (below
// 2^31, checked for the cache's extents) and the thread in whose chunk a
// warp's first tile falls leaves the chunk's first sequence and how many tiles
// behind it the warp begins.  `cta` becomes the CTA's number in the deal.
template <int TR, int NT, typename C>
__device__ Deal deal_out(const C& c, int2* start, int& cta, int grid) {
    constexpr int NW = NT / 32;
    __shared__ int warp_sum[NW], warp_max[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = (c.seqs + NT - 1) / NT;
    const int s0 = tid * chunk, s1 = min(c.seqs, s0 + chunk);
    int v = 0, most = 0;
    for (int s = s0; s < s1; ++s) {
        const int n = tiles_of<TR>(c, s);
        v += n;
        most = max(most, n);
    }
    v *= c.heads;
    most = __reduce_max_sync(FULL, most);
    if (lane == 0) warp_max[warp] = most;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = x - v, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
        most = max(most, warp_max[w]);
    }
    if (c.seqs * c.heads <= grid && (most + NW - 1) / NW <= (total + grid * NW - 1) / (grid * NW) + OWN_EXTRA) {
        // CTA `cta` has unit `cta` to itself, with tiles numbered from 0
        int h;
        const int s = c.by_heads.quot(cta, &h);
        const int n = s < c.seqs ? tiles_of<TR>(c, s) : 0;
        const Deal own(n, 1, NW);
        if (tid < NW) start[tid] = make_int2(s, h * n + own.begin_warp(tid));
        __syncthreads();
        cta = 0;
        return own;
    }
    const Deal deal(total, Deal::ctas(total, NW, grid), NW);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int t = deal.begin_warp(cta * NW + w);
        if (t >= before && t < before + v) start[w] = make_int2(s0, t - before);
    }
    __syncthreads();
    return deal;
}
// the place of the tile that is `left` tiles behind the first of sequence s
template <int TR, typename C>
__device__ __forceinline__ Pos walk(const C& c, int s, int left) {
    int nt;
    while (left >= (nt = tiles_of<TR>(c, s)) * c.heads) {
        left -= nt * c.heads;
        ++s;
    }
    const int h = left / nt;
    return Pos{s, h, left - h * nt, nt};
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int c0, int c1, int c2, int c3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(ptx::smem_u32(dst)),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(ptx::smem_u32(dst)),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(ptx::smem_u32(bar))
        : "memory");
}

// ---------------------------------------------------------------- bf16 tiles on the tensor cores
// 16 rows a tile.  A tile lands as two halves of 64 channels, [half][row][128
// bytes], 128-byte swizzled (16-byte chunk c of row r at c ^ (r & 7)), which
// keeps ldmatrix free of bank conflicts.
//   S[h][r] = q[h] . K[r]        m16n8k16: M = heads (NB blocks of 8), N = 8 rows
//   O[c][h] += V[r][c] P[h][r]   M = 16 channels, N = 8 heads, K = 16 rows
// bf16 products are exact and add up in fp32.  P is fed to the second product
// as three bf16 terms (P = hi + mid + lo holds all 24 bits; with two, the
// outputs were off by 1.2e-6 of their norm, now 4e-7).  A tile's products start
// from zero and join O by ordinary additions: the tensor core truncates what
// it accumulates, and over the 290 tiles of a warp at 256 units of 32k rows
// that alone put the outputs off by 1.1e-5.
template <int NB>
struct TilesBf16 {
    using T = __nv_bfloat16;
    static constexpr int TR = 16, SCRATCH = 0;
    static constexpr bool SWIZZLED = true, CHECKED = false;
    uint32_t qa[8][2 * NB];
    float o[NB][8][4];
    float mrun[NB], lrun[NB];  // of head lane / 4 + 8 b

    static __device__ __forceinline__ void load(unsigned char* dst, const CUtensorMap* tk, const CUtensorMap* tv,
                                                int page, int h, int slot, uint64_t* bar) {
        tma_load_5d(dst, tk, 0, slot, 0, h, page, bar);
        tma_load_5d(dst + STAGE / 2, tv, 0, slot, 0, h, page, bar);
    }
    __device__ __forceinline__ void reset(const T* q, long long stride, int g, float, int lane) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int j = (lane >> 2) + 8 * b;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t* qp = reinterpret_cast<const uint32_t*>(q + j * stride + 16 * ks) + (lane & 3);
                qa[ks][b] = j < g ? qp[0] : 0u;
                qa[ks][NB + b] = j < g ? qp[4] : 0u;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][mt][e] = 0.f;
            mrun[b] = -INFINITY;
            lrun[b] = 0.f;
        }
    }
    // n of the stage's rows are held; the others' V rows must count as zero
    __device__ __forceinline__ void tile(unsigned char* stage, float2*, int n, float qscale, int g, float* scores,
                                         size_t rows, int lane) {
        const uint32_t kb = ptx::smem_u32(stage), vb = kb + STAGE / 2;
        if (n < TR) {
            for (int i = n * 16 + lane; i < TR * 16; i += 32)
                *reinterpret_cast<uint4*>(stage + STAGE / 2 + (i & 1) * 2048 + (i >> 4) * 128 + ((i >> 1) & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        float s[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int chunk = 4 * kk + (lane >> 3);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int row = nt * 8 + (lane & 7);
                uint32_t b0, b1, b2, b3;
                ldsm_x4(kb + (chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), b0, b1, b2, b3);
                mma(s[nt], qa[2 * kk][0], NB == 2 ? qa[2 * kk][NB - 1] : 0u, qa[2 * kk][NB],
                    NB == 2 ? qa[2 * kk][2 * NB - 1] : 0u, b0, b1);
                mma(s[nt], qa[2 * kk + 1][0], NB == 2 ? qa[2 * kk + 1][NB - 1] : 0u, qa[2 * kk + 1][NB],
                    NB == 2 ? qa[2 * kk + 1][2 * NB - 1] : 0u, b2, b3);
            }
        }
        const int r0 = (lane & 3) * 2;
        uint32_t ph[NB][2], pm[NB][2], pl[NB][2];
        float sc[NB];
        bool grew = false;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = r0 + (e & 1) + 8 * (e >> 1);
                v[e] = r < n ? s[e >> 1][2 * b + (e & 1)] * qscale : -INFINITY;
            }
            const int j = (lane >> 2) + 8 * b;
            if (scores && j < g) {
                float* sp = scores + (size_t)j * rows + r0;
                *reinterpret_cast<float2*>(sp) = make_float2(v[0], v[1]);
                *reinterpret_cast<float2*>(sp + 8) = make_float2(v[2], v[3]);
            }
            float tm = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
            tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, 1));
            tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, 2));
            const float mnew = fmaxf(mrun[b], tm);
            const float ms = mnew == -INFINITY ? 0.f : mnew;  // -inf - -inf is avoided: ex2(-inf) = 0
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = ex2(v[e] - ms);
            sc[b] = 1.f;
            if (mnew != mrun[b]) {
                sc[b] = ex2(mrun[b] - ms);
                grew = true;
            }
            lrun[b] = lrun[b] * sc[b] + ((p[0] + p[1]) + (p[2] + p[3]));
            mrun[b] = mnew;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ph[b][i] = pack2(p[2 * i], p[2 * i + 1]);
                const float x = p[2 * i] - lo_of(ph[b][i]), y = p[2 * i + 1] - hi_of(ph[b][i]);
                pm[b][i] = pack2(x, y);
                pl[b][i] = pack2(x - lo_of(pm[b][i]), y - hi_of(pm[b][i]));
            }
        }
        if (__any_sync(FULL, grew)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float sc0 = __shfl_sync(FULL, sc[b], (lane & 3) * 8);
                const float sc1 = __shfl_sync(FULL, sc[b], (lane & 3) * 8 + 4);
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                    o[b][mt][0] *= sc0;
                    o[b][mt][1] *= sc1;
                    o[b][mt][2] *= sc0;
                    o[b][mt][3] *= sc1;
                }
            }
        }
        const int vrow = ((lane >> 3) >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            const int chunk = 2 * mt + ((lane >> 3) & 1);
            uint32_t a0, a1, a2, a3;
            ldsm_x4_t(vb + (chunk >> 3) * 2048 + vrow * 128 + (((chunk & 7) ^ (vrow & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                mma(t, a0, a1, a2, a3, pl[b][0], pl[b][1]);
                mma(t, a0, a1, a2, a3, pm[b][0], pm[b][1]);
                mma(t, a0, a1, a2, a3, ph[b][0], ph[b][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][mt][e] += t[e];
            }
        }
        // the next copy into the stage must come after the zeros
        if (n < TR) ptx::fence_proxy_async_smem();
    }
    // O[j][c] (times w_j), maxima and sums to `put(j, c, value)`, `stat(j, m, l)`
    template <typename Put, typename Stat>
    __device__ __forceinline__ void leave(int g, int lane, bool normalise, Put put, Stat stat) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float l = lrun[b];
            l += __shfl_xor_sync(FULL, l, 1);
            l += __shfl_xor_sync(FULL, l, 2);
            const int j = (lane >> 2) + 8 * b;
            if ((lane & 3) == 0 && j < g) stat(j, mrun[b], l);
            const float w = !normalise ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            const float w0 = __shfl_sync(FULL, w, (lane & 3) * 8), w1 = __shfl_sync(FULL, w, (lane & 3) * 8 + 4);
            const int j0 = (lane & 3) * 2 + 8 * b;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const int c = 16 * mt + (lane >> 2);
                if (j0 < g) {
                    put(j0, c, o[b][mt][0] * w0);
                    put(j0, c + 8, o[b][mt][2] * w0);
                }
                if (j0 + 1 < g) {
                    put(j0 + 1, c, o[b][mt][1] * w1);
                    put(j0 + 1, c + 8, o[b][mt][3] * w1);
                }
            }
        }
    }
};

// ---------------------------------------------------------------- fp32 tiles
// Sums v[0 .. N) over L neighbouring lanes; every lane keeps N / L of the sums
// (one where N < L), those from the returned index on: each step halves what a
// lane still adds up, so a value costs about one shuffle instead of log2 L.
template <int N, int L>
__device__ __forceinline__ int reduce_scatter(float* v, int lane) {
    if constexpr (L > 1) {
        constexpr int d = L / 2;
        if constexpr (N > 1) {
            const bool up = lane & d;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float send = up ? v[i] : v[i + N / 2], keep = up ? v[i + N / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(FULL, send, d);
            }
            return (up ? N / 2 : 0) + reduce_scatter<N / 2, d>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(FULL, v[0], d);
            return reduce_scatter<1, d>(v, lane);
        }
    }
    return 0;
}

// 8 rows a tile, [row][512 bytes].  Scores: LPR lanes share a row (16 bytes a
// lane at a time, so eight lanes read 128 consecutive bytes) and add up their
// parts; the tile's scores go through a small array in shared memory, in which
// a lane then holds the values of one head, j = lane % GP.  Output: a lane owns
// 4 channels of every head, the weights come back as pairs (p, p).
template <int GP>
struct TilesF32 {
    using T = float;
    static constexpr int TR = 8, SCRATCH = TR * GP;
    static constexpr bool SWIZZLED = false, CHECKED = false;
    static constexpr int LPR = GP > 2 ? 16 : 8;  // lanes per row: q takes 128 / LPR * GP registers
    static constexpr int QV = 32 / LPR;          // float4 of a row per lane
    static constexpr int RP = 32 / LPR;          // rows at a time
    static constexpr int NV = (TR * GP + 31) / 32;
    uint64_t qv[GP][QV][2];
    uint64_t o[GP][2];
    float mrun, lrun;

    static __device__ __forceinline__ void load(unsigned char* dst, const CUtensorMap* tk, const CUtensorMap* tv,
                                                int page, int h, int slot, uint64_t* bar) {
        tma_load_4d(dst, tk, 0, slot, h, page, bar);
        tma_load_4d(dst + STAGE / 2, tv, 0, slot, h, page, bar);
    }
    __device__ __forceinline__ void reset(const T* q, long long stride, int g, float, int lane) {
#pragma unroll
        for (int j = 0; j < GP; ++j) {
#pragma unroll
            for (int i = 0; i < QV; ++i) {
                const float4 x = j < g ? *reinterpret_cast<const float4*>(q + j * stride + 4 * ((lane % LPR) + LPR * i))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                qv[j][i][0] = pair(x.x, x.y);
                qv[j][i][1] = pair(x.z, x.w);
            }
            o[j][0] = o[j][1] = 0;
        }
        mrun = -INFINITY;
        lrun = 0.f;
    }
    __device__ __forceinline__ void tile(unsigned char* stage, float2* ps, int n, float qscale, int g, float* scores,
                                         size_t rows, int lane) {
        const ulonglong2* K = reinterpret_cast<const ulonglong2*>(stage);
        const ulonglong2* V = reinterpret_cast<const ulonglong2*>(stage + STAGE / 2);
        float s[TR / RP * GP];
#pragma unroll
        for (int rr = 0; rr < TR / RP; ++rr) {
            const int row = rr * RP + lane / LPR;
            uint64_t acc[GP];
#pragma unroll
            for (int j = 0; j < GP; ++j) acc[j] = 0;
#pragma unroll
            for (int i = 0; i < QV; ++i) {
                const ulonglong2 k = K[row * 32 + (lane % LPR) + LPR * i];
#pragma unroll
                for (int j = 0; j < GP; ++j) acc[j] = fma2(qv[j][i][1], k.y, fma2(qv[j][i][0], k.x, acc[j]));
            }
#pragma unroll
            for (int j = 0; j < GP; ++j) {
                const float2 f = unpair(acc[j]);
                s[rr * GP + j] = f.x + f.y;
            }
        }
        const int x0 = reduce_scatter<TR / RP * GP, LPR>(s, lane % LPR);
        constexpr int KEPT = TR / RP * GP > LPR ? TR / RP * GP / LPR : 1;
#pragma unroll
        for (int i = 0; i < KEPT; ++i) ps[((x0 + i) / GP * RP + lane / LPR) * GP + (x0 + i) % GP].x = s[i];
        __syncwarp();
        const int j = lane % GP;
        float v[NV], tm = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int x = lane + 32 * i, r = x / GP;
            v[i] = x < TR * GP && r < n ? ps[x].x * qscale : -INFINITY;
            if (scores && x < TR * GP && j < g) scores[(size_t)j * rows + r] = v[i];
            tm = fmaxf(tm, v[i]);
        }
#pragma unroll
        for (int d = GP; d < 32; d <<= 1) tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, d));
        const float mnew = fmaxf(mrun, tm), ms = mnew == -INFINITY ? 0.f : mnew;
        const bool grew = mnew != mrun;
        const float sc = grew ? ex2(mrun - ms) : 1.f;
        lrun *= sc;
        mrun = mnew;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float p = ex2(v[i] - ms);
            lrun += p;
            if (lane + 32 * i < TR * GP) ps[lane + 32 * i] = make_float2(p, p);
        }
        if (__any_sync(FULL, grew)) {
#pragma unroll
            for (int jj = 0; jj < GP; ++jj) {
                const float w = __shfl_sync(FULL, sc, jj);
                const uint64_t ww = pair(w, w);
                o[jj][0] = fma2(o[jj][0], ww, 0);
                o[jj][1] = fma2(o[jj][1], ww, 0);
            }
        }
        __syncwarp();
        auto row = [&](int r) {
            const ulonglong2 vv = V[r * 32 + lane];
            const uint64_t* pp = reinterpret_cast<const uint64_t*>(ps + r * GP);
#pragma unroll
            for (int jj = 0; jj < GP; ++jj) {
                const uint64_t p = pp[jj];
                o[jj][0] = fma2(p, vv.x, o[jj][0]);
                o[jj][1] = fma2(p, vv.y, o[jj][1]);
            }
        };
        if (n == TR) {
#pragma unroll
            for (int r = 0; r < TR; ++r) row(r);
        } else {  // rows not held are not read
#pragma unroll 1
            for (int r = 0; r < n; ++r) row(r);
        }
    }
    template <typename Put, typename Stat>
    __device__ __forceinline__ void leave(int g, int lane, bool normalise, Put put, Stat stat) {
        float l = lrun;
#pragma unroll
        for (int d = GP; d < 32; d <<= 1) l += __shfl_xor_sync(FULL, l, d);
        if (lane < GP && lane < g) stat(lane, mrun, l);
        const float w = !normalise ? 1.f : (l == 0.f ? 0.f : 1.f / l);
#pragma unroll
        for (int j = 0; j < GP; ++j) {
            const float wj = __shfl_sync(FULL, w, j);
            if (j < g) {
                const float2 x = unpair(o[j][0]), y = unpair(o[j][1]);
                put(j, 4 * lane, x.x * wj);
                put(j, 4 * lane + 1, x.y * wj);
                put(j, 4 * lane + 2, y.x * wj);
                put(j, 4 * lane + 3, y.y * wj);
            }
        }
    }
};

// fp32 on the tensor cores, for more than eight heads (96 units of up to 12k
// rows, before the look at the range below: 16 heads 155 us where the tiles
// above took 207; 8 heads 115 where those take 100, so up to eight they are
// used).  Bound by dependent arithmetic on two warps a scheduler (40 % of the
// issue slots, the tensor pipe 40 % active).  Every operand is taken apart into
// three bf16 terms (hi + mid + lo, which hold its 24 bits), and of the nine
// products the six down to 2^-18 of the largest are added up, the small ones
// first.  bf16 ends at 2^-133, so that the terms of a value below 2^-110 leave
// a rest of up to 2^-134.  K's rests put a score, 128 products, off by 2^-127
// times the largest query value; a weight is at most 1, and fp32's exponential
// ends at 2^-126; but rests of V or q may be all there is.  So a warp keeps the
// least value of those that are not zero, and where that is below 2^-110, or a
// query value times the scale past 2^96, it does its tiles of the unit again in
// plain fp32 (16 heads above: 158 us without the least value, 163 with it, 181
// with a look at every tile's).  8 rows a tile, four quarters of 32 channels,
// [quarter][row][128 bytes], 128-byte swizzled (16-byte chunk c of row r at c ^ r).
//   S[h][r] = q[h] . K[r]        m16n8k16: M = 16 heads, N = 8 rows
//   O[c][h] += V[r][c] P[h][r]   m16n8k8:  M = 16 channels, N = 8 heads, K = 8 rows
// Which channel is which k of the first product, and which m of the second, is
// free; it is chosen so that a lane reads 16 bytes of a row at a time and the
// eight lanes that read together read different chunks: in step ks lane (n, t)
// reads chunk 2 t + ks % 2 of quarter ks / 2 of row n, and of V chunk n of
// quarter f of rows 2 t and 2 t + 1.
template <int NB>
struct TilesF32Tc {
    using T = float;
    static constexpr int TR = 8, SCRATCH = 0;
    static constexpr bool SWIZZLED = true, CHECKED = true;
    static constexpr uint32_t TINY = (17u << 24) - 1;  // order() of 2^-110
    uint32_t qa[3][8][2 * NB];
    float o[NB][8][4];
    float mrun[NB], lrun[NB];  // of head lane / 4 + 8 b
    uint32_t least;            // order() of the lane's V and q; 0: a query value is too large

    struct Terms {
        uint32_t t[3];  // hi, mid, lo of two values
    };
    // hi saturates: a value that would round to infinity leaves its rest to mid
    static __device__ __forceinline__ Terms split(float x, float y) {
        Terms r;
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r.t[0]) : "f"(y), "f"(x));
        x -= lo_of(r.t[0]);
        y -= hi_of(r.t[0]);
        r.t[1] = pack2(x, y);
        r.t[2] = pack2(x - lo_of(r.t[1]), y - hi_of(r.t[1]));
        return r;
    }
    // the order of magnitudes, zero the largest
    static __device__ __forceinline__ uint32_t order(float x) { return 2u * __float_as_uint(x) - 1u; }
    static __device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
        asm volatile(
            "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(b0));
    }
    static __device__ __forceinline__ void load(unsigned char* dst, const CUtensorMap* tk, const CUtensorMap* tv,
                                                int page, int h, int slot, uint64_t* bar) {
        tma_load_5d(dst, tk, 0, slot, 0, h, page, bar);
        tma_load_5d(dst + STAGE / 2, tv, 0, slot, 0, h, page, bar);
    }
    __device__ __forceinline__ void reset(const T* q, long long stride, int g, float qscale, int lane) {
        float most = 0.f;
        least = 0xffffffffu;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int j = (lane >> 2) + 8 * b;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const float4 x = j < g ? *reinterpret_cast<const float4*>(q + j * stride + 32 * (ks >> 1) +
                                                                          4 * (2 * (lane & 3) + (ks & 1)))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                const Terms u = split(x.x, x.y), v = split(x.z, x.w);
                most = fmaxf(fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
                least = min(min(least, min(order(x.x), order(x.y))), min(order(x.z), order(x.w)));
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    qa[i][ks][b] = u.t[i];
                    qa[i][ks][NB + b] = v.t[i];
                }
            }
        }
        if (!(most * fabsf(qscale) < 0x1p96f)) least = 0;
        clear();
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][mt][e] = 0.f;
            mrun[b] = -INFINITY;
            lrun[b] = 0.f;
        }
    }
    // the terms in the six products, the smallest first; the largest is the last
    static __host__ __device__ constexpr int left(int i) { return i == 1 ? 2 : (i == 2 || i == 3 ? 1 : 0); }
    static __host__ __device__ constexpr int right(int i) { return i == 0 ? 2 : (i == 2 || i == 4 ? 1 : 0); }

    // the weights p of a tile's rows 2 t + e from its scores s[2 b + e]; the
    // running maximum, the sum and O follow
    __device__ __forceinline__ void weigh(const float (&s)[4], int n, float qscale, int g, float* scores, size_t rows,
                                          int lane, float (&p)[NB][2]) {
        const int row = lane >> 2, t = lane & 3;
        float sc[NB];
        bool grew = false;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) v[e] = 2 * t + e < n ? s[2 * b + e] * qscale : -INFINITY;
            const int j = row + 8 * b;
            if (scores && j < g) *reinterpret_cast<float2*>(scores + (size_t)j * rows + 2 * t) = make_float2(v[0], v[1]);
            float tm = fmaxf(v[0], v[1]);
            tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, 1));
            tm = fmaxf(tm, __shfl_xor_sync(FULL, tm, 2));
            const float mnew = fmaxf(mrun[b], tm);
            const float ms = mnew == -INFINITY ? 0.f : mnew;
#pragma unroll
            for (int e = 0; e < 2; ++e) p[b][e] = ex2(v[e] - ms);
            sc[b] = 1.f;
            if (mnew != mrun[b]) {
                sc[b] = ex2(mrun[b] - ms);
                grew = true;
            }
            lrun[b] = lrun[b] * sc[b] + (p[b][0] + p[b][1]);
            mrun[b] = mnew;
        }
        if (__any_sync(FULL, grew)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float sc0 = __shfl_sync(FULL, sc[b], t * 8), sc1 = __shfl_sync(FULL, sc[b], t * 8 + 4);
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                    o[b][mt][0] *= sc0;
                    o[b][mt][1] *= sc1;
                    o[b][mt][2] *= sc0;
                    o[b][mt][3] *= sc1;
                }
            }
        }
    }
    __device__ __forceinline__ void tile(unsigned char* stage, float2*, int n, float qscale, int g, float* scores,
                                         size_t rows, int lane) {
        const int row = lane >> 2, t = lane & 3;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const float4 k = *reinterpret_cast<const float4*>(stage + (ks >> 1) * 1024 + row * 128 +
                                                              (((2 * t + (ks & 1)) ^ row) << 4));
            const Terms u = split(k.x, k.y), v = split(k.z, k.w);
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                const uint32_t(&a)[2 * NB] = qa[left(i)][ks];
                mma(i < 5 ? small : s, a[0], NB == 2 ? a[NB - 1] : 0u, a[NB], NB == 2 ? a[2 * NB - 1] : 0u,
                    u.t[right(i)], v.t[right(i)]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += small[e];
        float p[NB][2];
        weigh(s, n, qscale, g, scores, rows, lane, p);
        Terms p3[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) p3[b] = split(p[b][0], p[b][1]);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            float x[2][4];  // rows not held count as zero
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * t + e;
                const float4 v = *reinterpret_cast<const float4*>(stage + STAGE / 2 + f * 1024 + r * 128 + ((row ^ r) << 4));
                const bool held = r < n;
                x[e][0] = held ? v.x : 0.f;
                x[e][1] = held ? v.y : 0.f;
                x[e][2] = held ? v.z : 0.f;
                x[e][3] = held ? v.w : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) least = min(least, order(x[e / 4][e % 4]));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const Terms u = split(x[0][2 * half], x[1][2 * half]), v = split(x[0][2 * half + 1], x[1][2 * half + 1]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 6; ++i) mma8(d, u.t[left(i)], v.t[left(i)], p3[b].t[right(i)]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[b][2 * f + half][e] += d[e];
                }
            }
        }
    }
    // tiles k0 .. k1 of unit u again, on fp32 products of the pool's values
    template <typename C>
    __device__ __forceinline__ void again(const AttnArgsOf<C>& a, int u, int k0, int k1, int lane) {
        const int row = lane >> 2, t = lane & 3;
        int h;
        const int seq = a.c.by_heads.quot(u, &h), len = rows_held(a.c, seq);
        const float* q = static_cast<const float*>(a.q) + seq * a.qst[0] + (long long)h * a.g * a.qst[1];
        clear();
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
            const int n = min(TR, len - k * TR);
            int slot;
            const int page = page_of(a.c, seq, k * TR, &slot);
            if (page < 0) continue;
            const unsigned char* K = a.c.K + page * a.c.ks[0] + h * a.c.ks[1] + slot * a.c.ks[2];
            const unsigned char* V = a.c.V + page * a.c.vs[0] + h * a.c.vs[1] + slot * a.c.vs[2];
            float s[4] = {0.f, 0.f, 0.f, 0.f}, p[NB][2];
#pragma unroll 1
            for (int c = 0; c < D / 4; ++c) {
                float4 x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x[e] = 2 * t + e < n ? *reinterpret_cast<const float4*>(K + (2 * t + e) * a.c.ks[2] + 16 * c)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (row + 8 * b >= a.g) continue;
                    const float4 y = *reinterpret_cast<const float4*>(q + (row + 8 * b) * a.qst[1] + 4 * c);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        s[2 * b + e] =
                            fmaf(y.w, x[e].w, fmaf(y.z, x[e].z, fmaf(y.y, x[e].y, fmaf(y.x, x[e].x, s[2 * b + e]))));
                }
            }
            weigh(s, n, a.qscale, a.g, a.scores ? a.scores + (size_t)u * a.g * a.c.rows + (size_t)k * TR : nullptr,
                  a.c.rows, lane, p);
#pragma unroll 1
            for (int r = 0; r < n; ++r) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float w = r & 1 ? p[b][1] : p[b][0];
                    const float w0 = __shfl_sync(FULL, w, 8 * t + (r >> 1)), w1 = __shfl_sync(FULL, w, 8 * t + 4 + (r >> 1));
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const float4 v = *reinterpret_cast<const float4*>(V + r * a.c.vs[2] + 128 * f + 16 * row);
                        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float(&to)[4] = o[b][2 * f + (e >> 1)];
                            to[2 * (e & 1)] = fmaf(w0, x[e], to[2 * (e & 1)]);
                            to[2 * (e & 1) + 1] = fmaf(w1, x[e], to[2 * (e & 1) + 1]);
                        }
                    }
                }
            }
        }
    }
    template <typename Put, typename Stat>
    __device__ __forceinline__ void leave(int g, int lane, bool normalise, Put put, Stat stat) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float l = lrun[b];
            l += __shfl_xor_sync(FULL, l, 1);
            l += __shfl_xor_sync(FULL, l, 2);
            const int j = (lane >> 2) + 8 * b;
            if ((lane & 3) == 0 && j < g) stat(j, mrun[b], l);
            const float w = !normalise ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            const float w0 = __shfl_sync(FULL, w, (lane & 3) * 8), w1 = __shfl_sync(FULL, w, (lane & 3) * 8 + 4);
            const int j0 = (lane & 3) * 2 + 8 * b;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const int c = 32 * (mt >> 1) + 4 * (lane >> 2) + 2 * (mt & 1);
                if (j0 < g) {
                    put(j0, c, o[b][mt][0] * w0);
                    put(j0, c + 1, o[b][mt][2] * w0);
                }
                if (j0 + 1 < g) {
                    put(j0 + 1, c, o[b][mt][1] * w1);
                    put(j0 + 1, c + 1, o[b][mt][3] * w1);
                }
            }
        }
    }
};

// ---------------------------------------------------------------- attention
struct Seg {
    int u, nt, a;  // unit (-1: none), its tiles, its first tile
};

// A partial result of a unit to merge with others, or what the merging gives.
struct Job {
    int src, n;  // its sources in the list of sources
    int u;       // final: the unit whose outputs it gives; else -1
    float* dst;  // not final: where the merged partial goes
};
// Head j of the partials src[0 .. n), merged in that order by a warp.
template <typename C>
__device__ __forceinline__ void merge_head(const AttnArgsOf<C>& a, const Job& job, const float* const* src, int j, int lane) {
    const int sm = a.g * D + j, sl = sm + a.g;  // where a partial keeps its maximum and sum
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < job.n; i += 32) M = fmaxf(M, src[i][sm]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    const float ms = M == -INFINITY ? 0.f : M;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < job.n; ++i) {
        const float* p = src[i];
        const float f = ex2(p[sm] - ms);
        const float4 v = *reinterpret_cast<const float4*>(p + j * D + 4 * lane);
        L += f * p[sl];
        o.x += f * v.x;
        o.y += f * v.y;
        o.z += f * v.z;
        o.w += f * v.w;
    }
    __syncwarp();  // the destination may be one of the sources
    float* dst = job.dst;
    if (job.u >= 0) {
        const size_t at = (size_t)job.u * a.g;
        dst = a.out + at * D;
        const float r = L == 0.f ? 0.f : 1.f / L;
        o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
        if (lane == 0) {
            const float z = L == 0.f ? -INFINITY : M + log2f(L);
            a.lse2[at + j] = z;
            if (a.lse) a.lse[at + j] = z * LN2;
        }
    } else if (lane == 0) {
        dst[sm] = M;
        dst[sl] = L;
    }
    *reinterpret_cast<float4*>(dst + j * D + 4 * lane) = o;
}

// mass_in of the four rows from r on, if one of them is below r1 (r is unsigned:
// it goes past the last row, which may be just below 2^31)
template <typename C>
__device__ __forceinline__ float4 old_weights(const AttnArgsOf<C>& a, int u, unsigned r, unsigned r1) {
    return a.mass_in && r < r1 ? *reinterpret_cast<const float4*>(a.mass_in + (size_t)u * a.c.rows + r)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
}
// mass_out = v + sum_j e^{s_j - lse_j} for those of the four rows that are below r1
template <typename C>
__device__ __forceinline__ void add_weights(const AttnArgsOf<C>& a, int u, unsigned r, unsigned r1, float4 v) {
    const float* lse2 = a.lse2 + (size_t)u * a.g;
    const float* sc = a.scores + (size_t)u * a.g * a.c.rows + r;
    const size_t o = (size_t)u * a.c.rows + r;
    float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < a.g; j += 4) {
        float4 x[4];
        float lz[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lz[i] = -INFINITY;
            if (j + i < a.g) {
                x[i] = *reinterpret_cast<const float4*>(sc + (size_t)(j + i) * a.c.rows);
                lz[i] = lse2[j + i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lz[i] != -INFINITY) {
                add.x += ex2(x[i].x - lz[i]);
                add.y += ex2(x[i].y - lz[i]);
                add.z += ex2(x[i].z - lz[i]);
                add.w += ex2(x[i].w - lz[i]);
            }
    }
    v.x += add.x;
    v.y += add.y;
    v.z += add.z;
    v.w += add.w;
    if (r + 4 <= r1) {
        *reinterpret_cast<float4*>(a.mass_out + o) = v;
    } else {  // the rows behind the last one stay as they are
        a.mass_out[o] = v.x;
        if (r + 1 < r1) a.mass_out[o + 1] = v.y;
        if (r + 2 < r1) a.mass_out[o + 2] = v.z;
    }
}

template <typename E, typename C>
__global__ void __launch_bounds__(WARPS * 32, 1)
    paged_attn_kernel(const __grid_constant__ AttnArgsOf<C> a, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv) {
    constexpr int TR = E::TR, NW = WARPS, NT = NW * 32;
    // OWN: the kernel before is the one that attends the rows left out.  It let this
    // one start only when it had itself waited for all that wrote the inputs, and
    // the two write nothing of each other's, so this one runs beside it, on the SMs
    // that the other leaves, and waits for it at its end only, for the kernel behind
    // both.  A wait is what makes writes visible; that the starts come in order does
    // not promise that no older copy of skip, lens or q is still at hand here, and the
    // fence drops one (a full fence took 0.6 us, this none).  CTAs that have no SM left
    // to them leave at once, so that the kernel behind can be brought in (there is
    // always one that waits).
    constexpr bool OWN = std::is_same<C, OwnRows>::value;
    using T = typename E::T;
    extern __shared__ unsigned char smem_raw[];
    // swizzled tiles need 1024-byte alignment
    unsigned char* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ int2 start[NW];
    __shared__ __align__(8) uint64_t full[NW][NST];
    __shared__ int4 meta[NW][NST];  // unit, held rows, tile in the unit, tiles of the unit
    __shared__ Seg segs[2 * NW];    // partials of warp w: [2 w] left on the way (heads), [2 w + 1] at the end (its ring)
    __shared__ __align__(16) float2 scratch[NW][E::SCRATCH ? E::SCRATCH : 1];
    // merging: jobs and their sources; the units shared with other CTAs (unit,
    // first CTA, CTAs; unit -1: none, or not this CTA's to merge)
    constexpr int MAX_SRC = 2 * NW + MAX_GRID;
    __shared__ const float* src[MAX_SRC];
    __shared__ Job jobs[2 * NW];
    __shared__ int n_jobs;
    __shared__ int4 shared_units[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) ptx::mbar_init(&full[warp][i], 1);
        ptx::fence_barrier_init();
        segs[2 * warp].u = segs[2 * warp + 1].u = -1;
    }
    if (threadIdx.x < 2) {
        ptx::prefetch_tmap(threadIdx.x ? &tv : &tk);
        shared_units[threadIdx.x].x = -1;
    }
    if (OWN) ptx::fence_acquire();
    else ptx::grid_dependency_wait();  // lens, table, K, V, q may come from the previous kernel
    ptx::allow_dependent_launch();
    if constexpr (std::is_same<C, GroupRows>::value) look_up_rows<NT>(a.c);
    const int grid = working_ctas(a.c);
    if (OWN && (int)blockIdx.x >= grid) return;
    int cta = blockIdx.x;
    const Deal deal = deal_out<TR, NT>(a.c, start, cta, grid);
    const bool works = cta < deal.n_cta && deal.total > 0;
    const int t_begin = works ? deal.begin_warp(cta * NW + warp) : 0;
    const int t_end = works ? deal.begin_warp(cta * NW + warp + 1) : 0;
    unsigned char* ring = smem + (size_t)warp * NST * STAGE;
    const size_t pf = part_floats(a.g);
    float* heads = reinterpret_cast<float*>(smem + NW * NST * STAGE);

    if (t_begin < t_end) {
        E e;
        int u, nt, first;  // the unit, its tiles, its first tile
        auto enter = [&](int s, int h, int tiles, int at) {
            u = s * a.c.heads + h;
            nt = tiles;
            first = at;
            e.reset(static_cast<const T*>(a.q) + s * a.qst[0] + (long long)h * a.g * a.qst[1], a.qst[1], a.g, a.qscale,
                    lane);
        };
        Pos base = walk<TR>(a.c, start[warp].x, start[warp].y);
        // q is asked for before the tiles: behind them it would wait for all
        // the copies in flight (some 4 us at full bandwidth)
        enter(base.s, base.h, base.nt, t_begin - base.k);
        // ---- the producer's view: lane l knows the place of tile block + l
        int block = t_begin - 32;
        int p_page = 0, p_slot = 0, p_rows = 0;
        Pos p{};
        bool gave_up = false, dead = false;  // a copy never landed: the rest of the share is walked without its rows
        auto issue = [&](int st, int t) {
            if (t >= block + 32) {
                block += 32;
                if (block + lane < t_end) {
                    p = advance<TR>(a.c, base, lane);
                    const int row = first_row(a.c, p.s) + p.k * TR;
                    p_rows = min(TR, rows_held(a.c, p.s) - row);
                    p_page = page_of(a.c, p.s, row, &p_slot);
                    if (p_page < 0) p_rows = 0;
                }
                if (block + 32 < t_end) {
                    const Pos end{__shfl_sync(FULL, p.s, 31), __shfl_sync(FULL, p.h, 31), __shfl_sync(FULL, p.k, 31),
                                  __shfl_sync(FULL, p.nt, 31)};
                    base = advance<TR>(a.c, end, 1);
                }
            }
            if (lane == t - block) {
                meta[warp][st] = make_int4(p.s * a.c.heads + p.h, p_rows, p.k, p.nt);
                if (dead || (a.stall && (warp & 1) && t == t_begin)) return;
                if (p_rows > 0) {
                    ptx::mbar_arrive_expect_tx(&full[warp][st], STAGE);
                    E::load(ring + st * STAGE, &tk, &tv, p_page, p.h, p_slot, &full[warp][st]);
                } else {
                    ptx::mbar_arrive(&full[warp][st]);  // a bad page id: nothing to load
                }
            }
        };
        auto leave = [&](bool tail) {
            if constexpr (E::CHECKED)
                if (!dead && __any_sync(FULL, e.least < E::TINY))
                    e.again(a, u, max(0, t_begin - first), min(nt, t_end - first), lane);
            // final where the whole unit was this warp's, else left to be merged
            const bool whole = first >= t_begin && first + nt <= t_end;
            const size_t o = (size_t)u * a.g;
            float* dst = whole ? a.out + o * D : (tail ? reinterpret_cast<float*>(ring) : heads + warp * pf);
            e.leave(a.g, lane, whole, [&](int j, int c, float v) { dst[j * D + c] = v; },
                    [&](int j, float m, float l) {
                        if (whole) {
                            const float z = l == 0.f ? -INFINITY : m + log2f(l);
                            a.lse2[o + j] = z;
                            if (a.lse) a.lse[o + j] = z * LN2;
                        } else {
                            dst[a.g * D + j] = m;
                            dst[a.g * D + a.g + j] = l;
                        }
                    });
            if (lane == 0 && !whole) segs[2 * warp + tail] = Seg{u, nt, first};
            if constexpr (OWN)
                if (lane == 0 && whole) a.c.left[u] = 0;
        };
        int st = 0, parity = 0;
        // the first NST turns only ask for tiles
        for (int t = t_begin - NST; t < t_end; ++t) {
            if (t >= t_begin) {
                if (!dead && !ptx::mbar_wait(&full[warp][st], parity, a.wait_limit, nullptr)) dead = true;
                if (__any_sync(FULL, dead) && !gave_up) {
                    dead = gave_up = true;
                    if (lane == 0) report(a.c.dev_err, CKV_DEV_TIMEOUT);
                    // the copies in flight get their time, the late one too:
                    // the rings are used for partials after this
                    for (int i = 0, s2 = st, p2 = parity; i < NST && t + i < t_end; ++i) {
                        ptx::mbar_wait(&full[warp][s2], p2, a.wait_limit, nullptr);
                        if (++s2 == NST) {
                            s2 = 0;
                            p2 ^= 1;
                        }
                    }
                }
                const int4 m = meta[warp][st];
                if (m.x != u) {
                    leave(false);
                    int h;
                    const int s = a.c.by_heads.quot(m.x, &h);
                    enter(s, h, m.w, t - m.z);
                }
                float* sc = a.scores ? a.scores + (size_t)u * a.g * a.c.rows + (size_t)m.z * TR : nullptr;
                if (m.y > 0 && !dead)
                    e.tile(ring + st * STAGE, scratch[warp], m.y, a.qscale, a.g, sc, a.c.rows, lane);
                else if (sc)
                    for (int i = lane; i < TR * a.g; i += 32) sc[(size_t)(i / TR) * a.c.rows + i % TR] = -INFINITY;
                __syncwarp();
            }
            if (t + NST < t_end) issue(st, t + NST);
            __syncwarp();
            if (++st == NST) {
                st = 0;
                parity ^= t >= t_begin;
            }
        }
        leave(true);
    }
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < a.c.seqs; s += NT) check_len(a.c, s);
    // units without rows: nothing else writes their outputs (OWN: the kernel behind does)
    for (int s = blockIdx.x; s < a.c.seqs && !OWN; s += grid)
        if (rows_attended(a.c, s) == 0)
            for (long long i = threadIdx.x; i < (long long)a.c.heads * a.g * D; i += NT) {
                const size_t o = (size_t)s * a.c.heads * a.g;
                a.out[o * D + i] = 0.f;
                if (a.lse && i < (long long)a.c.heads * a.g) a.lse[o + i] = -INFINITY;
            }
    if (!works) {
        if (OWN) ptx::grid_dependency_wait();
        return;
    }
    // a CTA that adds its unit's weights itself asks for the old ones in time
    const int unit_rows = a.fuse ? rows_held(a.c, a.c.by_heads.quot(blockIdx.x)) : 0;
    const float4 old = old_weights(a, blockIdx.x, 4 * threadIdx.x, unit_rows);
    __syncthreads();

    // ---- merging.  This code runs once a call, and its instructions come from
    // L2 at some 60 ns per 128 bytes, so that its length counts for more than
    // its work: round 0 merges the partials of this CTA's warps, in warp order;
    // later rounds, only in the CTA that is the last to leave its part of a
    // shared unit, merge the CTAs' parts, in CTA order, copied to the rings.
    const int cta_begin = deal.begin_cta(cta), cta_end = deal.begin_cta(cta + 1);
    const int cap = (int)((size_t)NW * NST * STAGE / (pf * sizeof(float))) - 1;  // parts a round
    for (int round = 0, x = 0, next = 0;; ++round) {
        if (round == 0) {
            if (warp == 0) {
                // lane l looks after partial l; those of a unit follow one another
                Seg sg{-1, 0, 0};
                bool leads = false;
                if (lane < 2 * NW) {
                    const int tb = deal.begin_warp(cta * NW + (lane >> 1));
                    sg = segs[lane];
                    leads = sg.u >= 0 && (sg.a >= tb || tb == cta_begin);
                }
                const unsigned held = __ballot_sync(FULL, sg.u >= 0), lead = __ballot_sync(FULL, leads);
                const unsigned below = (1u << lane) - 1u;
                const float* mine_at = lane & 1 ? reinterpret_cast<const float*>(smem + (size_t)(lane >> 1) * NST * STAGE)
                                                : heads + (lane >> 1) * pf;
                if (sg.u >= 0) src[__popc(held & below)] = mine_at;
                if (leads) {
                    const unsigned after = lead & ~below & ~(1u << lane);  // the next leader ends this job
                    const unsigned mine = held & ~below & (after ? (after & -after) - 1u : FULL);
                    const bool began = sg.a >= cta_begin, whole = began && sg.a + sg.nt <= cta_end;
                    jobs[__popc(lead & below)] = Job{__popc(held & below), __popc(mine), whole ? sg.u : -1,
                                                     a.part + ((size_t)blockIdx.x * 2 + began) * pf};
                    int c0 = 0, n = 0;
                    if (!whole) {
                        c0 = deal.cta_of(sg.a);
                        n = deal.cta_of(sg.a + sg.nt - 1) - c0 + 1;
                    }
                    if constexpr (OWN) {
                        // a few parts are merged by the kernel behind, together with the others' rows
                        const bool joined = n <= JOINED_PARTS;
                        if (began) a.c.left[sg.u] = joined ? n << 16 | c0 : 0;
                        if (joined) n = 0;
                    }
                    if (n) shared_units[began] = make_int4(sg.u, c0, n, 0);
                }
                if (lane == 0) n_jobs = __popc(lead);
            }
        } else {
            // the next unit, and of it the next parts: behind what the rounds
            // before have made of it (in slot 0 of the rings)
            while (x < 2 && (shared_units[x].x < 0 || next == shared_units[x].z)) {
                ++x;
                next = 0;
            }
            if (x == 2) break;
            const int4 su = shared_units[x];
            const int n = min(su.z - next, cap), had = next > 0;
            float* slots = reinterpret_cast<float*>(smem);
            for (int i = threadIdx.x; i < n + had; i += NT) src[i] = slots + (size_t)(i + !had) * pf;
            if (threadIdx.x == 0) {
                n_jobs = 1;
                jobs[0] = Job{0, n + had, next + n == su.z ? su.x : -1, slots};
            }
            const int pieces = (int)(pf / 4);  // of 16 bytes in a part
            for (int i = threadIdx.x; i < n * pieces; i += NT) {
                const int k = i / pieces, q = su.y + next + k;
                ptx::cp_async16(slots + (size_t)pf + (size_t)i * 4,
                                a.part + ((size_t)q * 2 + (q == su.y)) * pf + (size_t)(i - k * pieces) * 4);
            }
            ptx::cp_async_wait_all();
            next += n;
        }
        __syncthreads();
        for (int item = warp; item < n_jobs * a.g; item += NW) {
            const Job job = jobs[item / a.g];
            merge_head(a, job, src + job.src, item % a.g, lane);
        }
        __syncthreads();
        if (round == 0) {
            if (threadIdx.x < 2 && shared_units[threadIdx.x].x >= 0) {
                const int4 su = shared_units[threadIdx.x];
                unsigned before;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                             : "=r"(before)
                             : "l"(a.arrived + su.y)
                             : "memory");
                if (before == (unsigned)(su.z - 1)) a.arrived[su.y] = 0;  // the last one: for the next call
                else shared_units[threadIdx.x].x = -1;
            }
            __syncthreads();
        }
    }
    if (4 * (int)threadIdx.x < unit_rows) add_weights(a, blockIdx.x, 4 * threadIdx.x, unit_rows, old);
    if (OWN) ptx::grid_dependency_wait();
}

// ---------------------------------------------------------------- accumulated weights
// The second pass over the scores: the tiles of the attention
// kernel's warps, W_SPLIT CTAs to one of its, a lane four rows at a time.  Only
// the scores and the lse come from the attention kernel: the deal is derived
// again and the first rows' weights are loaded while its last CTAs still run.
// 1 / 2 / 3 / 4 / 6: 41.0 / 39.7 / 39.8 / 40.5 / 42.3 us for 256 units of 1.2k
// rows, 129.7 / 121.5 / 119.2 / 117.9 / 121.6 for 64 of up to 34k.
constexpr int W_SPLIT = 3;

template <int TR>
__global__ void __launch_bounds__(WARPS * 32) paged_weights_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int NW = WARPS;
    __shared__ int2 start[NW];
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int cta = blockIdx.x / W_SPLIT;
    const int part = blockIdx.x % W_SPLIT;
    // lens, table and mass_in are not written by the attention kernel, and it
    // began after what wrote them had ended
    const Deal deal = deal_out<TR, NW * 32>(a.c, start, cta, gridDim.x / W_SPLIT);
    int t = 0, t1 = 0;
    if (cta < deal.n_cta) {
        const int b0 = deal.begin_warp(cta * NW + warp), n = deal.begin_warp(cta * NW + warp + 1) - b0;
        t = b0 + n * part / W_SPLIT;
        t1 = b0 + n * (part + 1) / W_SPLIT;
    }
    Pos p{};
    int len = 0;
    float4 next = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < t1) {
        p = advance<TR>(a.c, walk<TR>(a.c, start[warp].x, start[warp].y), t - deal.begin_warp(cta * NW + warp));
        len = rows_held(a.c, p.s);
        next = old_weights(a, p.s * a.c.heads + p.h, (unsigned)p.k * TR + 4 * lane,
                           min(len, (p.k + min(p.nt - p.k, t1 - t)) * TR));
    }
    ptx::grid_dependency_wait();
    while (t < t1) {
        const int u = p.s * a.c.heads + p.h;
        const int n = min(p.nt - p.k, t1 - t);  // tiles of this unit
        const unsigned r1 = min(len, (p.k + n) * TR);
        for (unsigned r = (unsigned)p.k * TR + 4 * lane; r < r1; r += 128) {
            const float4 old = next;
            next = old_weights(a, u, r + 128, r1);
            add_weights(a, u, r, r1, old);
        }
        t += n;
        p = advance<TR>(a.c, p, n);
        if (t < t1) {
            len = rows_held(a.c, p.s);
            next = old_weights(a, p.s * a.c.heads + p.h, (unsigned)p.k * TR + 4 * lane,
                               min(len, (p.k + min(p.nt - p.k, t1 - t)) * TR));
        }
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
    static std::atomic<void*> fn{nullptr};
    void* p = fn.load(std::memory_order_relaxed);
    if (!p) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_relaxed);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

}  // namespace

// The pool as a tensor map whose boxes are tiles of one page and KV head: rows
// cut into pieces of 128 bytes and swizzled, [page][head][piece][slot][128
// bytes], or fp32 rows whole, [page][head][slot][128 channels].  A box has all
// pieces of its rows, or one where pieces_a_box says so.
bool encode_pool(CUtensorMap* m, const Cache& c, const void* base, const long long* st, bool bf16, bool swizzled,
                 int tile_rows, int pieces_a_box) {
    const auto enc = get_encode();
    if (!enc) return false;
    const cuuint64_t slot = (cuuint64_t)st[2], head = (cuuint64_t)st[1], page = (cuuint64_t)st[0];
    const cuuint32_t wide = bf16 ? 64 : 32, pieces = D / wide;
    const cuuint64_t dims5[5] = {wide, (cuuint64_t)c.page, pieces, (cuuint64_t)c.heads, (cuuint64_t)c.n_pages};
    const cuuint64_t str5[4] = {slot, 128, head, page};
    const cuuint32_t box5[5] = {wide, (cuuint32_t)tile_rows, pieces_a_box ? (cuuint32_t)pieces_a_box : pieces, 1, 1};
    const cuuint64_t dims4[4] = {D, (cuuint64_t)c.page, (cuuint64_t)c.heads, (cuuint64_t)c.n_pages};
    const cuuint64_t str4[3] = {slot, head, page};
    const cuuint32_t box4[4] = {D, (cuuint32_t)tile_rows, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const CUresult r =
        swizzled ? enc(m, type, 5, const_cast<void*>(base), dims5, str5, box5, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
                 : enc(m, type, 4, const_cast<void*>(base), dims4, str4, box4, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

namespace {

struct Layout {
    size_t part, lse2, scores, total;  // byte offsets; the arrivals come first
};
Layout layout_of(const Cache& c, int g, bool with_mass) {
    Layout l;
    const size_t units = (size_t)c.seqs * c.heads, pf = part_floats(g) * sizeof(float);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.part = MAX_GRID * sizeof(unsigned);
    l.lse2 = l.part + up(MAX_GRID * 2 * pf);
    l.scores = l.lse2 + up(units * g * sizeof(float));
    l.total = l.scores + (with_mass ? up(units * g * (size_t)c.rows * sizeof(float)) : 0);
    return l;
}

template <typename E, typename C>
cudaError_t launch(const AttnArgsOf<C>& a, int sms, int dev, cudaStream_t s) {
    constexpr bool bf16 = sizeof(typename E::T) == 2;
    CUtensorMap tk, tv;
    if (!encode_pool(&tk, a.c, a.c.K, a.c.ks, bf16, E::SWIZZLED, E::TR) ||
        !encode_pool(&tv, a.c, a.c.V, a.c.vs, bf16, E::SWIZZLED, E::TR))
        return cudaErrorInvalidValue;
    const long long most = (long long)a.c.seqs * a.c.heads * ceil_div(a.c.rows, E::TR);  // tiles
    const long long useful = (most + WARPS - 1) / WARPS, units = (long long)a.c.seqs * a.c.heads;
    int grid = sms < MAX_GRID ? sms : MAX_GRID;
    if (grid > useful) grid = (int)(useful > units || units > grid ? useful : units);
    // the rings, the partials that warps leave on the way, and room to align
    const size_t rings = (size_t)WARPS * NST * STAGE + 1024;
    const size_t smem = rings + WARPS * part_floats(a.g) * sizeof(float);
    static std::atomic<bool> set[MAX_DEVICES];
    if (!set[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<E, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   rings + WARPS * part_floats(MAX_G) * sizeof(float));
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    // Where the capacity alone says that every unit gets a CTA of its own, that
    // CTA adds the weights and the second kernel is not launched.
    AttnArgsOf<C> b = a;
    b.fuse = a.mass_out && units <= grid && ceil_div(ceil_div(a.c.rows, E::TR), WARPS) <= 1 + OWN_EXTRA;
    static_assert((1 + OWN_EXTRA) * WARPS * E::TR <= 4 * WARPS * 32, "a thread adds the weights of four rows at most");
    cudaError_t e = launch_dependent(paged_attn_kernel<E, C>, dim3(grid), dim3(WARPS * 32), smem, s, b, tk, tv);
    if constexpr (std::is_same<C, Cache>::value)
        if (e == cudaSuccess && a.mass_out && !b.fuse)
            e = launch_dependent(paged_weights_kernel<E::TR>, dim3(grid * W_SPLIT), dim3(WARPS * 32), 0, s, a);
    return e;
}

template <typename C>
cudaError_t launch_f32(const AttnArgsOf<C>& a, int sms, int dev, cudaStream_t s) {
    if (a.g == 1) return launch<TilesF32<1>>(a, sms, dev, s);
    if (a.g == 2) return launch<TilesF32<2>>(a, sms, dev, s);
    if (a.g <= 4) return launch<TilesF32<4>>(a, sms, dev, s);
    if (a.g <= 8) return launch<TilesF32<8>>(a, sms, dev, s);
    return launch<TilesF32Tc<2>>(a, sms, dev, s);
}
// what the calls without weights have in common
template <typename C>
void take(AttnArgsOf<C>* a, const void* q, const long long* q_stride, int g, float qscale, float* out, float* lse, void* workspace) {
    const Layout l = layout_of(a->c, g, false);
    unsigned char* w = static_cast<unsigned char*>(workspace);
    a->q = q;
    a->qst[0] = q_stride[0];
    a->qst[1] = q_stride[1];
    a->g = g;
    a->qscale = qscale;
    a->out = out;
    a->lse = lse;
    a->arrived = reinterpret_cast<unsigned*>(w);
    a->part = reinterpret_cast<float*>(w + l.part);
    a->lse2 = reinterpret_cast<float*>(w + l.lse2);
}

std::atomic<long long> wait_limit{WAIT_LIMIT};
std::atomic<int> stall_switch{0};

}  // namespace

void waits(long long* limit, int* stall) {
    *limit = wait_limit.load(std::memory_order_relaxed);
    *stall = stall_switch.load(std::memory_order_relaxed);
}

size_t attn_workspace(const Cache& c, int g, float** lse2, float** part, void* workspace) {
    const Layout l = layout_of(c, g, false);
    if (lse2) *lse2 = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + l.lse2);
    if (part) *part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + l.part);
    return l.total;
}

cudaError_t launch_attn_own_rows(const Cache& c, const int32_t* skip, const int32_t* ctas, int32_t* left, const void* q,
                                 const long long* q_stride, int g, float qscale, float* out, float* lse, void* workspace,
                                 cudaStream_t s) {
    AttnArgsOf<OwnRows> a = {};
    static_cast<Cache&>(a.c) = c;
    a.c.skip = skip;
    a.c.ctas = ctas;
    a.c.left = left;
    take(&a, q, q_stride, g, qscale, out, lse, workspace);
    waits(&a.wait_limit, &a.stall);
    a.stall = 0;  // the kernel before this one is the one to stall
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    return g <= 8 ? launch<TilesBf16<1>>(a, sms, dev, s) : launch<TilesBf16<2>>(a, sms, dev, s);
}

cudaError_t launch_attn_in_groups(const Cache& c, const Groups& groups, const void* q, const long long* q_stride, int g,
                                  float qscale, float* out, float* lse, void* workspace, cudaStream_t s) {
    AttnArgsOf<GroupRows> a = {};
    static_cast<Cache&>(a.c) = c;
    a.c.groups = groups;
    take(&a, q, q_stride, g, qscale, out, lse, workspace);
    waits(&a.wait_limit, &a.stall);
    int dev = 0;
    const int sms = sm_count(&dev);
    return sms < 1 ? cudaErrorInvalidDevice : launch_f32(a, sms, dev, s);
}

}  // namespace paged
}  // namespace ckv

using namespace ckv;
using namespace ckv::paged;

extern "C" ckv_status ckv_paged_set_wait_limit(int64_t cycles, int32_t stall) {
    CKV_TRACE("ckv_paged_set_wait_limit");
    if (cycles < 1 || cycles > MAX_WAIT_LIMIT || (stall != 0 && stall != 1)) return CKV_ERR_ARG;
    wait_limit.store(cycles, std::memory_order_relaxed);
    stall_switch.store(stall, std::memory_order_relaxed);
    return CKV_OK;
}

extern "C" ckv_status ckv_paged_attn_workspace(const ckv_paged_cache* cache, int32_t g, int32_t with_mass,
                                               int64_t* bytes) {
    Cache c;
    const ckv_status st = check_cache(cache, &c);
    if (st != CKV_OK) return st;
    if (!bytes || g < 1 || g > MAX_G) return CKV_ERR_ARG;
    *bytes = (int64_t)layout_of(c, g, with_mass != 0).total;
    return CKV_OK;
}

extern "C" ckv_status ckv_paged_decode_attn(const ckv_paged_cache* cache, const void* q, int32_t q_dtype,
                                            const int64_t* q_stride, int32_t g, float scale, float* out, float* lse,
                                            const float* mass_in, float* mass_out, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
    CKV_TRACE("ckv_paged_decode_attn");
    AttnArgs a;
    const ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (!q || !q_stride || !out || !workspace) return CKV_ERR_ARG;
    if (q_dtype != cache->kv_dtype) return CKV_ERR_DTYPE;
    if (g < 1 || g > MAX_G || !isfinite(scale * LOG2E) || (mass_in && !mass_out)) return CKV_ERR_ARG;
    const bool bf16 = q_dtype == CKV_BF16;
    const long long extent[2] = {a.c.seqs, (long long)a.c.heads * g};
    for (int i = 0; i < 2; ++i) {
        if (q_stride[i] < 0 || q_stride[i] > MAX_STRIDE) return CKV_ERR_ARG;
        a.qst[i] = extent[i] > 1 ? q_stride[i] : 0;  // a single extent is never multiplied by more than 0
        if (a.qst[i] * (bf16 ? 2 : 4) & 15) return CKV_ERR_ALIGN;
    }
    // tile numbers are 32-bit: 2^31 tiles of fp32 rows are 17 TB of K and V
    if ((long long)a.c.seqs * a.c.heads * ceil_div(a.c.rows, 8) > 0x7fff0000LL) return CKV_ERR_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(mass_in) || !aligned16(mass_out) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return CKV_ERR_ALIGN;
    if (!same_or_apart(mass_in, mass_out, (long long)a.c.seqs * a.c.heads * a.c.rows)) return CKV_ERR_ARG;
    const Layout l = layout_of(a.c, g, mass_out != nullptr);
    if (workspace_bytes < (int64_t)l.total) return CKV_ERR_CAPACITY;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    a.q = q;
    a.g = g;
    a.qscale = scale * LOG2E;
    a.out = out;
    a.lse = lse;
    a.mass_in = mass_in;
    a.mass_out = mass_out;
    a.arrived = reinterpret_cast<unsigned*>(w);
    a.part = reinterpret_cast<float*>(w + l.part);
    a.lse2 = reinterpret_cast<float*>(w + l.lse2);
    a.scores = mass_out ? reinterpret_cast<float*>(w + l.scores) : nullptr;
    a.fuse = 0;
    waits(&a.wait_limit, &a.stall);
    int dev = 0;
    const int grid = sm_count(&dev);
    if (grid < 1) return CKV_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (bf16) e = g <= 8 ? launch<TilesBf16<1>>(a, grid, dev, s) : launch<TilesBf16<2>>(a, grid, dev, s);
    else e = launch_f32(a, grid, dev, s);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
