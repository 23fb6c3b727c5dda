// Decode attention of a batch whose sequences share leading rows: those rows are
// read once for all queries of a group.
//
// For a group of m sequences with g query heads to a KV head, m g queries meet
// every shared row, 4 m g 128 operations on 512 bytes (bf16): from a few dozen
// queries on that is work for tensor-core tiles, and up to about 128 of them HBM
// still bounds it.  Four kernels, each launched while the one before ends:
//
//   paged_shared_prep    which rows are left to the groups (skip[s], group of s),
//                        and the groups' tiles, as running sums
//   paged_shared_kernel  the shared rows (below)
//   paged_attn_kernel    every sequence's own rows, from skip[s] on
//   paged_shared_join    o = sum_p e^{lse_p - lse} o_p over both
//
// paged_shared_kernel.  A tile is 128 queries by 128 shared rows of a KV head;
// the tiles of all (group, KV head, block of 128 queries), the units, are dealt
// out evenly to one persistent CTA an SM, which keeps its unit's queries in
// shared memory and streams K and V tiles through a ring of six 32 KB stages.
//   S = Q K^T           tcgen05 128 x 128 x 128, into tensor memory
//   P = 2^{S scale - m}  one thread a query, m its running maximum so far
//   T = P V             P from tensor memory, as three bf16 terms
//   O = O a + T b       in registers, one thread half of a query's channels
// A weight is the sum of three bf16 terms (its upper, middle and lower eight
// bits), so that the products are those of fp32 weights; with one term outputs
// would be off by 2^-9 where the decode attention of this library is off by
// 2^-21.  That makes four products a tile, some 1.1 us at the measured dense
// rate, against 1.5 us that an SM's share of HBM takes for the tile's 64 KB.  T starts from
// zero at each tile and joins O by an ordinary addition, as the tensor core
// truncates what it accumulates and O grows over hundreds of tiles.  It also
// leaves O's scaling off the path from one tile's maximum to the next one's
// product: two groups of four warps take the softmax of every other tile, each
// with a running maximum of its own, and O follows with the larger of both.
// Warp roles:
//   warp 0       asks for the tiles (TMA)
//   warp 1       owns tensor memory, issues the products
//   warps 2-9    softmax: four of even, four of odd tiles, a thread a query
//   warps 10-17  queries to shared memory; O, a thread 64 channels of a query
// Where a unit is several CTAs' its parts are joined by the last kernel in the
// order of its rows, so that results do not depend on timing.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "mma_sync.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace ckv {
namespace paged {
namespace {

using mmas::ex2;

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr int KT = 128;              // rows of a tile
constexpr int QT = 128;              // queries of a tile
constexpr int PANEL = 128 * 128;     // 64 channels of 128 rows
constexpr int STAGE = 2 * PANEL;     // K or V of a tile
constexpr int NST = 6;
constexpr int SOFT_WARPS = 8, OUT_WARPS = 8;
constexpr int THREADS = 32 * (2 + SOFT_WARPS + OUT_WARPS);
constexpr int PREP_THREADS = 1024;
constexpr int JOIN_WARPS = 8;
// columns of tensor memory: scores and weights of even and odd tiles, then T
constexpr uint32_t SP_COLS = 192, T_COL = 2 * SP_COLS;

// A group as the prep leaves it.
struct Group {
    int first, members;  // sequences
    int rows;            // shared, a multiple of TILE; 0: nothing is shared
    int blocks;          // of QT queries
};

struct SharedArgs {
    Cache c;
    const unsigned char* q;
    long long qst[2];  // byte strides: sequence, query head
    int g;
    float qscale;  // scale * log2(e)
    const int32_t* group_starts;
    const int32_t* prefix;
    int groups;
    int box_rows;  // rows of a copy: divides the page and KT
    float* out;
    float* lse;
    // workspace
    Group* group;       // [groups]
    int* tile_base;     // [groups + 1] tiles before the group
    int32_t* skip;      // [seqs] rows that the group attends
    int* group_of;      // [seqs]
    float* own_lse2;    // [seqs * heads * g] of the sequences' own rows, base 2
    // parts: O, and (maximum, sum) of even and odd tiles.  The CTA in which a
    // unit begins leaves its part by query, the others (each continues one unit at most) by CTA
    float* row_o;       // [seqs * heads * g][D]
    float4* row_ml;
    float* cta_o;       // [MAX_GRID][QT][D]
    float4* cta_ml;     // [MAX_GRID][QT]
    int grid;
    long long wait_limit;
    int stall;
};

// ---------------------------------------------------------------- the groups
// One CTA.  A thread has a chunk of neighbouring groups, then of sequences.
__global__ void __launch_bounds__(PREP_THREADS) paged_shared_prep(const __grid_constant__ SharedArgs a) {
    __shared__ int warp_val[PREP_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int chunk = (a.groups + PREP_THREADS - 1) / PREP_THREADS;
    const int i0 = min(a.groups, tid * chunk), i1 = min(a.groups, i0 + chunk);
    auto start_at = [&](int i) { return min(max(a.group_starts[i], 0), a.c.seqs); };
    // starts ascend: each is at least the largest before it
    int top = 0;
    for (int i = i0; i < i1; ++i) {
        const int raw = a.group_starts[i];
        if (raw < 0 || raw > a.c.seqs || raw > a.group_starts[i + 1] || a.prefix[i] < 0)
            report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        top = max(top, start_at(i));
    }
    int x = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x = max(x, y);
    }
    if (lane == 31) warp_val[warp] = x;
    __syncthreads();
    int before = __shfl_up_sync(FULL, x, 1);
    if (lane == 0) before = 0;
    for (int w = 0; w < warp; ++w) before = max(before, warp_val[w]);
    __syncthreads();
    int tiles = 0;
    for (int i = i0; i < i1; ++i) {
        const int first = max(before, start_at(i)), end = max(first, start_at(i + 1));
        before = first;
        Group gr{first, end - first, 0, 0};
        if (gr.members > 1) {
            gr.rows = min(max(a.prefix[i], 0), rows_held(a.c, first)) / TILE * TILE;
            gr.blocks = (int)(((long long)gr.members * a.g + QT - 1) / QT);
        }
        a.group[i] = gr;
        tiles += a.c.heads * gr.blocks * ((gr.rows + KT - 1) / KT);
    }
    x = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_val[warp] = x;
    __syncthreads();
    int at = x - tiles;
    for (int w = 0; w < warp; ++w) at += warp_val[w];
    for (int i = i0; i < i1; ++i) {
        a.tile_base[i] = at;
        const Group gr = a.group[i];
        at += a.c.heads * gr.blocks * ((gr.rows + KT - 1) / KT);
    }
    if (tid == PREP_THREADS - 1) {
        a.tile_base[a.groups] = at;
        const int end = a.group_starts[a.groups];
        if (end < 0 || end > a.c.seqs) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
    }
    __syncthreads();
    for (int s = tid; s < a.c.seqs; s += PREP_THREADS) {
        // the last group that begins at s or before
        int lo = -1, hi = a.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.group[mid].first <= s) lo = mid;
            else hi = mid;
        }
        int rows = 0;
        if (lo >= 0 && s < a.group[lo].first + a.group[lo].members) rows = a.group[lo].rows;
        if (rows > a.c.lens[s]) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        a.skip[s] = rows;
        a.group_of[s] = lo;
    }
}

// the group that tile t belongs to (tiles are numbered from 0; t is one of
// them), found by a warp
__device__ __forceinline__ int group_of_tile(const SharedArgs& a, int t, int from, int lane) {
    for (int i = from; i < a.groups; i += 32) {
        const bool past = i + lane < a.groups && a.tile_base[i + lane + 1] <= t;
        const unsigned m = __ballot_sync(FULL, past);
        if (m != FULL) return i + __popc(m);
    }
    return a.groups - 1;
}

// A CTA's share of one unit.
struct Run {
    int group, first, members, rows;
    int h, block;  // KV head, block of queries
    int k0, n;     // tiles [k0, k0 + n) of the unit
    bool begins;   // with the unit's first tile
    int queries;   // in the block
};
// The run that begins at tile t of a share that ends at t_end, for a whole warp.
__device__ __forceinline__ Run run_at(const SharedArgs& a, int t, int t_end, int* from, int lane) {
    Run r;
    r.group = *from = group_of_tile(a, t, *from, lane);
    const Group gr = a.group[r.group];
    r.first = gr.first;
    r.members = gr.members;
    r.rows = gr.rows;
    const int nt = (gr.rows + KT - 1) / KT;
    const int left = t - a.tile_base[r.group], unit = left / nt;
    r.k0 = left - unit * nt;
    r.h = unit / gr.blocks;
    r.block = unit - r.h * gr.blocks;
    r.n = min(nt - r.k0, t_end - t);
    r.begins = r.k0 == 0;
    r.queries = min(QT, gr.members * a.g - r.block * QT);
    return r;
}

struct __align__(8) Bars {
    uint64_t full[NST], empty[NST];
    uint64_t q_full;
    uint64_t s_full[2], p_full[2], m_empty[2];
    uint64_t t_full, t_empty;
    uint64_t never, drain;
    int rows[NST];     // of a K stage's tile: those whose page is good
    int s_rows[2], t_rows;
    uint32_t tmem_base;
    int abort;
};
struct __align__(1024) Smem {
    unsigned char q[STAGE];
    unsigned char ring[NST][STAGE];
    float m[2][QT];  // the maxima that the weights of an even, odd tile go by
    Bars bars;
};
static_assert(sizeof(Smem) <= 232448 - 1024, "shared memory of a CTA");

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars* b, const SharedArgs& a) {
    if (ptx::mbar_wait(bar, parity, a.wait_limit, &b->abort)) return true;
    if (atomicExch(&b->abort, 1) == 0) report(a.c.dev_err, CKV_DEV_TIMEOUT);
    return false;
}

__global__ void __launch_bounds__(THREADS, 1)
    paged_shared_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
    extern __shared__ unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023));
    Bars* bs = &sm.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            ptx::mbar_init(&bs->full[i], 1);
            ptx::mbar_init(&bs->empty[i], 1);
        }
        ptx::mbar_init(&bs->q_full, OUT_WARPS);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bs->s_full[i], 2);  // the product, and the thread that says of how many rows
            ptx::mbar_init(&bs->p_full[i], SOFT_WARPS / 2);
            ptx::mbar_init(&bs->m_empty[i], OUT_WARPS);
        }
        ptx::mbar_init(&bs->t_full, 2);
        ptx::mbar_init(&bs->t_empty, OUT_WARPS);
        ptx::mbar_init(&bs->never, 1);
        ptx::mbar_init(&bs->drain, 1);
        bs->abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&bs->tmem_base, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bs->tmem_base;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const int total = a.tile_base[a.groups];
    const Deal deal(total, Deal::ctas(total, 1, a.grid), 1);
    const bool works = (int)blockIdx.x < deal.n_cta && total > 0;
    const int t_begin = works ? deal.begin_cta(blockIdx.x) : 0, t_end = works ? deal.begin_cta(blockIdx.x + 1) : 0;
    int loads = 0;  // stages that the producer has asked for
    bool alive = true;
    int from = 0;  // the group to look from
    int j = 0;     // tiles so far

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane < 2) ptx::prefetch_tmap(lane ? &tv : &tk);
        const FastDiv& by_page = a.c.by_page;
        for (int t = t_begin; t < t_end && alive;) {
            const Run r = run_at(a, t, t_end, &from, lane);
            const int32_t* table = a.c.table + (size_t)r.first * a.c.max_pages;
            for (int k = r.k0; k < r.k0 + r.n && alive; ++k, ++j) {
                // lane l looks after the tile's l-th copy
                const int row = k * KT + lane * a.box_rows;
                int page = -1, slot = 0;
                const bool there = lane * a.box_rows < KT && row < r.rows;
                if (there) {
                    page = table[by_page.quot(row, &slot)];
                    if (page < 0 || page >= a.c.n_pages) {
                        report(a.c.dev_err, CKV_DEV_BAD_INDEX);
                        page = -1;
                    }
                }
                // rows of bad pages are left out: the others move up
                const unsigned good = __ballot_sync(FULL, page >= 0);
                const int place = __popc(good & ((1u << lane) - 1u)), copies = __popc(good);
                const int short_by = __reduce_max_sync(FULL, page >= 0 ? max(0, row + a.box_rows - r.rows) : 0);
                for (int half = 0; half < 2 && alive; ++half, ++loads) {
                    const int st = loads % NST;
                    if (loads >= NST && !__all_sync(FULL, wait(&bs->empty[st], (loads / NST - 1) & 1, bs, a))) {
                        alive = false;
                        break;
                    }
                    if (lane == 0) {
                        bs->rows[st] = copies * a.box_rows - short_by;
                        if (copies) ptx::mbar_arrive_expect_tx(&bs->full[st], copies * a.box_rows * 256);
                        else ptx::mbar_arrive(&bs->full[st]);
                    }
                    __syncwarp();
                    if (page >= 0) {
                        unsigned char* to = sm.ring[st] + place * a.box_rows * 128;
                        const CUtensorMap* map = half ? &tv : &tk;
#pragma unroll
                        for (int piece = 0; piece < 2; ++piece)
                            asm volatile(
                                "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                                "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(ptx::smem_u32(to + piece * PANEL)),
                                "l"(map), "r"(0), "r"(slot), "r"(piece), "r"(r.h), "r"(page),
                                "r"(ptx::smem_u32(&bs->full[st]))
                                : "memory");
                    }
                    __syncwarp();
                }
            }
            t += r.n;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ the products
        const uint32_t ring = ptx::smem_u32(sm.ring), qa = ptx::smem_u32(sm.q);
        constexpr uint32_t ID_S = ptx::idesc_bf16_f32(QT, KT);
        constexpr uint32_t ID_T = ptx::idesc_bf16_f32(QT, D) | ptx::IDESC_B_MN_MAJOR;
        int runs = 0;
        // all lanes keep step for the runs; lane 0 waits and issues
        for (int t = t_begin; t < t_end && alive; ++runs) {
            const Run r = run_at(a, t, t_end, &from, lane);
            if (lane == 0) {
                if (runs == 0 && a.stall && !wait(&bs->never, 0, bs, a)) alive = false;
                if (alive && !wait(&bs->q_full, runs & 1, bs, a)) alive = false;
                auto score = [&](int jj) {  // S of the CTA's jj-th tile
                    const int it = 2 * jj, st = it % NST, b = jj & 1;
                    if (!wait(&bs->full[st], (it / NST) & 1, bs, a)) return false;
                    ptx::tc_fence_after();
                    const int n = bs->rows[st];
                    bs->s_rows[b] = n;
                    if (n > 0)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t at = (ks >> 2) * PANEL + (ks & 3) * 32;
                            ptx::mma_bf16(tmem + b * SP_COLS, ptx::smem_desc_sw128(qa + at),
                                          ptx::smem_desc_sw128(ring + st * STAGE + at), ID_S, ks > 0);
                        }
                    ptx::mma_commit(&bs->empty[st]);
                    ptx::mma_commit(&bs->s_full[b]);
                    ptx::mbar_arrive(&bs->s_full[b]);
                    return true;
                };
                auto value = [&](int jj) {  // T of the CTA's jj-th tile
                    const int it = 2 * jj + 1, st = it % NST, b = jj & 1;
                    if (!wait(&bs->full[st], (it / NST) & 1, bs, a) || !wait(&bs->p_full[b], (jj >> 1) & 1, bs, a) ||
                        (jj > 0 && !wait(&bs->t_empty, (jj - 1) & 1, bs, a)))
                        return false;
                    ptx::tc_fence_after();
                    const int n = bs->s_rows[b], steps = n / 16;
                    bs->t_rows = n;
                    // the low terms first
                    const uint32_t p = tmem + b * SP_COLS;
                    for (int term = 0; term < 3; ++term)
                        for (int ks = 0; ks < steps; ++ks) {
                            const uint32_t at = term == 1 ? 128 + 8 * ks : (ks >> 1) * 32 + (ks & 1) * 8 + (term ? 0 : 16);
                            ptx::mma_bf16_ts(tmem + T_COL, p + at,
                                             ptx::smem_desc_sw128_mn(ring + st * STAGE + ks * 2048, PANEL), ID_T,
                                             term > 0 || ks > 0);
                        }
                    ptx::mma_commit(&bs->empty[st]);
                    ptx::mma_commit(&bs->t_full);
                    ptx::mbar_arrive(&bs->t_full);
                    return true;
                };
                for (int k = 0; k <= r.n && alive; ++k) {
                    if (k < r.n) alive = score(j + k);
                    if (k > 0 && alive) alive = value(j + k - 1);
                }
            }
            alive = __shfl_sync(FULL, (int)alive, 0);
            j += r.n;
            t += r.n;
        }
    } else if (warp < 2 + SOFT_WARPS) {
        // ------------------------------------------------------------ softmax
        const int odd = (warp - 2) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t sp = tmem + ((uint32_t)(quarter * 32) << 16) + odd * SP_COLS;
        const float qs = fabsf(a.qscale);  // its sign is in the queries
        for (int t = t_begin; t < t_end && alive;) {
            const Run r = run_at(a, t, t_end, &from, lane);
            const bool busy = quarter * 32 < r.queries;  // some of the warp's queries exist
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < r.n && alive; ++k) {
                if (((j + k) & 1) != odd) continue;
                const int use = (j + k) >> 1;  // of this buffer
                if (!__all_sync(FULL, wait(&bs->s_full[odd], use & 1, bs, a)) ||
                    (use > 0 && !__all_sync(FULL, wait(&bs->m_empty[odd], (use - 1) & 1, bs, a)))) {
                    alive = false;
                    break;
                }
                const int n = bs->s_rows[odd];
                if (busy && n > 0) {
                    ptx::tc_fence_after();
                    const int chunks = (n + 31) / 32;
                    float top = -INFINITY;
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t s[32];
                        ptx::tmem_ld32(sp + c * 32, s);
                        ptx::tmem_ld_wait();
                        float t0 = -INFINITY, t1 = -INFINITY;
                        if (c * 32 + 32 <= n) {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                t0 = fmaxf(t0, __uint_as_float(s[e]));
                                t1 = fmaxf(t1, __uint_as_float(s[e + 1]));
                            }
                        } else {  // 16 rows
#pragma unroll
                            for (int e = 0; e < 16; ++e) t0 = fmaxf(t0, __uint_as_float(s[e]));
                        }
                        top = fmaxf(top, fmaxf(t0, t1));
                    }
                    const float grown = fmaxf(m, top * qs), ms = grown == -INFINITY ? 0.f : grown;
                    l *= ex2(m - ms);
                    m = grown;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t s[32], hi[16], mid[16], lo[16];
                        ptx::tmem_ld32(sp + c * 32, s);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float p[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                p[i] = ex2(fmaf(__uint_as_float(s[e + i]), qs, -ms));
                                if (e + i >= 16 && c * 32 + 32 > n) p[i] = 0.f;
                                sum[(e + i) & 3] += p[i];
                            }
                            // a float's upper 16 bits are a bf16, and what they leave is exact
                            uint32_t u[3][2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                u[0][i] = __float_as_uint(p[i]);
                                const float x = p[i] - __uint_as_float(u[0][i] & 0xffff0000u);
                                u[1][i] = __float_as_uint(x);
                                u[2][i] = __float_as_uint(x - __uint_as_float(u[1][i] & 0xffff0000u));
                            }
                            hi[e / 2] = __byte_perm(u[0][0], u[0][1], 0x7632);
                            mid[e / 2] = __byte_perm(u[1][0], u[1][1], 0x7632);
                            lo[e / 2] = __byte_perm(u[2][0], u[2][1], 0x7632);
                        }
                        // over the scores just read: upper and lower terms; the middle ones behind
                        ptx::tmem_st16(sp + c * 32, hi);
                        ptx::tmem_st16(sp + c * 32 + 16, lo);
                        ptx::tmem_st16(sp + 128 + c * 16, mid);
                    }
                    ptx::tmem_st_wait();
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    ptx::tc_fence_before();
                    sm.m[odd][row] = m;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bs->p_full[odd]);
            }
            if (alive && row < r.queries) {
                const int x = r.block * QT + row, member = x / a.g;
                const size_t query = ((size_t)(r.first + member) * a.c.heads + r.h) * a.g + (x - member * a.g);
                float4* to = r.begins ? a.row_ml + query : a.cta_ml + (size_t)blockIdx.x * QT + row;
                reinterpret_cast<float2*>(to)[odd] = make_float2(m, l);
            }
            j += r.n;
            t += r.n;
        }
    } else {
        // ------------------------------------------------------------ queries, O
        const int half = (warp - 2 - SOFT_WARPS) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, tid = threadIdx.x - 32 * (2 + SOFT_WARPS);
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + T_COL + half * 64;
        const uint32_t sign = a.qscale < 0.f ? 0x80008000u : 0u;
        // the run's queries to shared memory, swizzled as TMA does
        auto queries = [&](const Run& r) {
            for (int i = tid; i < QT * 16; i += 32 * OUT_WARPS) {
                const int y = i >> 4, piece = i & 15;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (y < r.queries) {
                    const int x = r.block * QT + y, member = x / a.g;
                    v = *reinterpret_cast<const uint4*>(a.q + (r.first + member) * a.qst[0] +
                                                        ((long long)r.h * a.g + (x - member * a.g)) * a.qst[1] + piece * 16);
                    v.x ^= sign, v.y ^= sign, v.z ^= sign, v.w ^= sign;
                }
                *reinterpret_cast<uint4*>(sm.q + (piece >> 3) * PANEL + y * 128 + (((piece & 7) ^ (y & 7)) << 4)) = v;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bs->q_full);
        };
        Run r{};
        if (t_begin < t_end) {
            r = run_at(a, t_begin, t_end, &from, lane);
            queries(r);
        }
        for (int t = t_begin; t < t_end && alive;) {
            const bool busy = quarter * 32 < r.queries;
            float o[64], m = -INFINITY;
#pragma unroll
            for (int c = 0; c < 64; ++c) o[c] = 0.f;
            for (int k = 0; k < r.n; ++k) {
                const int jj = j + k;
                if (!__all_sync(FULL, wait(&bs->t_full, jj & 1, bs, a))) {
                    alive = false;
                    break;
                }
                if (busy && bs->t_rows > 0) {
                    ptx::tc_fence_after();
                    const float mt = sm.m[jj & 1][row], grown = fmaxf(m, mt), ms = grown == -INFINITY ? 0.f : grown;
                    const float x = ex2(m - ms), y = ex2(mt - ms);
                    m = grown;
                    const bool plain = __all_sync(FULL, x == 1.f && y == 1.f);
#pragma unroll
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t v[16];
                        ptx::tmem_ld16(at + c, v);
                        ptx::tmem_ld_wait();
                        if (plain) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[c + e] += __uint_as_float(v[e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[c + e] = fmaf(o[c + e], x, __uint_as_float(v[e]) * y);
                        }
                    }
                    ptx::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(&bs->t_empty);
                    ptx::mbar_arrive(&bs->m_empty[jj & 1]);
                }
            }
            if (!alive) break;
            // every product of the run has ended with its last T: the queries make room
            const Run done = r;
            j += r.n;
            t += r.n;
            if (t < t_end) {
                r = run_at(a, t, t_end, &from, lane);
                queries(r);
            }
            if (row < done.queries) {
                const int x = done.block * QT + row, member = x / a.g;
                const size_t query = ((size_t)(done.first + member) * a.c.heads + done.h) * a.g + (x - member * a.g);
                float* to = (done.begins ? a.row_o + query * D : a.cta_o + ((size_t)blockIdx.x * QT + row) * D) + half * 64;
#pragma unroll
                for (int c = 0; c < 64; c += 4)
                    *reinterpret_cast<float4*>(to + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (bs->abort) {
        // a wait gave up: the copies asked for and the products issued get their
        // time (bounded) before shared memory and tensor memory are given back
        if (warp == 0 && lane == 0)
            for (int i = loads > NST ? loads - NST : 0; i < loads; ++i)
                ptx::mbar_wait(&bs->full[i % NST], (i / NST) & 1, a.wait_limit, nullptr);
        if (warp == 1 && lane == 0) {
            ptx::mma_commit(&bs->drain);
            ptx::mbar_wait(&bs->drain, 0, a.wait_limit, nullptr);
        }
    }
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- joining
// A warp a query, four channels a lane: what its sequence's own rows gave, in
// out and own_lse2, with the parts of its unit.
__global__ void __launch_bounds__(JOIN_WARPS * 32) paged_shared_join(const __grid_constant__ SharedArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int lane = threadIdx.x & 31, heads_q = a.c.heads * a.g;
    const long long n = (long long)a.c.seqs * heads_q, step = (long long)gridDim.x * JOIN_WARPS;
    const int total = a.tile_base[a.groups];
    const Deal deal(total, Deal::ctas(total, 1, a.grid), 1);
    for (long long query = (long long)blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5); query < n; query += step) {
        const int s = (int)(query / heads_q), hq = (int)(query - (long long)s * heads_q);
        if (a.skip[s] == 0) continue;
        const int i = a.group_of[s];
        const Group gr = a.group[i];
        const int nt = (gr.rows + KT - 1) / KT, h = hq / a.g;
        const int x = (s - gr.first) * a.g + (hq - h * a.g), block = x / QT;
        const int t0 = a.tile_base[i] + (h * gr.blocks + block) * nt;
        const int c0 = deal.cta_of(t0), c1 = deal.cta_of(t0 + nt - 1);
        float4 acc = *reinterpret_cast<const float4*>(a.out + query * D + 4 * lane);
        float m = a.own_lse2[query], l = m == -INFINITY ? 0.f : 1.f;
        for (int c = c0; c <= c1; ++c) {
            const size_t at = c == c0 ? (size_t)query : (size_t)c * QT + (x - block * QT);
            const float4 ml = (c == c0 ? a.row_ml : a.cta_ml)[at];
            const float4 o = reinterpret_cast<const float4*>((c == c0 ? a.row_o : a.cta_o) + at * D)[lane];
            const float mp = fmaxf(ml.x, ml.z);  // the maximum that O goes by
            if (mp == -INFINITY) continue;
            const float lp = ml.y * ex2(ml.x - mp) + ml.w * ex2(ml.z - mp);
            const float grown = fmaxf(m, mp), u = ex2(m - grown), v = ex2(mp - grown);
            l = l * u + lp * v;
            acc.x = acc.x * u + o.x * v;
            acc.y = acc.y * u + o.y * v;
            acc.z = acc.z * u + o.z * v;
            acc.w = acc.w * u + o.w * v;
            m = grown;
        }
        const float w = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<float4*>(a.out + query * D + 4 * lane) = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
        if (a.lse && lane == 0) a.lse[query] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
}

// ---------------------------------------------------------------- host side
struct Layout {
    size_t attn, group, tile_base, skip, group_of, row_o, row_ml, cta_o, cta_ml, total;
};
Layout layout_of(const Cache& c, int g) {
    Layout l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t S = c.seqs, queries = S * c.heads * g;
    l.attn = 0;
    l.group = up(attn_workspace(c, g, nullptr, nullptr));
    l.tile_base = l.group + up(S * sizeof(Group));
    l.skip = l.tile_base + up((S + 1) * sizeof(int));
    l.group_of = l.skip + up(S * sizeof(int));
    l.row_o = l.group_of + up(S * sizeof(int));
    l.row_ml = l.row_o + up(queries * D * sizeof(float));
    l.cta_o = l.row_ml + up(queries * sizeof(float4));
    l.cta_ml = l.cta_o + (size_t)MAX_GRID * QT * D * sizeof(float);
    l.total = l.cta_ml + (size_t)MAX_GRID * QT * sizeof(float4);
    return l;
}

cudaError_t launch_shared(SharedArgs& a, void* workspace, cudaStream_t s) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    a.grid = sms < MAX_GRID ? sms : MAX_GRID;
    a.box_rows = KT;
    while (a.c.page % a.box_rows) a.box_rows /= 2;  // pages are multiples of 16
    CUtensorMap tk, tv;
    if (!encode_pool(&tk, a.c, a.c.K, a.c.ks, true, true, a.box_rows, 1) ||
        !encode_pool(&tv, a.c, a.c.V, a.c.vs, true, true, a.box_rows, 1))
        return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(Smem) + 1024;
    static std::atomic<bool> set[MAX_DEVICES];
    if (!set[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e =
            cudaFuncSetAttribute(paged_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    cudaError_t e = launch_dependent(paged_shared_prep, dim3(1), dim3(PREP_THREADS), 0, s, a);
    if (e == cudaSuccess) e = launch_dependent(paged_shared_kernel, dim3(a.grid), dim3(THREADS), smem, s, a, tk, tv);
    const long long qst[2] = {a.qst[0] / 2, a.qst[1] / 2};
    if (e == cudaSuccess)
        e = launch_attn_own_rows(a.c, a.skip, a.q, qst, a.g, a.qscale, a.out, a.lse, workspace, s);
    const long long queries = (long long)a.c.seqs * a.c.heads * a.g, blocks = (queries + JOIN_WARPS - 1) / JOIN_WARPS;
    if (e == cudaSuccess)
        e = launch_dependent(paged_shared_join, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(JOIN_WARPS * 32), 0,
                             s, a);
    return e;
}

}  // namespace
}  // namespace paged
}  // namespace ckv

using namespace ckv;
using namespace ckv::paged;

extern "C" ckv_status ckv_paged_shared_workspace(const ckv_paged_cache* cache, int32_t g, int64_t* bytes) {
    Cache c;
    const ckv_status st = check_cache(cache, &c);
    if (st != CKV_OK) return st;
    if (!bytes || g < 1 || g > MAX_G) return CKV_ERR_ARG;
    *bytes = (int64_t)layout_of(c, g).total;
    return CKV_OK;
}

extern "C" ckv_status ckv_paged_shared_attn(const ckv_paged_cache* cache, const void* q, int32_t q_dtype,
                                            const int64_t* q_stride, int32_t g, float scale,
                                            const int32_t* group_starts, const int32_t* prefix, int32_t groups,
                                            float* out, float* lse, void* workspace, int64_t workspace_bytes,
                                            void* stream) {
    CKV_TRACE("ckv_paged_shared_attn");
    SharedArgs a = {};
    const ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (groups < 0 || groups > a.c.seqs || (groups > 0 && (!group_starts || !prefix))) return CKV_ERR_ARG;
    if (g < 1 || g > MAX_G || !workspace) return CKV_ERR_ARG;
    const Layout l = layout_of(a.c, g);
    if (workspace_bytes < (int64_t)l.total) return CKV_ERR_CAPACITY;
    if (groups == 0 || cache->kv_dtype != CKV_BF16)
        return ckv_paged_decode_attn(cache, q, q_dtype, q_stride, g, scale, out, lse, nullptr, nullptr, workspace,
                                     workspace_bytes, stream);
    if (!q || !q_stride || !out) return CKV_ERR_ARG;
    if (q_dtype != cache->kv_dtype) return CKV_ERR_DTYPE;
    a.qscale = scale * LOG2E;
    if (!isfinite(a.qscale)) return CKV_ERR_ARG;
    const long long extent[2] = {a.c.seqs, (long long)a.c.heads * g};
    for (int i = 0; i < 2; ++i) {
        if (q_stride[i] < 0 || q_stride[i] > MAX_STRIDE) return CKV_ERR_ARG;
        a.qst[i] = extent[i] > 1 ? q_stride[i] * 2 : 0;
        if (a.qst[i] & 15) return CKV_ERR_ALIGN;
    }
    // tiles, of the own rows too, are counted in 32 bits
    if (extent[0] * a.c.heads * ceil_div(a.c.rows, 8) > 0x7fff0000LL) return CKV_ERR_ARG;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return CKV_ERR_ALIGN;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    a.q = static_cast<const unsigned char*>(q);
    a.g = g;
    a.group_starts = group_starts;
    a.prefix = prefix;
    a.groups = groups;
    a.out = out;
    a.lse = lse;
    a.group = reinterpret_cast<Group*>(w + l.group);
    a.tile_base = reinterpret_cast<int*>(w + l.tile_base);
    a.skip = reinterpret_cast<int32_t*>(w + l.skip);
    a.group_of = reinterpret_cast<int*>(w + l.group_of);
    attn_workspace(a.c, g, &a.own_lse2, workspace);
    a.row_o = reinterpret_cast<float*>(w + l.row_o);
    a.row_ml = reinterpret_cast<float4*>(w + l.row_ml);
    a.cta_o = reinterpret_cast<float*>(w + l.cta_o);
    a.cta_ml = reinterpret_cast<float4*>(w + l.cta_ml);
    waits(&a.wait_limit, &a.stall);
    const cudaError_t e = launch_shared(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
