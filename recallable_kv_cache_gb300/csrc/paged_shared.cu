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

using namespace mmas;

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
constexpr int PREP_THREADS = 256;
constexpr int JOIN_ROWS = 8;
constexpr int JOIN_THREADS = JOIN_ROWS * D / 4;
// columns of tensor memory: scores and weights of two tiles, then T.  The upper
// and lower terms of 32 weights take the place of their scores, sixteen columns
// each, and the middle ones stand behind.
constexpr int NSP = 2;
constexpr uint32_t MID_COL = 128, SP_COLS = 192, T_COL = NSP * SP_COLS;

__device__ __forceinline__ float upper(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// A group as the prep leaves it.
struct Group {
    int first, members;  // sequences
    int rows;            // shared, a multiple of TILE; 0: nothing is shared
    int blocks;          // of QT queries
    int parts, cta;      // of a unit, and the CTA of the group's first one, where units have CTAs of their own
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
    int* ctas;          // [1] CTAs that have a unit's part, 0: the even deal
    float* own_lse2;    // [seqs * heads * g] of the sequences' own rows, base 2
    // Parts: O as [channel / 4][query of the block] of four, and (maximum, sum) of
    // even and odd tiles.  The CTA in which a unit begins leaves its part behind
    // those of the units before it, the others (each continues one at most) by CTA.
    float4* unit_o;     // [seqs * heads * g][D / 4] in all
    float4* unit_ml;    // [seqs * heads * g]
    float4* cta_o;      // [MAX_GRID][D / 4][QT]
    float4* cta_ml;     // [MAX_GRID][QT]
    int grid;
    long long wait_limit;
    int stall;
};

// ---------------------------------------------------------------- the groups
// sums (or maxima) of v over the threads before, and over all
template <bool MAX>
__device__ __forceinline__ int scan(int v, int* warp_val, int* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x = MAX ? max(x, y) : x + y;
    }
    if (lane == 31) warp_val[warp] = x;
    __syncthreads();
    int before = __shfl_up_sync(FULL, x, 1);
    if (lane == 0) before = 0;
    int total = 0;
#pragma unroll
    for (int w = 0; w < PREP_THREADS / 32; ++w) {
        if (w < warp) before = MAX ? max(before, warp_val[w]) : before + warp_val[w];
        total = MAX ? max(total, warp_val[w]) : total + warp_val[w];
    }
    __syncthreads();
    *all = total;
    return before;
}

// One CTA.  A thread has a chunk of neighbouring groups, then of sequences.
// How the tiles are dealt out: evenly, a CTA's share beginning and ending
// anywhere, or every unit in equal parts of its own to whole CTAs.  Where a
// share passes from one unit to the next the products wait for the new queries
// and the softmax for the products, as long as some two tiles, so the second
// deal is taken where its largest part is at most OWN_EXTRA tiles above an even
// share.
constexpr int OWN_EXTRA = 2;
__global__ void __launch_bounds__(PREP_THREADS) paged_shared_prep(const __grid_constant__ SharedArgs a) {
    __shared__ int warp_val[PREP_THREADS / 32];
    __shared__ int ctas_with[OWN_EXTRA + 1];
    const int tid = threadIdx.x;
    if (tid <= OWN_EXTRA) ctas_with[tid] = 0;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int chunk = (a.groups + PREP_THREADS - 1) / PREP_THREADS;
    const int i0 = min(a.groups, tid * chunk), i1 = min(a.groups, i0 + chunk);
    auto start_at = [&](int i) { return min(max(a.group_starts[i], 0), a.c.seqs); };
    auto tiles_of = [](const Group& gr) { return (gr.rows + KT - 1) / KT; };
    // starts ascend: each is at least the largest before it
    int top = 0, all;
    for (int i = i0; i < i1; ++i) {
        const int raw = a.group_starts[i];
        if (raw < 0 || raw > a.c.seqs || raw > a.group_starts[i + 1] || a.prefix[i] < 0)
            report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        top = max(top, start_at(i));
    }
    int before = scan<true>(top, warp_val, &all), tiles = 0;
    for (int i = i0; i < i1; ++i) {
        const int first = max(before, start_at(i)), end = max(first, start_at(i + 1));
        before = first;
        Group gr{first, end - first, 0, 0, 0, 0};
        if (gr.members > 1) {
            gr.rows = min(max(a.prefix[i], 0), rows_held(a.c, first)) / TILE * TILE;
            gr.blocks = (int)(((long long)gr.members * a.g + QT - 1) / QT);
        }
        a.group[i] = gr;
        tiles += a.c.heads * gr.blocks * tiles_of(gr);
    }
    int total, at = scan<false>(tiles, warp_val, &total);
    const int even = (total + a.grid - 1) / a.grid;
    int ctas[OWN_EXTRA + 1] = {};
    for (int i = i0; i < i1; ++i) {
        a.tile_base[i] = at;
        const Group gr = a.group[i];
        const int nt = tiles_of(gr), units = a.c.heads * gr.blocks;
        at += units * nt;
        for (int x = 0; x <= OWN_EXTRA && even > 0; ++x)
            ctas[x] = min(a.grid + 1, ctas[x] + min(a.grid + 1, units) * min(a.grid + 1, (nt + even + x - 1) / (even + x)));
    }
    for (int x = 0; x <= OWN_EXTRA; ++x)
        if (ctas[x]) atomicAdd(&ctas_with[x], ctas[x]);
    if (tid == 0) {
        a.tile_base[a.groups] = total;
        const int end = a.group_starts[a.groups];
        if (end < 0 || end > a.c.seqs) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
    }
    __syncthreads();
    int part = 0;  // tiles of a part, 0: the even deal
    for (int x = OWN_EXTRA; x >= 0; --x)
        if (total > 0 && ctas_with[x] <= a.grid) part = even + x;
    int mine = 0;
    for (int i = i0; i < i1 && part; ++i) {
        const Group gr = a.group[i];
        mine += a.c.heads * gr.blocks * ((tiles_of(gr) + part - 1) / part);
    }
    at = scan<false>(mine, warp_val, &all);
    for (int i = i0; i < i1 && part; ++i) {
        a.group[i].parts = (tiles_of(a.group[i]) + part - 1) / part;
        a.group[i].cta = at;
        at += a.c.heads * a.group[i].blocks * a.group[i].parts;
    }
    if (tid == 0) *a.ctas = part ? all : 0;
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

// the group that tile t (one of those there are) belongs to, found by a warp
__device__ __forceinline__ int group_of_tile(const SharedArgs& a, int t, int from, int lane) {
    for (int i = from; i < a.groups; i += 32) {
        const bool past = i + lane < a.groups && a.tile_base[i + lane + 1] <= t;
        const unsigned m = __ballot_sync(FULL, past);
        if (m != FULL) return i + __popc(m);
    }
    return a.groups - 1;
}
// the tiles of a CTA
__device__ __forceinline__ int2 share_of(const SharedArgs& a, int cta, int lane) {
    const int total = a.tile_base[a.groups], ctas = *a.ctas;
    if (ctas == 0) {
        const Deal deal(total, Deal::ctas(total, 1, a.grid), 1);
        if (cta >= deal.n_cta || total == 0) return make_int2(0, 0);
        return make_int2(deal.begin_cta(cta), deal.begin_cta(cta + 1));
    }
    if (cta >= ctas) return make_int2(0, 0);
    // the last group with CTAs that begins at this one or before
    int i = 0;
    for (int b = 0; b < a.groups; b += 32) {
        const bool here = b + lane < a.groups && a.group[b + lane].parts > 0 && a.group[b + lane].cta <= cta;
        const unsigned m = __ballot_sync(FULL, here);
        if (m) i = b + 31 - __clz(m);
    }
    const Group gr = a.group[i];
    const int nt = (gr.rows + KT - 1) / KT, unit = (cta - gr.cta) / gr.parts, p = cta - gr.cta - unit * gr.parts;
    const int t = a.tile_base[i] + unit * nt;
    return make_int2(t + (int)((long long)nt * p / gr.parts), t + (int)((long long)nt * (p + 1) / gr.parts));
}

// A CTA's share of one unit.
struct Run {
    int group, first, members, rows;
    int h, block;  // KV head, block of queries
    int k0, n;     // tiles [k0, k0 + n) of the unit
    int queries;   // in the block
    bool begins;   // with the unit's first tile
    long long row; // of the block's first query among all units'
};
// The block's queries in the order of the parts: group, KV head, member, query head.
__device__ __forceinline__ long long row_of(const SharedArgs& a, const Group& gr, int h, int block) {
    return ((long long)gr.first * a.c.heads + (long long)h * gr.members) * a.g + (long long)block * QT;
}
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
    r.row = row_of(a, gr, r.h, r.block);
    return r;
}

// Places of a CTA's j-th K and V in the order of the loads: K0 K1 V0 K2 V1 ...
__device__ __forceinline__ int k_index(int j) { return j < 1 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_index(int j) { return 2 * j + 2; }

struct __align__(8) Bars {
    uint64_t full[NST], empty[NST];
    uint64_t q_full;
    uint64_t s_full[NSP], p_full[NSP], m_empty[NSP];
    uint64_t t_full, t_empty;
    uint64_t never, drain;
    int asked[NST];    // the last phase of a stage that was asked for
    int rows[NST];     // of a K stage's tile: those whose page is good
    int s_rows[NSP], t_rows;
    uint32_t tmem_base;
    int abort;
};
struct __align__(1024) Smem {
    unsigned char q[STAGE];
    unsigned char ring[NST][STAGE];
    float m[NSP][QT];  // the maxima that a tile's weights go by
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
            bs->asked[i] = -1;
        }
        ptx::mbar_init(&bs->q_full, OUT_WARPS);
        for (int i = 0; i < NSP; ++i) {
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

    const int2 share = share_of(a, blockIdx.x, lane);
    const int t_begin = share.x, t_end = share.y, n_tiles = t_end - t_begin;
    bool alive = true;
    int from = 0;  // the group to look from
    int j = 0;     // tiles so far
    const bool leader = ptx::elect_one();  // the lane of warp 1 that issues the products

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // In the order in which the products take them: K of a tile, then V of
        // the tile before it.
        if (lane < 2) ptx::prefetch_tmap(lane ? &tv : &tk);
        const FastDiv& by_page = a.c.by_page;
        // this lane's copy of a tile: its page (-1: none), slot and place in the
        // stage; the tile's copies and rows, and its KV head
        struct Copy {
            int page, slot, place, copies, rows, h;
        };
        Copy now{}, last{};
        auto load = [&](const Copy& c, int idx, const CUtensorMap* map) {
            const int st = idx % NST;
            if (idx >= NST && !__all_sync(FULL, wait(&bs->empty[st], (idx / NST - 1) & 1, bs, a))) return false;
            if (lane == 0) {
                bs->asked[st] = idx / NST;
                bs->rows[st] = c.rows;
                if (c.copies) ptx::mbar_arrive_expect_tx(&bs->full[st], c.copies * a.box_rows * 256);
                else ptx::mbar_arrive(&bs->full[st]);
            }
            __syncwarp();
            if (c.page >= 0) {
                unsigned char* to = sm.ring[st] + c.place * a.box_rows * 128;
#pragma unroll
                for (int piece = 0; piece < 2; ++piece)
                    asm volatile(
                        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(ptx::smem_u32(to + piece * PANEL)),
                        "l"(map), "r"(0), "r"(c.slot), "r"(piece), "r"(c.h), "r"(c.page),
                        "r"(ptx::smem_u32(&bs->full[st]))
                        : "memory");
            }
            __syncwarp();
            return true;
        };
        Run r{};
        int k = 0, k_end = 0;
        for (; j <= n_tiles && alive; ++j) {
            last = now;
            if (j < n_tiles) {
                if (k == k_end) {
                    r = run_at(a, t_begin + j, t_end, &from, lane);
                    k = r.k0;
                    k_end = r.k0 + r.n;
                }
                // lane l looks after the tile's l-th copy
                const int row = k * KT + lane * a.box_rows;
                now.page = -1;
                now.h = r.h;
                if (lane * a.box_rows < KT && row < r.rows) {
                    now.page = a.c.table[(size_t)r.first * a.c.max_pages + by_page.quot(row, &now.slot)];
                    if (now.page < 0 || now.page >= a.c.n_pages) {
                        report(a.c.dev_err, CKV_DEV_BAD_INDEX);
                        now.page = -1;
                    }
                }
                // rows of bad pages are left out: the others move up
                const unsigned good = __ballot_sync(FULL, now.page >= 0);
                now.place = __popc(good & ((1u << lane) - 1u));
                now.copies = __popc(good);
                now.rows = now.copies * a.box_rows -
                           __reduce_max_sync(FULL, now.page >= 0 ? max(0, row + a.box_rows - r.rows) : 0);
                ++k;
                alive = load(now, k_index(j), &tk);
                // the first K before all else: with every stage asked for at once
                // it came with the last of them, 4 us later
                if (j == 0 && alive) alive = __all_sync(FULL, wait(&bs->full[0], 0, bs, a));
            }
            if (j > 0 && alive) alive = load(last, v_index(j - 1), &tv);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ the products
        const uint32_t ring = ptx::smem_u32(sm.ring), qa = ptx::smem_u32(sm.q);
        constexpr uint32_t ID_S = ptx::idesc_bf16_f32(QT, KT);
        constexpr uint32_t ID_T = ptx::idesc_bf16_f32(QT, D) | ptx::IDESC_B_MN_MAJOR;
        int runs = 0;
        // all lanes keep step for the runs; one waits and issues
        for (int t = t_begin; t < t_end && alive; ++runs) {
            const Run r = run_at(a, t, t_end, &from, lane);
            if (leader) {
                if (runs == 0 && a.stall && !wait(&bs->never, 0, bs, a)) alive = false;
                if (alive && !wait(&bs->q_full, runs & 1, bs, a)) alive = false;
                auto score = [&](int jj) {  // S of the CTA's jj-th tile
                    const int it = k_index(jj), st = it % NST, b = jj % NSP;
                    if (!wait(&bs->full[st], (it / NST) & 1, bs, a)) return false;
                    ptx::tc_fence_after();
                    const int n = bs->rows[st];
                    bs->s_rows[b] = n;
                    const uint64_t qd = ptx::smem_desc_sw128(qa), kd = ptx::smem_desc_sw128(ring + st * STAGE);
                    if (n > 0)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t at = ((ks >> 2) * PANEL + (ks & 3) * 32) >> 4;
                            ptx::mma_bf16(tmem + b * SP_COLS, qd + at, kd + at, ID_S, ks > 0);
                        }
                    ptx::mma_commit(&bs->empty[st]);
                    ptx::mma_commit(&bs->s_full[b]);
                    ptx::mbar_arrive(&bs->s_full[b]);
                    return true;
                };
                auto value = [&](int jj) {  // T of the CTA's jj-th tile
                    const int it = v_index(jj), st = it % NST, b = jj % NSP;
                    if (!wait(&bs->full[st], (it / NST) & 1, bs, a) || !wait(&bs->p_full[b], (jj / NSP) & 1, bs, a) ||
                        (jj > 0 && !wait(&bs->t_empty, (jj - 1) & 1, bs, a)))
                        return false;
                    ptx::tc_fence_after();
                    const int n = bs->s_rows[b], steps = n / 16;
                    bs->t_rows = n;
                    // the low terms first; eight columns hold a term of 16 rows
                    const uint32_t p = tmem + b * SP_COLS;
                    const uint64_t v = ptx::smem_desc_sw128_mn(ring + st * STAGE, PANEL);
#pragma unroll
                    for (int term = 0; term < 3; ++term)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t at = term == 1 ? MID_COL + 8 * ks : (ks >> 1) * 32 + (ks & 1) * 8 + (term ? 0 : 16);
                            if (ks < steps)
                                ptx::mma_bf16_ts(tmem + T_COL, p + at, v + (ks * 2048 >> 4), ID_T, term > 0 || ks > 0);
                        }
                    ptx::mma_commit(&bs->empty[st]);
                    ptx::mma_commit(&bs->t_full);
                    ptx::mbar_arrive(&bs->t_full);
                    return true;
                };
                // scores run a tile ahead of the values, into the buffer that the
                // value before has read
                for (int k = 0; k <= r.n && alive; ++k) {
                    if (k < r.n) alive = score(j + k);
                    if (k > 0 && alive) alive = value(j + k - 1);
                }
            }
            alive = __all_sync(FULL, alive);
            j += r.n;
            t += r.n;
        }
    } else if (warp < 2 + SOFT_WARPS) {
        // ------------------------------------------------------------ softmax
        const int odd = (warp - 2) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        // its sign is in the queries; not 0, so that it leaves -inf what it is
        const float qs = fmaxf(fabsf(a.qscale), 1.17549435e-38f);
        const uint64_t qs2 = pair(qs, qs), minus2 = pair(-1.f, -1.f);
        for (int t = t_begin; t < t_end && alive;) {
            const Run r = run_at(a, t, t_end, &from, lane);
            const bool busy = quarter * 32 < r.queries;  // some of the warp's queries exist
            float m = -INFINITY, l = 0.f;
            for (int k = (j & 1) == odd ? 0 : 1; k < r.n; k += 2) {
                const int b = (j + k) % NSP, use = (j + k) / NSP;
                const uint32_t sp = tmem + ((uint32_t)(quarter * 32) << 16) + b * SP_COLS;
                if (!__all_sync(FULL, wait(&bs->s_full[b], use & 1, bs, a)) ||
                    (use > 0 && !__all_sync(FULL, wait(&bs->m_empty[b], (use - 1) & 1, bs, a)))) {
                    alive = false;
                    break;
                }
                const int n = bs->s_rows[b];
                if (busy && n > 0) {
                    ptx::tc_fence_after();
                    const int chunks = (n + 31) / 32;
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t s[32];
                        ptx::tmem_ld32(sp + c * 32, s);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
                        if (c * 32 + 32 <= n)  // else 16 rows
#pragma unroll
                            for (int e = 16; e < 32; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(s[e]));
                    }
                    const float grown = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * qs);
                    const float ms = grown == -INFINITY ? 0.f : grown;
                    l *= ex2(m - ms);
                    m = grown;
                    const uint64_t ms2 = pair(-ms, -ms);
                    uint64_t sum[2] = {0, 0};
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t s[32], hi[16], mid[16], lo[16];
                        ptx::tmem_ld32(sp + c * 32, s);
                        ptx::tmem_ld_wait();
                        if (c * 32 + 32 > n)  // 16 rows: the others weigh nothing
#pragma unroll
                            for (int e = 16; e < 32; ++e) s[e] = 0xff800000u;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 x = unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), qs2, ms2));
                            const float p0 = ex2(x.x), p1 = ex2(x.y);
                            const uint64_t p = pair(p0, p1);
                            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], p);
                            // a float's upper 16 bits are a bf16, and what they leave is exact
                            hi[e / 2] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                            const uint64_t rest = fma2(pair(upper(p0), upper(p1)), minus2, p);
                            const float2 y = unpair(rest);
                            mid[e / 2] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
                            const float2 z = unpair(fma2(pair(upper(y.x), upper(y.y)), minus2, rest));
                            lo[e / 2] = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
                        }
                        ptx::tmem_st16(sp + c * 32, hi);
                        ptx::tmem_st16(sp + c * 32 + 16, lo);
                        ptx::tmem_st16(sp + MID_COL + c * 16, mid);
                    }
                    ptx::tmem_st_wait();
                    const float2 x = unpair(add2(sum[0], sum[1]));
                    l += x.x + x.y;
                    ptx::tc_fence_before();
                    sm.m[b][row] = m;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bs->p_full[b]);
            }
            if (alive && row < r.queries)
                reinterpret_cast<float2*>(r.begins ? a.unit_ml + r.row + row
                                                   : a.cta_ml + (size_t)blockIdx.x * QT + row)[odd] = make_float2(m, l);
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
            const int piece = tid & 15;
            uint4 v[QT * 16 / (32 * OUT_WARPS)];
#pragma unroll
            for (int i = 0; i < QT * 16 / (32 * OUT_WARPS); ++i) {
                const int y = (tid >> 4) + i * 2 * OUT_WARPS;
                v[i] = make_uint4(0, 0, 0, 0);
                if (y < r.queries) {
                    const int x = r.block * QT + y, member = x / a.g;
                    v[i] = *reinterpret_cast<const uint4*>(a.q + (r.first + member) * a.qst[0] +
                                                           ((long long)r.h * a.g + (x - member * a.g)) * a.qst[1] + piece * 16);
                    v[i].x ^= sign, v[i].y ^= sign, v[i].z ^= sign, v[i].w ^= sign;
                }
            }
#pragma unroll
            for (int i = 0; i < QT * 16 / (32 * OUT_WARPS); ++i) {
                const int y = (tid >> 4) + i * 2 * OUT_WARPS;
                *reinterpret_cast<uint4*>(sm.q + (piece >> 3) * PANEL + y * 128 + (((piece & 7) ^ (y & 7)) << 4)) = v[i];
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
                    const float mt = sm.m[jj % NSP][row], grown = fmaxf(m, mt), ms = grown == -INFINITY ? 0.f : grown;
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
                    ptx::mbar_arrive(&bs->m_empty[jj % NSP]);
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
                const int stride = done.begins ? done.queries : QT;
                float4* to = (done.begins ? a.unit_o + done.row * (D / 4) : a.cta_o + (size_t)blockIdx.x * QT * (D / 4)) +
                             half * 16 * stride + row;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    to[c * stride] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (bs->abort) {
        // a wait gave up: the copies asked for and the products issued get their
        // time (bounded) before shared memory and tensor memory are given back
        if (warp == 0 && lane == 0)
            for (int i = 0; i < NST; ++i)
                if (bs->asked[i] >= 0) ptx::mbar_wait(&bs->full[i], bs->asked[i] & 1, a.wait_limit, nullptr);
        if (warp == 1 && leader) {
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
// What the sequences' own rows gave, in out and own_lse2, with the parts of the
// units.  A block has eight queries in the order of the parts, a thread four
// channels of one, so that a part's channels come in whole lines; PARTS parts
// are under way at a time (one after the other 20 parts took 12 us).
constexpr int PARTS = 8;
__global__ void __launch_bounds__(JOIN_THREADS) paged_shared_join(const __grid_constant__ SharedArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int channel = threadIdx.x / JOIN_ROWS, heads_q = a.c.heads * a.g;  // four channels
    const long long n = (long long)a.c.seqs * heads_q, step = (long long)gridDim.x * JOIN_ROWS;
    const int total = a.tile_base[a.groups], ctas = *a.ctas;
    const Deal deal(total, Deal::ctas(total, 1, a.grid), 1);
    for (long long row = (long long)blockIdx.x * JOIN_ROWS + threadIdx.x % JOIN_ROWS; row < n; row += step) {
        const int some = (int)(row / heads_q);  // a sequence of the group
        if (a.skip[some] == 0) continue;
        const int i = a.group_of[some];
        const Group gr = a.group[i];
        const int nt = (gr.rows + KT - 1) / KT, all = gr.members * a.g;
        const int left = (int)(row - (long long)gr.first * heads_q), h = left / all, x = left - h * all;
        const int block = x / QT, y = x - block * QT, queries = min(QT, all - block * QT), unit = h * gr.blocks + block;
        const int member = x / a.g;
        const size_t query = (size_t)(gr.first + member) * heads_q + h * a.g + (x - member * a.g);
        const int t0 = a.tile_base[i] + unit * nt;
        const int c0 = ctas ? gr.cta + unit * gr.parts : deal.cta_of(t0);
        const int parts = ctas ? gr.parts : deal.cta_of(t0 + nt - 1) - c0 + 1;
        float4* out = reinterpret_cast<float4*>(a.out + query * D) + channel;
        float4 acc = *out;
        float m = a.own_lse2[query], l = m == -INFINITY ? 0.f : 1.f;
        for (int p0 = 0; p0 < parts; p0 += PARTS) {
            float4 o[PARTS], ml[PARTS];
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const int p = p0 + k;
                ml[k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                if (p < parts) {
                    ml[k] = p ? a.cta_ml[(size_t)(c0 + p) * QT + y] : a.unit_ml[row];
                    o[k] = p ? a.cta_o[((size_t)(c0 + p) * (D / 4) + channel) * QT + y]
                             : a.unit_o[(row - y) * (D / 4) + channel * queries + y];
                }
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const float mp = fmaxf(ml[k].x, ml[k].z);  // the maximum that O goes by
                if (mp == -INFINITY) continue;
                const float lp = ml[k].y * ex2(ml[k].x - mp) + ml[k].w * ex2(ml[k].z - mp);
                const float grown = fmaxf(m, mp), u = ex2(m - grown), v = ex2(mp - grown);
                l = l * u + lp * v;
                acc.x = acc.x * u + o[k].x * v;
                acc.y = acc.y * u + o[k].y * v;
                acc.z = acc.z * u + o[k].z * v;
                acc.w = acc.w * u + o[k].w * v;
                m = grown;
            }
        }
        const float w = l == 0.f ? 0.f : 1.f / l;
        *out = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
        if (a.lse && channel == 0) a.lse[query] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
}

// ---------------------------------------------------------------- host side
struct Layout {
    size_t attn, group, tile_base, skip, group_of, ctas, unit_o, unit_ml, cta_o, cta_ml, total;
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
    l.ctas = l.group_of + up(S * sizeof(int));
    l.unit_o = l.ctas + up(sizeof(int));
    l.unit_ml = l.unit_o + up(queries * D * sizeof(float));
    l.cta_o = l.unit_ml + up(queries * sizeof(float4));
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
    const long long queries = (long long)a.c.seqs * a.c.heads * a.g, blocks = (queries + JOIN_ROWS - 1) / JOIN_ROWS;
    if (e == cudaSuccess)
        e = launch_dependent(paged_shared_join, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(JOIN_THREADS), 0, s, a);
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
    a.ctas = reinterpret_cast<int*>(w + l.ctas);
    a.unit_o = reinterpret_cast<float4*>(w + l.unit_o);
    a.unit_ml = reinterpret_cast<float4*>(w + l.unit_ml);
    a.cta_o = reinterpret_cast<float4*>(w + l.cta_o);
    a.cta_ml = reinterpret_cast<float4*>(w + l.cta_ml);
    waits(&a.wait_limit, &a.stall);
    const cudaError_t e = launch_shared(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
