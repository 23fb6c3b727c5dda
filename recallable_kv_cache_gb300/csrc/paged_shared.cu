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
//   P = 2^{S scale - m}  m a query's running maximum, P in the place of S
//   T = P V             P from tensor memory, as three bf16 terms
//   O = O a + T         in registers, a = 2^{m before - m}
// A weight is the sum of three bf16 terms (its upper, middle and lower eight
// bits), so that the products are those of fp32 weights.  With one term outputs
// would be off by 2^-9, with two by 1.4e-6 of the largest, with three by 4e-7,
// which is what the decode attention of this library is off by.  That makes four
// products a tile, 1.33 us at the measured dense rate, against 1.5 us that an SM's
// share of HBM takes for the tile's 64 KB.  T starts from zero at each tile
// and joins O by an ordinary addition, as the tensor core truncates what it
// accumulates and O grows over hundreds of tiles; that also leaves O's scaling
// off the path from one tile's maximum to the next one's product.
// What bounds a long run of tiles is the way of a tile through the roles below,
// about 1.5 us (32 sequences behind 64k rows, 8 heads of 4 queries: 61 us, 4.4
// TB/s of their 268 MB): scores, some 2500 cycles of softmax, products and the
// steps between them come to 6000 for each of the two buffers that tensor memory
// has room for.  Slower were two groups of softmax warps that each took every
// other tile, T in two halves of 64 channels, T begun with half of the rows while
// the softmax is at the others, sixteen warps for both softmax and O, and
// registers moved from the other roles to the softmax's (by 3 to 9 % for 160
// sequences behind 16k rows, which take 71 us).
// Warp roles:
//   warps 0, 18  ask for the tiles of K and of V (TMA)
//   warp 1       owns tensor memory, issues S and T
//   warps 2-9    softmax, a thread 64 rows of a query
//   warps 10-17  queries to shared memory; O, a thread 64 channels of a query
// Where a unit is several CTAs' its parts are joined by the last kernel in the
// order of its rows, so that results do not depend on timing.
#include <cuda.h>
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
constexpr int KT = 128;              // rows of a tile
constexpr int QT = 128;              // queries of a tile
constexpr int PANEL = 128 * 128;     // 64 channels of 128 rows
constexpr int STAGE = 2 * PANEL;     // K or V of a tile
constexpr int NST = 6;
constexpr int SOFT_WARPS = 8, OUT_WARPS = 8;
constexpr int V_WARP = 2 + SOFT_WARPS + OUT_WARPS;
constexpr int THREADS = 32 * (V_WARP + 1);
constexpr int PREP_THREADS = 256;
constexpr int JOIN_ROWS = 4;
constexpr int JOIN_THREADS = JOIN_ROWS * D / 4;
// columns of tensor memory: scores and weights of two tiles, then T.  The upper
// and lower terms of 32 weights take the place of their scores, sixteen columns
// each, and the middle ones stand behind.
constexpr int NSP = 2;
constexpr uint32_t LOW_COL = 16, MID_COL = 128, SP_COLS = 192, T_COL = NSP * SP_COLS;

// Two bf16 in a register, as floats.  (Taken from the packed pair, as the shift
// can be a multiplication: packing and masking take the other unit up.)
__device__ __forceinline__ uint64_t floats(uint32_t x) {
    return pair(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// A group as the prep leaves it.
struct Group {
    int first, members;  // sequences
    int rows;            // shared, a multiple of TILE; 0: nothing is shared
    int blocks;          // of QT queries
    int parts, cta;      // of a unit, and the CTA of the group's first one, where units have CTAs of their own
};

// A CTA's share of a unit.
struct Run {
    int first, members, rows;  // of the group
    int h, block;              // KV head, block of queries
    int k0, n;                 // tiles [k0, k0 + n) of the unit
};
// The tiles [t, t_end) of a CTA, the group of the first, and the run it is in.
struct __align__(16) Share {
    int t, t_end, group, pad[2];
    Run run;
};
static_assert(sizeof(Share) == 48, "read as three times 16 bytes");

struct SharedArgs {
    Cache c;
    const unsigned char* q;
    long long qst[2];  // byte strides: sequence, query head
    int g;
    FastDiv by_g;
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
    Share* share;       // [grid]
    int2* deal;         // [1] CTAs with a unit's part, 0: the even deal; CTAs that it goes to
    int* own_ctas;      // [1] CTAs for the sequences' own rows
    // the sequences' own rows: the lse (base 2) [seqs * heads * g], parts, and
    // what there is of a unit [seqs * heads]
    float* own_lse2;
    const float* own_part;
    int32_t* own_left;
    // Parts: O as [channel / 4][query of the block] of four, and for either half
    // of the tiles' rows (the maximum that O goes by, the sum).  The CTA in which
    // a unit begins leaves its part behind those of the units before it, the
    // others (each continues one at most) by CTA.
    float4* unit_o;     // [seqs * heads * g][D / 4] in all
    float4* unit_ml;    // [seqs * heads * g]
    float4* cta_o;      // [MAX_GRID][D / 4][QT]
    float4* cta_ml;     // [MAX_GRID][QT]
    int grid;
    long long wait_limit;
    int stall;
};

// ---------------------------------------------------------------- the groups
// the sum of v over the lanes before (the largest of theirs where MAX), v not negative
template <bool MAX>
__device__ __forceinline__ int lanes_before(int v, int lane) {
    int x = __shfl_up_sync(FULL, v, 1);
    if (lane == 0) x = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x = MAX ? max(x, y) : x + y;
    }
    return x;
}
// the same over the threads of the CTA, and over all
template <bool MAX>
__device__ __forceinline__ int2 threads_before(int v, int* warp_val) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = lanes_before<MAX>(v, lane), all = 0;
    if (lane == 31) warp_val[warp] = MAX ? max(x, v) : x + v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < PREP_THREADS / 32; ++w) {
        const int y = warp_val[w];
        if (w < warp) x = MAX ? max(x, y) : x + y;
        all = MAX ? max(all, y) : all + y;
    }
    __syncthreads();
    return make_int2(x, all);
}
__device__ __forceinline__ int parts_of(int n, int d) { return (int)(((unsigned)n + d - 1) / (unsigned)d); }
__device__ __forceinline__ int tiles_of(const Group& gr) { return (int)((unsigned)(gr.rows + KT - 1) / KT); }

// How the SMs and the tiles are dealt out.
//
// The shared rows and the sequences' own rows are attended side by side, on SMs
// of their own (one after the other the second would begin with some 4 us of
// latency and end with as much, while HBM idles).  One SM would take TILE_COST
// for a tile of shared rows, OWN_COST for 16 own rows of a KV head and UNIT_COST
// for each (sequence, KV head) with some, and merging the latter takes
// MERGE_COST longer at the end: the P SMs of the G there are for the shared rows
// are those with which both end together, x / P = y / (G - P) + MERGE_COST.  (Found
// by trying over the cases that have both: a tile by itself takes 1.5, the rest is
// a share of what comes before and after.  TILE_COST 1.5 and 1.7, OWN_COST .15 to
// .18, UNIT_COST .1 and .4, MERGE_COST 3 to 10 were equal to 8 % slower.)
//
// The tiles of shared rows go to CTAs evenly, a CTA's share beginning and ending
// anywhere, or every unit goes in equal parts to CTAs of its own.  Where a share
// passes from one unit to the next the products wait for the new queries and the
// softmax for the products, as long as some three tiles, so the second deal is
// taken where its largest part is at most OWN_EXTRA tiles above an even share.
constexpr float TILE_COST = 1.6f, OWN_COST = 0.13f, UNIT_COST = 0.2f, MERGE_COST = 6.f;  // us
constexpr int OWN_EXTRA = 3;
// The SMs for the shared rows, of `grid`: `total` tiles of these, and of the own
// rows `own` tiles of 16 of `units` (sequence, KV head) pairs.
__device__ __forceinline__ int ctas_for_shared(int grid, int total, float own, int units) {
    if (total == 0 || units == 0) return total ? grid : 0;
    if (total + (long long)units <= grid) return total;  // an SM for each
    const float x = total * TILE_COST, y = own * OWN_COST + units * UNIT_COST;
    // P = x / t, G - P = y / (t - MERGE_COST)
    const float b = grid * MERGE_COST + x + y, root = __fsqrt_rn(b * b - 4.f * grid * MERGE_COST * x);
    return max(1, min(grid - 1, (int)(__fdividef(2.f * grid * x, b + root) + 0.5f)));
}
// the run that begins at tile t, in a group whose tiles begin at `base`, of a share that ends at t_end
__device__ __forceinline__ Run run_in(const Group& gr, int base, int t, int t_end) {
    const int nt = tiles_of(gr), unit = (int)((unsigned)(t - base) / (unsigned)nt), k0 = t - base - unit * nt;
    const int h = (int)((unsigned)unit / (unsigned)gr.blocks);
    return Run{gr.first, gr.members, gr.rows, h, unit - h * gr.blocks, k0, min(nt - k0, t_end - t)};
}

// One CTA.  A thread has a chunk of neighbouring groups, then every
// PREP_THREADS-th sequence, then CTAs.  FEW: at most 32 groups, which are warp
// 0's, a lane each, and FEW_SEQS sequences, with their numbers in shared memory.
// It is the latency of a chain of small steps, 1.1 us of it the first loads.
// LENS: fp32 rows, which every sequence attends by itself.  The groups are looked
// at all the same, and skip[s] becomes the rows that s attends: its own number, or
// the group's where that is more.  (Few groups the attention looks at itself: 12
// sequences of two groups took 22 us with this in front, 20 without.)
template <bool FEW, bool LENS>
__global__ void __launch_bounds__(PREP_THREADS) paged_shared_prep(const __grid_constant__ SharedArgs a) {
    __shared__ int warp_val[PREP_THREADS / 32];
    __shared__ int ctas_with[OWN_EXTRA + 1], own_tiles, own_units, of_deal[4];
    __shared__ Group group_here[FEW ? FEW_GROUPS : 1];
    __shared__ int base_here[FEW ? FEW_GROUPS : 1], lens_here[FEW ? FEW_SEQS : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid <= OWN_EXTRA) ctas_with[tid] = 0;
    if (tid == 0) own_tiles = own_units = 0;
    Group* group = FEW ? group_here : a.group;
    int* base = FEW ? base_here : a.tile_base;
    const int* lens = FEW ? lens_here : a.c.lens;
    const int chunk = FEW ? 1 : (a.groups + PREP_THREADS - 1) / PREP_THREADS;
    const int i0 = min(a.groups, tid * chunk), i1 = min(a.groups, i0 + chunk);
    auto before = [&](bool largest, int v) {
        if (FEW) {
            const int x = largest ? lanes_before<true>(v, lane) : lanes_before<false>(v, lane);
            return make_int2(x, __shfl_sync(FULL, x + v, 31));  // (the largest of all is not asked for)
        }
        return largest ? threads_before<true>(v, warp_val) : threads_before<false>(v, warp_val);
    };
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    // what goes by no other load, side by side
    int start = 0, next = 0, shared = 0;
    if (FEW) {
#pragma unroll 1
        for (int s = tid; s < a.c.seqs; s += PREP_THREADS) lens_here[s] = a.c.lens[s];
        if (i0 < i1) {
            start = a.group_starts[i0];
            next = a.group_starts[i0 + 1];
            shared = a.prefix[i0];
        }
        __syncthreads();
    }
    int total = 0, sum = 0;
    if (!FEW || warp == 0) {
        // starts ascend: each is at least the largest before it
        int top = 0, tiles = 0;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            if (!FEW) start = a.group_starts[i], next = a.group_starts[i + 1], shared = a.prefix[i];
            if (start < 0 || next > a.c.seqs || start > next || shared < 0) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
            top = max(top, min(start, a.c.seqs));
        }
        int from = before(true, top).x;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            if (!FEW) start = a.group_starts[i], next = a.group_starts[i + 1], shared = a.prefix[i];
            const int first = max(from, min(start, a.c.seqs)), members = max(first, min(next, a.c.seqs)) - first;
            from = first;
            Group gr{first, members, 0, 0, 0, 0};
            if (members > 1) {
                gr.rows = max(0, min(shared, min(lens[first], a.c.rows))) & ~(TILE - 1);
                gr.blocks = (int)(((unsigned)members * a.g + QT - 1) / QT);
            }
            group[i] = gr;
            tiles += a.c.heads * gr.blocks * tiles_of(gr);
        }
        const int2 at = before(false, tiles);
        total = at.y;
        sum = at.x;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            base[i] = sum;
            sum += a.c.heads * group[i].blocks * tiles_of(group[i]);
        }
        if (FEW && i0 < i1) a.tile_base[i0] = base[i0];
    }
    __syncthreads();
    // the sequences; a thread counts up to 2^20 tiles of own rows, more changes no share
    int own = 0, units = 0;
#pragma unroll 1
    for (int s = tid; s < a.c.seqs; s += PREP_THREADS) {
        const int held = lens[s];
        // the last group that begins at s or before
        int lo = -1, hi = a.groups;
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (group[mid].first <= s) lo = mid;
            else hi = mid;
        }
        const int rows = lo >= 0 && s < group[lo].first + group[lo].members ? group[lo].rows : 0;
        if (rows > held) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        a.skip[s] = LENS ? max(held, rows) : rows;
        if (LENS) continue;
        a.group_of[s] = lo;
        const int left = max(0, min(held, a.c.rows) - rows);
        own = min(1 << 20, own + (int)((unsigned)(left + TILE - 1) / TILE));
        units += left > 0;
    }
    if (LENS) return;
    own = __reduce_add_sync(FULL, own);
    units = __reduce_add_sync(FULL, units);
    if (lane == 0 && own) {
        atomicAdd(&own_tiles, own);
        atomicAdd(&own_units, units);
    }
    __syncthreads();
    if (!FEW || warp == 0) {
        const int grid = ctas_for_shared(a.grid, total, (float)own_tiles * a.c.heads, own_units * a.c.heads);
        // units with CTAs of their own
        const int even = grid ? parts_of(total, grid) : 0;
        int ctas[OWN_EXTRA + 1] = {};
#pragma unroll 1
        for (int i = i0; i < i1 && even; ++i) {
            const int n = min(grid + 1, a.c.heads * group[i].blocks);
#pragma unroll
            for (int x = 0; x <= OWN_EXTRA; ++x)
                ctas[x] = min(grid + 1, ctas[x] + n * min(grid + 1, parts_of(tiles_of(group[i]), even + x)));
        }
#pragma unroll
        for (int x = 0; x <= OWN_EXTRA; ++x) {
            ctas[x] = __reduce_add_sync(FULL, ctas[x]);
            if (!FEW && lane == 0) atomicAdd(&ctas_with[x], ctas[x]);
        }
        if (!FEW) __syncthreads();
        int part = 0;  // tiles of a part, 0: the even deal
#pragma unroll
        for (int x = OWN_EXTRA; x >= 0; --x)
            if (even && (FEW ? ctas[x] : ctas_with[x]) <= grid) part = even + x;
        int mine = 0;
#pragma unroll 1
        for (int i = i0; i < i1 && part; ++i) {
            group[i].parts = parts_of(tiles_of(group[i]), part);
            mine += a.c.heads * group[i].blocks * group[i].parts;
        }
        const int2 cta = before(false, mine);
        sum = cta.x;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            group[i].cta = sum;
            sum += a.c.heads * group[i].blocks * group[i].parts;
            if (FEW) a.group[i] = group[i];
        }
        if (tid == 0) {
            const int used = part ? cta.y : min(grid, total);
            of_deal[0] = part;
            of_deal[1] = used;
            of_deal[2] = total;
            a.tile_base[a.groups] = total;
            *a.own_ctas = max(1, a.grid - used);
            *a.deal = make_int2(part ? used : 0, max(1, used));
        }
    }
    __syncthreads();
    const bool part = of_deal[0];
    const int used = of_deal[1];
    const Deal deal(of_deal[2], max(1, used), 1);
#pragma unroll 1
    for (int c = tid; c < a.grid; c += PREP_THREADS) {
        Share v{};
        if (c < used) {
            if (!part) {
                v.t = deal.begin_cta(c);
                v.t_end = deal.begin_cta(c + 1);
            }
            int lo = 0, hi = a.groups;  // the last group whose CTAs (or tiles) begin at this one or before
#pragma unroll 1
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (part ? group[mid].cta <= c : base[mid] <= v.t) lo = mid;
                else hi = mid;
            }
            const Group gr = group[lo];
            if (part) {
                const int nt = tiles_of(gr), unit = (int)((unsigned)(c - gr.cta) / (unsigned)gr.parts);
                const int p = c - gr.cta - unit * gr.parts;
                // the first nt % parts of the equal parts have a tile more
                const int each = (int)((unsigned)nt / (unsigned)gr.parts), more = nt - each * gr.parts;
                const int h = (int)((unsigned)unit / (unsigned)gr.blocks), k0 = p * each + min(p, more);
                v.t = base[lo] + unit * nt + k0;
                v.t_end = v.t + each + (p < more);
                v.run = Run{gr.first, gr.members, gr.rows, h, unit - h * gr.blocks, k0, v.t_end - v.t};
            } else {
                v.run = run_in(gr, base[lo], v.t, v.t_end);
            }
            v.group = lo;
        }
        a.share[c] = v;
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
// The run that begins at tile t of a share that ends at t_end, for a whole warp.
__device__ __forceinline__ Run run_at(const SharedArgs& a, int t, int t_end, int* from, int lane) {
    const int i = *from = group_of_tile(a, t, *from, lane);
    return run_in(a.group[i], a.tile_base[i], t, t_end);
}
__device__ __forceinline__ int queries_of(const SharedArgs& a, const Run& r) {
    return min(QT, r.members * a.g - r.block * QT);
}
// The block's first query in the order of the parts: group, KV head, member, query head.
__device__ __forceinline__ long long row_of(const SharedArgs& a, const Run& r) {
    return ((long long)r.first * a.c.heads + (long long)r.h * r.members) * a.g + (long long)r.block * QT;
}

// Places of a CTA's j-th K and V in the order in which the products take them:
// K0 K1 V0 K2 V1 ...
__device__ __forceinline__ int k_index(int j) { return j < 1 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_index(int j) { return 2 * j + 2; }

struct __align__(8) Bars {
    uint64_t full[NST], empty[NST];
    uint64_t q_full;
    uint64_t started;                // the first K and the queries are there, and K's producer has seen it
    uint64_t s_full[NSP], p_full[NSP], top_empty[NSP];
    uint64_t top_full[4];            // of a quarter of the queries
    uint64_t t_full, t_empty;
    uint64_t never, drain;
    int asked[NST];    // the last phase of a stage that was asked for
    int rows[NST];     // of a K stage's tile: those whose page is good
    int s_rows[NSP], t_rows;
    uint32_t tmem_base;
    int abort;
};
struct Smem {
    unsigned char q[STAGE];
    unsigned char ring[NST][STAGE];
    float top[NSP][2][QT];  // a tile's largest scores, of either half of its rows
};
constexpr int SMEM_MOST = 232448;  // of a CTA
static_assert(sizeof(Smem) + 1024 <= SMEM_MOST && sizeof(Bars) <= 1024, "the barriers take what aligning leaves");

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars* b, const SharedArgs& a) {
    if (ptx::mbar_wait(bar, parity, a.wait_limit, &b->abort)) return true;
    if (atomicExch(&b->abort, 1) == 0) report(a.c.dev_err, CKV_DEV_TIMEOUT);
    return false;
}

__global__ void __launch_bounds__(THREADS, 1)
    paged_shared_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
    extern __shared__ unsigned char smem_raw[];
    // swizzled tiles need 1024-byte alignment; the barriers stand before them
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023));
    __shared__ Bars bars;
    Bars* bs = &bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            ptx::mbar_init(&bs->full[i], 1);
            ptx::mbar_init(&bs->empty[i], 1);
            bs->asked[i] = -1;
        }
        ptx::mbar_init(&bs->q_full, OUT_WARPS);
        ptx::mbar_init(&bs->started, 1);
        for (int i = 0; i < NSP; ++i) {
            ptx::mbar_init(&bs->s_full[i], 2);  // the product, and the thread that says of how many rows
            ptx::mbar_init(&bs->p_full[i], SOFT_WARPS);
            ptx::mbar_init(&bs->top_empty[i], OUT_WARPS);
        }
        ptx::mbar_init(&bs->t_full, 2);
        ptx::mbar_init(&bs->t_empty, OUT_WARPS);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&bs->top_full[i], 2);
        ptx::mbar_init(&bs->never, 1);
        ptx::mbar_init(&bs->drain, 1);
        bs->abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane < 2) ptx::prefetch_tmap(lane ? &tv : &tk);
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

    const Share share = a.share[blockIdx.x];
    const int t_begin = share.t, t_end = share.t_end, n_tiles = t_end - t_begin;
    bool alive = true;
    int from = share.group;  // the group to look from
    int j = 0;     // tiles so far
    const bool leader = ptx::elect_one();  // the lane that issues the warp's products
    // the scale without its sign, which is in the queries; not 0, so that it
    // leaves -inf what it is
    const float qs = fmaxf(fabsf(a.qscale), 1.17549435e-38f);

    // ---------------------------------------------------------------- producers
    // One of K, one of V: each lane's copy takes its own time to ask for, so that
    // one warp for both was late where pages are short (28 units of 2600 tiles:
    // 61 us with 16 rows a page, now 49; 48 to 49.5 with 128).
    auto produce = [&](auto of_v) {
        constexpr bool values = decltype(of_v)::value;
        const CUtensorMap* map = values ? &tv : &tk;
        const FastDiv& by_page = a.c.by_page;
        Run r = share.run;
        int k = r.k0, k_end = r.k0 + r.n;
        // The first K and the queries before all else: with every stage asked for
        // at once they came with the last of them, 4 us later.  K's producer looks
        // at them, and V's waits for that: without the first V nothing goes on, so
        // neither barrier can be a phase further when it looks (a first run of one
        // tile brings the next queries, and V goes ahead into the first K's stage).
        if (values && n_tiles > 0) alive = __all_sync(FULL, wait(&bs->started, 0, bs, a));
        for (; j < n_tiles && alive; ++j) {
            if (k == k_end) {
                r = run_at(a, t_begin + j, t_end, &from, lane);
                k = r.k0;
                k_end = r.k0 + r.n;
            }
            // lane l looks after the tile's l-th copy: its page (-1: none), slot
            // and place in the stage
            const int row = k * KT + lane * a.box_rows;
            int page = -1, slot = 0;
            if (lane * a.box_rows < KT && row < r.rows) {
                page = a.c.table[(size_t)r.first * a.c.max_pages + by_page.quot(row, &slot)];
                if (page < 0 || page >= a.c.n_pages) {
                    if (!values) report(a.c.dev_err, CKV_DEV_BAD_INDEX);
                    page = -1;
                }
            }
            // rows of bad pages are left out: the others move up
            const unsigned good = __ballot_sync(FULL, page >= 0);
            const int place = __popc(good & ((1u << lane) - 1u)), copies = __popc(good);
            const int rows = copies * a.box_rows - __reduce_max_sync(FULL, page >= 0 ? max(0, row + a.box_rows - r.rows) : 0);
            ++k;
            const int idx = values ? v_index(j) : k_index(j), st = idx % NST;
            alive = idx < NST || __all_sync(FULL, wait(&bs->empty[st], (idx / NST - 1) & 1, bs, a));
            if (!alive) break;
            if (lane == 0) {
                bs->asked[st] = idx / NST;
                bs->rows[st] = rows;
                if (copies) ptx::mbar_arrive_expect_tx(&bs->full[st], copies * a.box_rows * 256);
                else ptx::mbar_arrive(&bs->full[st]);
            }
            __syncwarp();
            if (page >= 0) {
                unsigned char* to = sm.ring[st] + place * a.box_rows * 128;
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
            if (j == 0 && !values) {
                alive = __all_sync(FULL, wait(&bs->full[0], 0, bs, a) && wait(&bs->q_full, 0, bs, a));
                if (alive && lane == 0) ptx::mbar_arrive(&bs->started);
            }
        }
    };
    if (warp == 0) {
        produce(std::integral_constant<bool, false>{});
    } else if (warp == V_WARP) {
        produce(std::integral_constant<bool, true>{});
    } else if (warp == 1) {
        // ------------------------------------------------------------ the products
        // The lanes keep step for the runs; one waits and issues.  S of the tile
        // two on follows T of a tile, into the buffer whose weights that has read.
        const uint32_t ring = ptx::smem_u32(sm.ring);
        const uint64_t q = ptx::smem_desc_sw128(ptx::smem_u32(sm.q));
        constexpr uint32_t ID_S = ptx::idesc_bf16_f32(QT, KT), ID_T = ptx::idesc_bf16_f32(QT, D) | ptx::IDESC_B_MN_MAJOR;
        auto scores = [&](int jj) {
            const int it = k_index(jj), st = it % NST, b = jj % NSP;
            if (!wait(&bs->full[st], (it / NST) & 1, bs, a)) return false;
            ptx::tc_fence_after();
            const int n = bs->rows[st];
            bs->s_rows[b] = n;
            ptx::mbar_arrive(&bs->s_full[b]);
            const uint64_t kd = ptx::smem_desc_sw128(ring + st * STAGE);
            if (n > 0)
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t at = ((ks >> 2) * PANEL + (ks & 3) * 32) >> 4;
                    ptx::mma_bf16(tmem + b * SP_COLS, q + at, kd + at, ID_S, ks > 0);
                }
            ptx::mma_commit(&bs->s_full[b]);
            return true;
        };
        auto values = [&](int jj) {
            const int it = v_index(jj), st = it % NST, b = jj % NSP;
            if (!wait(&bs->full[st], (it / NST) & 1, bs, a) || !wait(&bs->p_full[b], (jj / NSP) & 1, bs, a) ||
                (jj > 0 && !wait(&bs->t_empty, (jj - 1) & 1, bs, a)))
                return false;
            const int n = bs->s_rows[b], steps = n / 16;
            const uint32_t p = tmem + b * SP_COLS;
            const uint64_t v = ptx::smem_desc_sw128_mn(ring + st * STAGE, PANEL);
            ptx::tc_fence_after();
            bs->t_rows = n;
            ptx::mbar_arrive(&bs->t_full);
            // the low terms first; eight columns hold a term of 16 rows.
            // (Straight code for all 24 products takes 5 us at its first pass,
            // when it has to be fetched.)
#pragma unroll 1
            for (int term = 0; term < 3; ++term) {
                uint32_t at = p + (term == 1 ? MID_COL : term ? 0 : LOW_COL);
                const uint32_t pairs = term == 1 ? 16 : 32;  // columns from two steps' terms to the next two's
#pragma unroll
                for (int ks = 0; ks < 8; ks += 2) {
                    if (ks < steps)
                        ptx::mma_bf16_ts(tmem + T_COL, at, v + (ks * 2048 >> 4), ID_T, term > 0 || ks > 0);
                    if (ks + 1 < steps)
                        ptx::mma_bf16_ts(tmem + T_COL, at + 8, v + ((ks + 1) * 2048 >> 4), ID_T, 1);
                    at += pairs;
                }
            }
            ptx::mma_commit(&bs->t_full);
            return true;
        };
        int runs = 0;
        Run r = share.run;
        for (int t = t_begin; t < t_end && alive; ++runs) {
            if (runs > 0) r = run_at(a, t, t_end, &from, lane);
            if (leader) {
                if (runs == 0 && a.stall && !wait(&bs->never, 0, bs, a)) alive = false;
                if (alive) alive = wait(&bs->q_full, runs & 1, bs, a);
#pragma unroll 1
                for (int jj = j - 2; jj < j + r.n && alive; ++jj) {
                    if (jj >= j) alive = values(jj);
                    if (alive && jj + 2 < j + r.n) alive = scores(jj + 2);
                }
            }
            alive = __all_sync(FULL, alive);
            j += r.n;
            t += r.n;
        }
    } else if (warp < 2 + SOFT_WARPS) {
        // ------------------------------------------------------------ softmax
        const int half = (warp - 2) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint64_t qs2 = pair(qs, qs), minus2 = pair(-1.f, -1.f);
        int exchanges = 0;
        Run r = share.run;
        for (int t = t_begin; t < t_end && alive;) {
            if (t > t_begin) r = run_at(a, t, t_end, &from, lane);
            const bool busy = quarter * 32 < queries_of(a, r);  // some of the warp's queries exist
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < r.n; ++k) {
                const int b = (j + k) % NSP, use = (j + k) / NSP;
                const uint32_t sp = tmem + ((uint32_t)(quarter * 32) << 16) + b * SP_COLS;
                alive = __all_sync(FULL, wait(&bs->s_full[b], use & 1, bs, a) &&
                                             (use == 0 || wait(&bs->top_empty[b], (use - 1) & 1, bs, a)));
                if (!alive) break;
                if (warp == 2 && lane == 0) ptx::mbar_arrive(&bs->empty[k_index(j + k) % NST]);
                const int n = bs->s_rows[b], mine = n - 64 * half;  // rows of this half of the tile
                if (busy && n > 0) {
                    ptx::tc_fence_after();
                    // 16 rows at a time, of which there are `mine` / 16 at most four
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    {
                        uint32_t s[2][32];
                        ptx::tmem_ld32(sp + half * 64, s[0]);
                        ptx::tmem_ld32(sp + half * 64 + 32, s[1]);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (16 * c < mine)
#pragma unroll
                                for (int e = 16 * (c & 1); e < 16 * (c & 1) + 16; e += 2)
                                    top[(e >> 1) & 3] = fmaxf(fmaxf(top[(e >> 1) & 3], __uint_as_float(s[c >> 1][e])),
                                                              __uint_as_float(s[c >> 1][e + 1]));
                    }
                    const float own = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // the other half's, so that all of a query's weights go by one maximum
                    sm.top[b][half][row] = own;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bs->top_full[quarter]);
                    alive = __all_sync(FULL, wait(&bs->top_full[quarter], exchanges & 1, bs, a));
                    if (!alive) break;
                    ++exchanges;
                    const float grown = fmaxf(m, fmaxf(own, sm.top[b][1 - half][row]) * qs);
                    const float ms = grown == -INFINITY ? 0.f : grown;
                    l *= ex2(m - ms);
                    m = grown;
                    const uint64_t ms2 = pair(-ms, -ms);
                    uint64_t sum[2] = {0, 0};
#pragma unroll 1
                    for (int c = 0; c < 64 && c < mine; c += 32) {
                        uint32_t s[32], hi[16], mid[16], lo[16];
                        ptx::tmem_ld32(sp + half * 64 + c, s);
                        ptx::tmem_ld_wait();
                        if (c + 16 >= mine)  // 16 rows: the others weigh nothing
#pragma unroll
                            for (int e = 16; e < 32; ++e) s[e] = 0xff800000u;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 x = unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), qs2, ms2));
                            s[e] = __float_as_uint(ex2(x.x));
                            s[e + 1] = __float_as_uint(ex2(x.y));
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float p0 = __uint_as_float(s[e]), p1 = __uint_as_float(s[e + 1]);
                            const uint64_t p = pair(p0, p1);
                            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], p);
                            // a float's upper 16 bits are a bf16, and what they leave is exact
                            hi[e / 2] = __byte_perm(s[e], s[e + 1], 0x7632);
                            const uint64_t rest = fma2(floats(hi[e / 2]), minus2, p);
                            const float2 y = unpair(rest);
                            mid[e / 2] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
                            const float2 z = unpair(fma2(floats(mid[e / 2]), minus2, rest));
                            lo[e / 2] = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
                        }
                        // over the scores just read
                        ptx::tmem_st16(sp + half * 64 + c, hi);
                        ptx::tmem_st16(sp + half * 64 + c + LOW_COL, lo);
                        ptx::tmem_st16(sp + MID_COL + half * 32 + c / 2, mid);
                    }
                    ptx::tmem_st_wait();
                    const float2 x = unpair(add2(sum[0], sum[1]));
                    l += x.x + x.y;
                    ptx::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bs->p_full[b]);
            }
            if (alive && row < queries_of(a, r))
                reinterpret_cast<float2*>(r.k0 == 0 ? a.unit_ml + row_of(a, r) + row
                                                    : a.cta_ml + (size_t)blockIdx.x * QT + row)[half] = make_float2(m, l);
            j += r.n;
            t += r.n;
        }
    } else {
        // ------------------------------------------------------------ queries, O
        const int half = (warp - 2 - SOFT_WARPS) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, tid = threadIdx.x - 32 * (2 + SOFT_WARPS);
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + T_COL + half * 64;
        const uint32_t sign = a.qscale < 0.f ? 0x80008000u : 0u;
        auto both = [](const uint32_t (&v)[16], int e) { return pair(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])); };
        // the run's queries to shared memory, swizzled as TMA does
        auto queries = [&](const Run& r) {
            constexpr int N = QT * 16 / (32 * OUT_WARPS);  // pieces of 16 bytes that a thread brings
            const int piece = tid & 15, all = queries_of(a, r);
            const unsigned char* from = a.q + r.first * a.qst[0] + (long long)r.h * a.g * a.qst[1] + piece * 16;
            uint4 v[N];
            // all of them under way at once: a row behind the last is the last one again
#pragma unroll
            for (int i = 0; i < N; ++i) {
                int head;
                const int member = a.by_g.quot(r.block * QT + min((tid >> 4) + i * 2 * OUT_WARPS, all - 1), &head);
                v[i] = *reinterpret_cast<const uint4*>(from + member * a.qst[0] + head * a.qst[1]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int y = (tid >> 4) + i * 2 * OUT_WARPS;
                v[i].x ^= sign, v[i].y ^= sign, v[i].z ^= sign, v[i].w ^= sign;
                *reinterpret_cast<uint4*>(sm.q + (piece >> 3) * PANEL + y * 128 + (((piece & 7) ^ (y & 7)) << 4)) = v[i];
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bs->q_full);
        };
        Run r = share.run;
        if (t_begin < t_end) queries(r);
        for (int t = t_begin; t < t_end && alive;) {
            const bool busy = quarter * 32 < queries_of(a, r);
            uint64_t o[32];
            float m = -INFINITY;
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0;
            for (int k = 0; k < r.n; ++k) {
                const int jj = j + k;
                // the softmax's running maximum, made the same way, while T is made:
                // the next T waits for this one to be read
                const int b = jj % NSP;
                if (!__all_sync(FULL, wait(&bs->p_full[b], (jj / NSP) & 1, bs, a))) {
                    alive = false;
                    break;
                }
                const float grown = fmaxf(m, fmaxf(sm.top[b][0][row], sm.top[b][1][row]) * qs);
                const float x = ex2(m - (grown == -INFINITY ? 0.f : grown));
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bs->top_empty[b]);
                if (!__all_sync(FULL, wait(&bs->t_full, jj & 1, bs, a))) {
                    alive = false;
                    break;
                }
                if (busy && bs->t_rows > 0) {
                    ptx::tc_fence_after();
                    m = grown;
                    const uint64_t x2 = pair(x, x);
                    // two loads under way at a time
                    uint32_t v[2][16];
                    ptx::tmem_ld16(at, v[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        ptx::tmem_ld_wait();
                        if (c < 3) {
                            ptx::tmem_ld16(at + 16 * (c + 1), v[(c + 1) & 1]);
                        } else {
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&bs->t_empty);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[8 * c + e] = fma2(o[8 * c + e], x2, both(v[c & 1], e));
                    }
                } else {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bs->t_empty);
                }
                if (lane == 0 && warp == 1 + SOFT_WARPS + OUT_WARPS) ptx::mbar_arrive(&bs->empty[v_index(jj) % NST]);
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
            if (row < queries_of(a, done)) {
                const int stride = done.k0 == 0 ? queries_of(a, done) : QT;
                float4* to = (done.k0 == 0 ? a.unit_o + row_of(a, done) * (D / 4) : a.cta_o + (size_t)blockIdx.x * QT * (D / 4)) +
                             half * 16 * stride + row;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 u = unpair(o[2 * c]), v = unpair(o[2 * c + 1]);
                    to[c * stride] = make_float4(u.x, u.y, v.x, v.y);
                }
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
// The parts of the units, and what the sequences' own rows gave: results, or
// parts of up to JOINED_PARTS CTAs (merged here and not by the last of these: 18.1
// to 15.9 us for 8 sequences behind 512 rows, 83 to 82 for 160 behind 16k).  A
// block has four rows of the output, a thread four channels of one, so that the g
// heads of a part come side by side.  Its time is the latency of its loads and of
// its instructions, which come from L2: PARTS parts are under way at a time (one
// after the other 20 parts took 12 us; eight at a time 1 to 2 us more than six).
constexpr int PARTS = 6;
__global__ void __launch_bounds__(JOIN_THREADS) paged_shared_join(const __grid_constant__ SharedArgs a) {
    const int channel = threadIdx.x / JOIN_ROWS, heads_q = a.c.heads * a.g;  // four channels
    const long long n = (long long)a.c.seqs * heads_q, step = (long long)gridDim.x * JOIN_ROWS;
    bool waited = false;
    ptx::allow_dependent_launch();
    // What the prep has left is whole: the kernel before this one began after it.
    // It is looked up while that one is still at work, behind a fence, as no wait of
    // this kernel's own has made it visible yet.
    ptx::fence_acquire();
#pragma unroll 1
    for (long long row = (long long)blockIdx.x * JOIN_ROWS + threadIdx.x % JOIN_ROWS; row < n; row += step) {
        const int s = (int)(row / heads_q), hq = (int)(row - (long long)s * heads_q);
        const int i = a.group_of[s], skip = a.skip[s], held = a.c.lens[s], total = a.tile_base[a.groups];
        const int2 dealt = *a.deal;
        float4* out = reinterpret_cast<float4*>(a.out + row * D) + channel;
        int head, c0 = 0, parts = 0;
        const int h = a.by_g.quot(hq, &head);
        const float4 *unit_o = a.unit_o, *unit_ml = a.unit_ml, *cta_o = a.cta_o, *cta_ml = a.cta_ml;
        if (skip > 0) {
            const Group gr = a.group[i];
            const int x = (s - gr.first) * a.g + head;
            const int block = x / QT, y = x - block * QT, unit = h * gr.blocks + block;
            c0 = gr.cta + unit * gr.parts;
            parts = gr.parts;
            if (dealt.x == 0) {
                const Deal deal(total, Deal::ctas(total, 1, dealt.y), 1);
                const int nt = tiles_of(gr), t0 = a.tile_base[i] + unit * nt;
                c0 = deal.cta_of(t0);
                parts = deal.cta_of(t0 + nt - 1) - c0 + 1;
            }
            const Run r{gr.first, gr.members, gr.rows, h, block, 0, 0};
            unit_ml += row_of(a, r) + y;
            unit_o += row_of(a, r) * (D / 4) + channel * queries_of(a, r) + y;
            cta_ml += (size_t)c0 * QT + y;
            cta_o += ((size_t)c0 * (D / 4) + channel) * QT + y;
        }
        const bool own = min(held, a.c.rows) > skip;  // it has rows of its own
        const int32_t* own_left = a.own_left + (size_t)s * a.c.heads + h;
        if (!waited) ptx::grid_dependency_wait();
        waited = true;
        const int left = own ? *own_left : 0, own_parts = left >> 16;
        if (skip == 0 && own && own_parts == 0) continue;  // in no group, and whole
        const float own_m = own ? a.own_lse2[row] : -INFINITY;
        const float4 own_o = own ? *out : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int p0 = 0; p0 < parts; p0 += PARTS) {
            float4 o[PARTS], ml[PARTS];
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                ml[k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                if (p0 + k < parts) {
                    const bool first = k == 0 && p0 == 0;
                    ml[k] = first ? *unit_ml : cta_ml[k * QT];
                    o[k] = first ? *unit_o : cta_o[k * (D / 4) * QT];
                }
            }
            cta_ml += PARTS * QT;
            cta_o += PARTS * (D / 4) * QT;
            float grown = m;  // (either half of a part's rows has the same maximum)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) grown = fmaxf(grown, ml[k].x);
            const float ms = grown == -INFINITY ? 0.f : grown;  // (all products NaN: the sum says so)
            const float u = ex2(m - ms);
            m = grown;
            l *= u;
            acc = make_float4(acc.x * u, acc.y * u, acc.z * u, acc.w * u);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const float v = ex2(ml[k].x - ms);
                l += (ml[k].y + ml[k].w) * v;
                acc.x += o[k].x * v;
                acc.y += o[k].y * v;
                acc.z += o[k].z * v;
                acc.w += o[k].w * v;
            }
        }
        constexpr int AT_A_TIME = 4;
#pragma unroll 1
        for (int p0 = 0; own && p0 < max(1, own_parts); p0 += AT_A_TIME) {
            float4 o[AT_A_TIME];
            float pm[AT_A_TIME], pl[AT_A_TIME];
#pragma unroll
            for (int k = 0; k < AT_A_TIME; ++k) {
                const bool whole = k == 0 && own_parts == 0;
                o[k] = whole ? own_o : make_float4(0.f, 0.f, 0.f, 0.f);
                pm[k] = whole ? own_m : -INFINITY;
                pl[k] = whole ? 1.f : 0.f;
                if (p0 + k < own_parts) {
                    const float* p = a.own_part + (size_t)(2 * ((left & 0xffff) + p0 + k) + (p0 + k == 0)) * part_floats(a.g);
                    o[k] = *reinterpret_cast<const float4*>(p + head * D + 4 * channel);
                    pm[k] = p[a.g * D + head];
                    pl[k] = p[a.g * D + a.g + head];
                }
            }
            float grown = m;
#pragma unroll
            for (int k = 0; k < AT_A_TIME; ++k) grown = fmaxf(grown, pm[k]);
            const float ms = grown == -INFINITY ? 0.f : grown;  // (all products NaN: the sum says so)
            const float u = ex2(m - ms);
            m = grown;
            l *= u;
            acc = make_float4(acc.x * u, acc.y * u, acc.z * u, acc.w * u);
#pragma unroll
            for (int k = 0; k < AT_A_TIME; ++k) {
                const float v = ex2(pm[k] - ms);
                l += pl[k] * v;
                acc.x += o[k].x * v;
                acc.y += o[k].y * v;
                acc.z += o[k].z * v;
                acc.w += o[k].w * v;
            }
        }
        const float w = l == 0.f ? 0.f : 1.f / l;
        *out = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
        if (a.lse && channel == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
    // the kernel behind waits for this one, and this one for all before it
    if (!waited) ptx::grid_dependency_wait();
}

// ---------------------------------------------------------------- host side
struct Layout {
    size_t attn, group, tile_base, skip, group_of, share, deal, own_ctas, own_left, unit_o, unit_ml, cta_o, cta_ml, total;
};
Layout layout_of(const Cache& c, int g) {
    Layout l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t S = c.seqs, queries = S * c.heads * g;
    l.attn = 0;
    l.group = up(attn_workspace(c, g, nullptr, nullptr, nullptr));
    l.tile_base = l.group + up(S * sizeof(Group));
    l.skip = l.tile_base + up((S + 1) * sizeof(int));
    l.group_of = l.skip + up(S * sizeof(int));
    l.share = l.group_of + up(S * sizeof(int));
    l.deal = l.share + up(MAX_GRID * sizeof(Share));
    l.own_ctas = l.deal + up(sizeof(int2));
    l.own_left = l.own_ctas + up(sizeof(int));
    l.unit_o = l.own_left + up(S * c.heads * sizeof(int32_t));
    l.unit_ml = l.unit_o + up(queries * D * sizeof(float));
    l.cta_o = l.unit_ml + up(queries * sizeof(float4));
    l.cta_ml = l.cta_o + (size_t)MAX_GRID * QT * D * sizeof(float);
    l.total = l.cta_ml + (size_t)MAX_GRID * QT * sizeof(float4);
    return l;
}

bool few(const SharedArgs& a) { return a.groups <= FEW_GROUPS && a.c.seqs <= FEW_SEQS; }

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
    // all of an SM's but what the barriers take: aligned behind them the rest is there
    constexpr size_t smem = SMEM_MOST - (sizeof(Bars) + 15) / 16 * 16;
    static_assert((sizeof(Bars) + 15) / 16 * 16 + smem >= 1024 + sizeof(Smem), "tiles behind the barriers");
    static std::atomic<bool> set[MAX_DEVICES];
    if (!set[dev].load(std::memory_order_relaxed)) {
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, paged_shared_kernel);
        if (e == cudaSuccess && at.sharedSizeBytes > (sizeof(Bars) + 15) / 16 * 16) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(paged_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    cudaError_t e = launch_dependent(few(a) ? paged_shared_prep<true, false> : paged_shared_prep<false, false>, dim3(1),
                                     dim3(PREP_THREADS), 0, s, a);
    if (e == cudaSuccess) e = launch_dependent(paged_shared_kernel, dim3(a.grid), dim3(THREADS), smem, s, a, tk, tv);
    const long long qst[2] = {a.qst[0] / 2, a.qst[1] / 2};
    if (e == cudaSuccess)
        e = launch_attn_own_rows(a.c, a.skip, a.own_ctas, a.own_left, a.q, qst, a.g, a.qscale, a.out, a.lse, workspace, s);
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
    if (groups == 0)
        return ckv_paged_decode_attn(cache, q, q_dtype, q_stride, g, scale, out, lse, nullptr, nullptr, workspace,
                                     workspace_bytes, stream);
    if (!q || !q_stride || !out) return CKV_ERR_ARG;
    if (q_dtype != cache->kv_dtype) return CKV_ERR_DTYPE;
    a.qscale = scale * LOG2E;
    if (!isfinite(a.qscale)) return CKV_ERR_ARG;
    const bool bf16 = cache->kv_dtype == CKV_BF16;
    const long long extent[2] = {a.c.seqs, (long long)a.c.heads * g};
    for (int i = 0; i < 2; ++i) {
        if (q_stride[i] < 0 || q_stride[i] > MAX_STRIDE) return CKV_ERR_ARG;
        a.qst[i] = extent[i] > 1 ? q_stride[i] * (bf16 ? 2 : 4) : 0;
        if (a.qst[i] & 15) return CKV_ERR_ALIGN;
    }
    // tiles, of the own rows too, are counted in 32 bits
    if (extent[0] * a.c.heads * ceil_div(a.c.rows, 8) > 0x7fff0000LL) return CKV_ERR_ARG;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return CKV_ERR_ALIGN;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    a.q = static_cast<const unsigned char*>(q);
    a.g = g;
    a.by_g = FastDiv((uint32_t)g);
    a.group_starts = group_starts;
    a.prefix = prefix;
    a.groups = groups;
    a.out = out;
    a.lse = lse;
    a.group = reinterpret_cast<Group*>(w + l.group);
    a.tile_base = reinterpret_cast<int*>(w + l.tile_base);
    a.skip = reinterpret_cast<int32_t*>(w + l.skip);
    a.group_of = reinterpret_cast<int*>(w + l.group_of);
    float* own_part;
    attn_workspace(a.c, g, &a.own_lse2, &own_part, workspace);
    a.own_part = own_part;
    a.own_left = reinterpret_cast<int32_t*>(w + l.own_left);
    a.share = reinterpret_cast<Share*>(w + l.share);
    a.deal = reinterpret_cast<int2*>(w + l.deal);
    a.own_ctas = reinterpret_cast<int*>(w + l.own_ctas);
    a.unit_o = reinterpret_cast<float4*>(w + l.unit_o);
    a.unit_ml = reinterpret_cast<float4*>(w + l.unit_ml);
    a.cta_o = reinterpret_cast<float4*>(w + l.cta_o);
    a.cta_ml = reinterpret_cast<float4*>(w + l.cta_ml);
    if (!bf16) {
        cudaStream_t s = (cudaStream_t)stream;
        if (few(a)) {
            const Groups of{group_starts, prefix, groups};
            const long long qst[2] = {a.qst[0] / 4, a.qst[1] / 4};
            return launch_attn_in_groups(a.c, of, q, qst, g, a.qscale, out, lse, workspace, s) == cudaSuccess ? CKV_OK
                                                                                                             : CKV_ERR_CUDA;
        }
        if (launch_dependent(paged_shared_prep<false, true>, dim3(1), dim3(PREP_THREADS), 0, s, a) != cudaSuccess)
            return CKV_ERR_CUDA;
        ckv_paged_cache attended = *cache;
        attended.lens = a.skip;
        return ckv_paged_decode_attn(&attended, q, q_dtype, q_stride, g, scale, out, lse, nullptr, nullptr, workspace,
                                     workspace_bytes, stream);
    }
    waits(&a.wait_limit, &a.stall);
    const cudaError_t e = launch_shared(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
