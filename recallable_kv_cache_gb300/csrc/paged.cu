// Paged cache: appending rows and evicting rows by accumulated attention
// weight (the attention over the pages is in paged_attn.cu).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "paged.h"
#include "ptx.cuh"

namespace ckv {
namespace paged {

int sm_count(int* dev_out) {
    static std::atomic<int> sms[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return 0;
    if (dev_out) *dev_out = dev;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

namespace {

// byte strides of a [..][extent[i]].. operand; false if one is too small
bool strides_ok(const int64_t* st, const int32_t* extent, int n, int elem, long long* out) {
    for (int i = 0; i < n; ++i) {
        long long b = (long long)st[i];
        if (extent[i] > 1 && (b < D || b > MAX_STRIDE)) return false;
        if (extent[i] <= 1) b = D;  // never multiplied by more than 0
        out[i] = b * elem;
    }
    return true;
}
bool strides_aligned(const long long* b, int n) {
    for (int i = 0; i < n; ++i)
        if (b[i] & 15) return false;
    return true;
}

}  // namespace

ckv_status check_cache(const ckv_paged_cache* c, Cache* o) {
    if (!c || !c->K || !c->V || !c->table || !c->lens) return CKV_ERR_ARG;
    if (c->kv_dtype != CKV_F32 && c->kv_dtype != CKV_BF16) return CKV_ERR_DTYPE;
    if (c->d != D || c->n_pages < 1 || c->heads < 1 || c->seqs < 1 || c->max_pages < 1 || c->page_size < TILE ||
        c->page_size % TILE)
        return CKV_ERR_ARG;
    const long long rows = (long long)c->max_pages * c->page_size;
    if (rows > 0x7fffffffLL - TILE || (long long)c->seqs * c->heads > 0x7fffffffLL) return CKV_ERR_ARG;
    const int elem = c->kv_dtype == CKV_BF16 ? 2 : 4;
    const int32_t extent[3] = {c->n_pages, c->heads, c->page_size};
    if (!strides_ok(c->k_stride, extent, 3, elem, o->ks) || !strides_ok(c->v_stride, extent, 3, elem, o->vs))
        return CKV_ERR_ARG;
    if (!aligned16(c->K) || !aligned16(c->V) || !aligned16(c->mass) || !aligned16(c->pos) ||
        !strides_aligned(o->ks, 3) || !strides_aligned(o->vs, 3))
        return CKV_ERR_ALIGN;
    if (c->pos && !c->seen) return CKV_ERR_ARG;
    o->K = static_cast<unsigned char*>(c->K);
    o->V = static_cast<unsigned char*>(c->V);
    o->table = c->table;
    o->lens = c->lens;
    o->mass = c->mass;
    o->pos = c->pos;
    o->seen = c->seen;
    o->dev_err = c->dev_err;
    o->n_pages = c->n_pages;
    o->heads = c->heads;
    o->page = c->page_size;
    o->seqs = c->seqs;
    o->max_pages = c->max_pages;
    o->rows = (int)rows;
    o->by_page = FastDiv((uint32_t)c->page_size);
    o->by_heads = FastDiv((uint32_t)c->heads);
    return CKV_OK;
}

namespace {

constexpr unsigned FULL = 0xffffffffu;

// ---------------------------------------------------------------- append
constexpr int APPEND_THREADS = 256;
constexpr int IN_FLIGHT = 4;  // rows whose K and V pieces a thread has in flight

struct AppendArgs {
    Cache c;
    const unsigned char* k_src;
    const unsigned char* v_src;
    long long kst[3], vst[3];  // byte strides: sequence, head, row
    const int32_t* counts;
    const int32_t* start;
    const int32_t* first;
    int n;
    FastDiv by_blocks;  // blocks per sequence
    int advance;  // this kernel writes lens and seen
};

// r0, p0 and the row count of sequence s; count -1 if it must be left alone
__device__ __forceinline__ int append_plan(const AppendArgs& a, int s, int* r0, int* p0) {
    *r0 = a.start ? a.start[s] : a.c.lens[s];
    *p0 = a.first ? a.first[s] : (a.c.seen ? a.c.seen[s] : 0);
    const int cnt = a.counts ? a.counts[s] : a.n;
    if (*r0 < 0 || cnt < 0 || cnt > a.n || (long long)*r0 + cnt > a.c.rows) return -1;
    if (a.c.seen && (*p0 < 0 || (long long)*p0 + cnt > 0x7fffffffLL)) return -1;
    return cnt;
}
__device__ __forceinline__ void append_advance(const AppendArgs& a, int s, int r0, int p0, int cnt) {
    if (cnt < 0) {
        report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        return;
    }
    a.c.lens[s] = r0 + cnt;
    if (a.c.seen) a.c.seen[s] = p0 + cnt;
}

// A copy of 16-byte pieces, VPR of them per row of 128 channels; consecutive
// threads take consecutive pieces of a row, then the KV heads of a token.  One
// token's rows of 256 units are a matter of latency (2 us); long prompts of
// bandwidth, for which every thread has the pieces of IN_FLIGHT rows under way.
template <int VPR>
__global__ void __launch_bounds__(APPEND_THREADS) paged_append_kernel(const __grid_constant__ AppendArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    constexpr int ROWS = APPEND_THREADS / VPR;
    int b;
    const int s = a.by_blocks.quot(blockIdx.x, &b);
    int r0, p0;
    const int cnt = append_plan(a, s, &r0, &p0);
    const int piece = threadIdx.x % VPR;
    const int items = cnt < 0 ? 0 : cnt * a.c.heads;  // rows of all KV heads, the heads of a token side by side
    const unsigned char* ksrc = a.k_src + s * a.kst[0] + piece * 16;
    const unsigned char* vsrc = a.v_src + s * a.vst[0] + piece * 16;
    unsigned char* K = a.c.K + piece * 16;
    unsigned char* V = a.c.V + piece * 16;
    for (int i0 = b * ROWS * IN_FLIGHT + threadIdx.x / VPR; i0 < items; i0 += a.by_blocks.d * ROWS * IN_FLIGHT) {
        uint4 kv[IN_FLIGHT], vv[IN_FLIGHT];
        int j[IN_FLIGHT], h[IN_FLIGHT], pg[IN_FLIGHT], slot[IN_FLIGHT];
#pragma unroll
        for (int x = 0; x < IN_FLIGHT; ++x) {
            const int i = i0 + x * ROWS;
            pg[x] = -1;
            if (i < items) {
                j[x] = a.c.by_heads.quot(i, &h[x]);
                kv[x] = *reinterpret_cast<const uint4*>(ksrc + h[x] * a.kst[1] + j[x] * a.kst[2]);
                vv[x] = *reinterpret_cast<const uint4*>(vsrc + h[x] * a.vst[1] + j[x] * a.vst[2]);
                pg[x] = page_of(a.c, s, r0 + j[x], &slot[x]);
            }
        }
#pragma unroll
        for (int x = 0; x < IN_FLIGHT; ++x) {
            if (pg[x] < 0) continue;
            *reinterpret_cast<uint4*>(K + pg[x] * a.c.ks[0] + h[x] * a.c.ks[1] + slot[x] * a.c.ks[2]) = kv[x];
            *reinterpret_cast<uint4*>(V + pg[x] * a.c.vs[0] + h[x] * a.c.vs[1] + slot[x] * a.c.vs[2]) = vv[x];
            if (piece == 0) {
                const size_t o = ((size_t)s * a.c.heads + h[x]) * a.c.rows + r0 + j[x];
                if (a.c.pos) a.c.pos[o] = p0 + j[x];
                if (a.c.mass) a.c.mass[o] = 0.f;
            }
        }
    }
    if (a.advance) {
        // the plan was read by every thread of the sequence's only block
        // (advance in place), or from arrays that nothing here writes
        __syncthreads();
        if (b == 0 && threadIdx.x == 0) append_advance(a, s, r0, p0, cnt);
    }
}

__global__ void __launch_bounds__(128) paged_advance_kernel(const __grid_constant__ AppendArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int s = blockIdx.x * 128 + threadIdx.x;
    if (s >= a.c.seqs) return;
    int r0, p0;
    const int cnt = append_plan(a, s, &r0, &p0);
    append_advance(a, s, r0, p0, cnt);
}

// ---------------------------------------------------------------- eviction: selection
constexpr int SEL_LONG = 4096;        // rows of a CTA from which it has 1024 threads, below 512
constexpr int SEL_BINS = 4096;        // 12 bits of the key a pass: 12, 12 and 8
constexpr int SEL_LIST = 1024;        // keys of one bin that are listed
constexpr int SEL_CAND = 256;         // keys of one bin that are ranked directly
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_MAX_SLICE = 40960;  // keys of one CTA that stay in shared memory (160 KB)

struct SelectArgs {
    Cache c;
    int budget, sinks, recent, max_moves;
    int32_t* moves;
    int32_t* n_moves;
};

// Rank of a row as an unsigned key, larger = kept first: protected rows are
// the largest value, the others the mass in the order of the reals (NaN
// lowest; a float's bits compare like an integer after flipping the sign bit
// of non-negative and all bits of negative values; adding +0 turns -0 into +0).
__device__ __forceinline__ uint32_t evict_key(float mass, int pos, int sinks, int recent_from) {
    if (pos < sinks || pos >= recent_from) return 0xffffffffu;
    if (mass != mass) return 0u;
    const uint32_t b = __float_as_uint(mass + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// adds v to the word at p (an address of this CTA's shared memory) in the CTA of that rank
__device__ __forceinline__ void peer_add(int* p, uint32_t rank, int v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
// word at p (an address of this CTA's shared memory) in the CTA of that rank
__device__ __forceinline__ int peer_word(const int* p, uint32_t rank) {
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// A cluster of CS CTAs per (sequence, KV head), each with a slice of its rows.
// One pass over mass and pos turns them into keys, kept in shared memory
// (CACHED; longer caches read them again: 32 units of 327001 rows 66 us, of
// 400001 137 us), and counts the keys' top 12 bits;
// the key of the budget-th row follows digit by digit from the histograms, to
// which every CTA adds its occupied bins in all its peers' shared memory (few
// are occupied; every CTA reading all bins of its peers took 97 us for 32
// units of 128k rows where this takes 20 us).  Where a digit leaves at most
// SEL_LIST keys (a first digit's bin is an eighth of a power of two) they are
// listed, and later digits look at the list alone; where it leaves at most
// SEL_CAND, the CTAs exchange them and the key T of the wanted rank is found by
// counting, with no further digit and no further exchange.
// A row is kept if its key is above T, or equal and among the first that fit.
// With gt(r), eq(r) the rows before r above and equal, kept(r) = gt(r) +
// min(eq(r), fitting) rows are kept before r, so the k-th hole is the row r <
// budget, not kept, with r - kept(r) = k and the k-th mover the kept row r >=
// budget with kept(r) - kept(budget) = k.  The pass that lists (or else the one
// that counts) leaves a bit for every row that may be kept, and the writing pass
// looks at those rows and at the ones below the budget only.
template <int CS, int THREADS, bool CACHED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) paged_select_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int WARPS = THREADS / 32;
    constexpr int WORDS = THREADS == 1024 ? SEL_MAX_SLICE / 1024 : SEL_LONG / 512 + 4;  // bits of a warp's rows
    extern __shared__ __align__(16) int sel_smem[];
    // two histograms of the unit (the third pass takes the first again), one of this CTA's rows, the keys
    int* mine = sel_smem + 2 * SEL_BINS;
    uint32_t* keys = reinterpret_cast<uint32_t*>(sel_smem + (CS > 1 ? 3 : 2) * SEL_BINS);
    __shared__ int warp_sum[WARPS];
    __shared__ int4 counts[WARPS];  // a warp's rows above, equal; those of them below the budget
    __shared__ int4 totals;         // the CTA's (not ranked)
    __shared__ int found[3];
    __shared__ uint32_t list[SEL_LIST];  // of this CTA's rows, and where they are in the slice
    __shared__ int list_at[SEL_LIST];
    __shared__ __align__(16) uint32_t cand[SEL_CAND];  // of the unit
    __shared__ uint32_t own_cand[SEL_CAND];            // of this CTA's rows
    __shared__ int cand_low[SEL_CAND], own_low[SEL_CAND];    // whether the row is below the budget
    __shared__ int own_n[4];                         // keys listed, exchanged; rows above them, of those below the budget
    __shared__ int before_cta[4], unit_low[2];       // rows above and equal in the CTAs before; below the budget
    __shared__ uint32_t maybe[WARPS][CACHED ? WORDS + 2 : 1];  // read up to two words past a warp's rows
    const int u = blockIdx.x / CS, s = a.c.by_heads.quot(u);
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto sync_all = [] {
        if (CS > 1) cluster_sync();
        else __syncthreads();
    };
    for (int i = tid; i < (CS > 1 ? 3 : 2) * SEL_BINS / 4; i += THREADS)
        reinterpret_cast<int4*>(sel_smem)[i] = make_int4(0, 0, 0, 0);
    if (tid < 4) own_n[tid] = before_cta[tid] = 0;
    if (tid < 2) unit_low[tid] = 0;
    if (CACHED)
        for (int i = tid; i < WARPS * (WORDS + 2); i += THREADS) (&maybe[0][0])[i] = 0;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    if (tid == 0 && rank == 0) check_len(a.c, s);
    const int len = rows_held(a.c, s);
    if (len <= a.budget) {  // for every CTA of the cluster
        if (tid == 0 && rank == 0) a.n_moves[u] = 0;
        return;
    }
    const int slice = ((len + CS - 1) / CS + 127) / 128 * 128;
    const int r0 = min(len, rank * slice), n = min(slice, len - r0);  // r0 + slice may pass 2^31
    const float* mass = a.c.mass + (size_t)u * a.c.rows + r0;
    const int32_t* pos = a.c.pos + (size_t)u * a.c.rows + r0;
    const int recent_from = a.c.seen[s] - a.recent;
    int* local = CS > 1 ? mine : sel_smem;
    auto key_at = [&](int i) { return CACHED ? keys[i] : evict_key(mass[i], pos[i], a.sinks, recent_from); };
    sync_all();  // every CTA's histograms are cleared
    // rows are a multiple of 16 per (sequence, KV head): reading up to three
    // past n stays inside
#pragma unroll 2
    for (int i = 4 * tid; i < n; i += 4 * THREADS) {
        const float4 m = *reinterpret_cast<const float4*>(mass + i);
        const int4 p = *reinterpret_cast<const int4*>(pos + i);
        const uint32_t k[4] = {evict_key(m.x, p.x, a.sinks, recent_from), evict_key(m.y, p.y, a.sinks, recent_from),
                               evict_key(m.z, p.z, a.sinks, recent_from), evict_key(m.w, p.w, a.sinks, recent_from)};
        if (CACHED) *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < n) atomicAdd(&local[k[e] >> 20], 1);
    }
    // every warp's share of the slice, in row order
    const int sub = ((n + WARPS - 1) / WARPS + 127) / 128 * 128;
    const int w0 = min(n, warp * sub), w1 = min(n, w0 + sub);
    const int low_end = a.budget - r0;  // indices below it are rows below the budget
    // f(key, index) for the warp's rows, four in a row to a lane; true for those
    // that may be kept, and their bits are left where `mark`
    auto each = [&](bool mark, auto f) {
#pragma unroll 2
        for (int b = w0; b < w1; b += 128) {
            const int i = b + 4 * lane;
            uint32_t k[4] = {0u, 0u, 0u, 0u};
            if (CACHED) {
                if (i < w1) {
                    const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
                    k[0] = v.x;
                    k[1] = v.y;
                    k[2] = v.z;
                    k[3] = v.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) k[e] = i + e < w1 ? key_at(i + e) : 0u;
            }
            unsigned bits = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < w1 && f(k[e], i + e)) bits |= 1u << e;
            if (CACHED && mark) {
                bits <<= 4 * (lane & 7);
                bits |= __shfl_xor_sync(FULL, bits, 1);
                bits |= __shfl_xor_sync(FULL, bits, 2);
                bits |= __shfl_xor_sync(FULL, bits, 4);
                if ((lane & 7) == 0) maybe[warp][(b - w0) / 32 + lane / 8] = bits;
            }
        }
    };
    uint32_t prefix = 0, mask = 0;
    int need = a.budget;  // rows still to take among those whose key matches the prefix
    int gt = 0, eq = 0, gt_b = 0, eq_b = 0;  // rows above, equal; the same of rows below the budget
    bool listed = false, ranked = false;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 20 : (pass == 1 ? 8 : 0);
        const uint32_t digit = pass == 2 ? 255u : 4095u;
        int* unit = sel_smem + (pass & 1) * SEL_BINS;
        if (pass > 0) {
            if (CS == 1) local = unit;
            if (listed) {
                for (int x = tid; x < own_n[0]; x += THREADS)
                    if ((list[x] & mask) == prefix) atomicAdd(&local[(list[x] >> shift) & digit], 1);
            } else {
                each(false, [&](uint32_t k, int) {
                    if ((k & mask) == prefix) atomicAdd(&local[(k >> shift) & digit], 1);
                    return false;
                });
            }
        }
        if (CS > 1) {
            __syncthreads();
            for (int i = tid; i < SEL_BINS; i += THREADS) {
                const int v = mine[i];
                if (v == 0) continue;
                mine[i] = 0;
#pragma unroll
                for (int r = 0; r < CS; ++r) peer_add(&unit[i], r, v);
            }
        }
        sync_all();
        // BPT bins a thread, from the highest down
        constexpr int BPT = SEL_BINS / THREADS;
        int c[BPT], sum = 0;
#pragma unroll
        for (int e = 0; e < BPT; ++e) {
            c[e] = unit[SEL_BINS - 1 - (tid * BPT + e)];
            sum += c[e];
            // nobody else looks at this copy; the third pass fills it again, and
            // peers only after the second pass's sync
            unit[SEL_BINS - 1 - (tid * BPT + e)] = 0;
        }
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        int before = x - sum;
        const int mine_w = lane < WARPS ? warp_sum[lane] : 0;
        before += __reduce_add_sync(FULL, lane < warp ? mine_w : 0);
        if (before < need && need <= before + sum) {
#pragma unroll
            for (int e = 0; e < BPT; ++e) {
                if (before < need && need <= before + c[e]) {
                    found[0] = SEL_BINS - 1 - (tid * BPT + e);
                    found[1] = need - before;
                    found[2] = c[e];
                }
                before += c[e];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        need = found[1];
        mask |= digit << shift;
        const int all = found[2];
        if (!listed && all <= SEL_LIST) {
            // the keys of this bin, in any order; those above it count whatever
            // the last digits are
            each(true, [&](uint32_t k, int i) {
                if ((k & mask) < prefix) return false;
                if ((k & mask) > prefix) {
                    ++gt;
                    gt_b += i < low_end;
                } else {
                    const int at = atomicAdd(&own_n[0], 1);
                    list[at] = k;
                    list_at[at] = i;
                }
                return true;
            });
            listed = true;
            __syncthreads();
        }
        if (!listed || all > SEL_CAND) continue;
        if (CS > 1) {
            // what the peers must know: the rows above the bin, and its keys
            const int g = __reduce_add_sync(FULL, gt), gb = __reduce_add_sync(FULL, gt_b);
            if (lane == 0 && g) atomicAdd(&own_n[2], g);
            if (lane == 0 && gb) atomicAdd(&own_n[3], gb);
        }
        for (int x = tid; x < own_n[0]; x += THREADS) {
            const uint32_t k = list[x];
            const bool low = list_at[x] < low_end;
            if ((k & mask) == prefix) {
                const int at = atomicAdd(&own_n[1], 1);
                (CS > 1 ? own_cand : cand)[at] = k;
                own_low[at] = low;
            } else if (CS > 1 && (k & mask) > prefix) {
                atomicAdd(&own_n[2], 1);
                if (low) atomicAdd(&own_n[3], 1);
            }
        }
        sync_all();
        int from = 0, to = 0;
        if (CS > 1) {
            // warp r copies what CTA r has, behind what the CTAs before it have
            const int m = lane < CS ? peer_word(&own_n[1], lane) : 0;
            from = __shfl_sync(FULL, m, warp & 31);
            to = __reduce_add_sync(FULL, lane < warp ? m : 0);
            if (warp < CS)
                for (int i = lane; i < from; i += 32) {
                    cand[to + i] = (uint32_t)peer_word(reinterpret_cast<const int*>(own_cand + i), warp);
                    cand_low[to + i] = peer_word(own_low + i, warp);
                }
            if (warp < CS && lane == 0) {
                if (warp < rank) atomicAdd(&before_cta[0], peer_word(&own_n[2], warp));
                atomicAdd(&unit_low[0], peer_word(&own_n[3], warp));
            }
            __syncthreads();
        }
        if (tid < all) {
            const uint32_t k = cand[tid];
            int above = 0, same = 0, x = 0;
#pragma unroll 4
            for (; x + 4 <= all; x += 4) {
                const uint4 y = *reinterpret_cast<const uint4*>(cand + x);
                above += (y.x > k) + (y.y > k) + (y.z > k) + (y.w > k);
                same += (y.x == k) + (y.y == k) + (y.z == k) + (y.w == k);
            }
            for (; x < all; ++x) {
                above += cand[x] > k;
                same += cand[x] == k;
            }
            if (above < need && need <= above + same) {  // all rows of that key write the same
                found[0] = (int)k;
                found[1] = need - above;
            }
        }
        __syncthreads();
        prefix = (uint32_t)found[0];
        need = found[1];
        if (CS > 1 && warp < CS)
            for (int i = lane; i < from; i += 32) {
                const uint32_t k = cand[to + i];
                if (k < prefix) continue;
                const int which = k == prefix;
                if (warp < rank) atomicAdd(&before_cta[which], 1);
                if (cand_low[to + i]) atomicAdd(&unit_low[which], 1);
            }
        ranked = true;
        break;
    }
    auto count = [&](uint32_t k, int i) {
        gt += k > prefix;
        eq += k == prefix;
        gt_b += k > prefix && i < low_end;
        eq_b += k == prefix && i < low_end;
        return k >= prefix;
    };
    if (!listed)
        each(true, count);
    else
        for (int x = lane; x < own_n[0]; x += 32)
            if (list_at[x] >= w0 && list_at[x] < w1) count(list[x], list_at[x]);
    gt = __reduce_add_sync(FULL, gt);
    eq = __reduce_add_sync(FULL, eq);
    gt_b = __reduce_add_sync(FULL, gt_b);
    eq_b = __reduce_add_sync(FULL, eq_b);
    if (lane == 0) counts[warp] = make_int4(gt, eq, gt_b, eq_b);
    __syncthreads();
    // rows above and equal before this warp's, in this CTA and in those before
    // it; rows below the budget of the whole unit
    int4 c = lane < WARPS ? counts[lane] : make_int4(0, 0, 0, 0);
    int g = __reduce_add_sync(FULL, lane < warp ? c.x : 0), e = __reduce_add_sync(FULL, lane < warp ? c.y : 0);
    int gb = __reduce_add_sync(FULL, c.z), eb = __reduce_add_sync(FULL, c.w);
    if (CS > 1 && ranked) {
        g += before_cta[0];
        e += before_cta[1];
        gb = unit_low[0];
        eb = unit_low[1];
    } else if (CS > 1) {
        const int all_g = __reduce_add_sync(FULL, c.x), all_e = __reduce_add_sync(FULL, c.y);
        if (tid == 0) totals = make_int4(all_g, all_e, gb, eb);
        cluster_sync();
        c = make_int4(0, 0, 0, 0);
        if (lane < CS) {
            const int* p = reinterpret_cast<const int*>(&totals);
            c = make_int4(peer_word(p, lane), peer_word(p + 1, lane), peer_word(p + 2, lane), peer_word(p + 3, lane));
        }
        g += __reduce_add_sync(FULL, lane < rank ? c.x : 0);
        e += __reduce_add_sync(FULL, lane < rank ? c.y : 0);
        gb = __reduce_add_sync(FULL, c.z);
        eb = __reduce_add_sync(FULL, c.w);
    }
    // this thread has read its peers' shared memory for the last time
    if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    const int kept_b = gb + min(eb, need);  // rows kept before the budget
    int32_t* out = a.moves + (size_t)u * a.max_moves * 2;
    // a lane looks after rpl rows in a row
    const int rpl = CACHED ? min(32, sub / 32) : 4;
    for (int b = w0; b < w1; b += 32 * rpl) {
        const int base = b + rpl * lane;
        const unsigned own_rows = base + rpl <= w1 ? FULL >> (32 - rpl) : (base < w1 ? (1u << (w1 - base)) - 1u : 0u);
        unsigned look = own_rows, mg = 0, me = 0;  // rows that may be kept; above, equal
        if (CACHED) {
            const int bit = min(base, w1) - w0;
            look &= __funnelshift_r(maybe[warp][bit >> 5], maybe[warp][(bit >> 5) + 1], bit & 31);
        }
        for (unsigned left = look; left; left &= left - 1) {
            const unsigned bit = left & -left;
            const uint32_t k = key_at(base + __ffs(left) - 1);
            if (k > prefix) mg |= bit;
            else if (k == prefix) me |= bit;
        }
        const int own = __popc(mg) | __popc(me) << 16;
        int x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        const int all = __shfl_sync(FULL, x, 31), gl = g + ((x - own) & 0xffff), el = e + ((x - own) >> 16);
        for (unsigned todo = base < low_end ? own_rows : mg | me; todo; todo &= todo - 1) {
            const unsigned bit = todo & -todo;
            const int r = r0 + base + __ffs(todo) - 1, eq_before = el + __popc(me & (bit - 1));
            const int kept_before = gl + __popc(mg & (bit - 1)) + min(eq_before, need);
            const bool kept = (mg & bit) || ((me & bit) && eq_before < need);
            const int m = kept_before - kept_b, h = r - kept_before;
            if (kept && r >= a.budget && m < a.max_moves) out[2 * m] = r;
            if (!kept && r < a.budget && h < a.max_moves) out[2 * h + 1] = r;
        }
        g += all & 0xffff;
        e += all >> 16;
    }
    if (tid == 0 && rank == 0) a.n_moves[u] = a.budget - kept_b;
    if (CS > 1) asm volatile("barrier.cluster.wait;" ::: "memory");  // no CTA leaves while a peer may read from it
}

template <int CS, int THREADS, bool CACHED>
cudaError_t launch_select_cs(const SelectArgs& a, int dev, cudaStream_t s) {
    const int slice = round_up(ceil_div(a.c.rows, CS), 128);
    const size_t bins = (size_t)(CS > 1 ? 3 : 2) * SEL_BINS * sizeof(int), smem = bins + (CACHED ? (size_t)slice * 4 : 0);
    static std::atomic<bool> set[MAX_DEVICES];
    if (!set[dev].load(std::memory_order_relaxed)) {
        const size_t rows = !CACHED ? 0 : (THREADS == 1024 ? SEL_MAX_SLICE : SEL_LONG + 128);
        const cudaError_t e = cudaFuncSetAttribute(paged_select_kernel<CS, THREADS, CACHED>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, bins + rows * 4);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.c.seqs * a.c.heads * CS));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CS;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_select_kernel<CS, THREADS, CACHED>, a);
}

template <int CS>
cudaError_t launch_select_rows(const SelectArgs& a, int dev, cudaStream_t s) {
    // 512 threads are quicker through their barriers, 1024 through many rows:
    // as replayed graphs, 8.8 against 12.4 us for 256 units of 1344 rows, 10.3
    // against 9.6 for 128 of 4096, 28.7 against 22.7 for 32 of 128k on four
    // CTAs each (10.3 against 10.2 where the limit is, at 4080 rows)
    return a.c.rows / CS < SEL_LONG ? launch_select_cs<CS, 512, true>(a, dev, s)
                                    : launch_select_cs<CS, 1024, true>(a, dev, s);
}

cudaError_t launch_evict_select(const SelectArgs& a, int sms, int dev, cudaStream_t s) {
    const long long units = (long long)a.c.seqs * a.c.heads;
    // more CTAs per unit while each has an SM of its own and rows to work on
    // (two to an SM: 19.7 us instead of 12.2 for 128 units of 8k rows), and as
    // many as the keys need.  lens is not known here, so all this goes by the
    // capacity: 256 units of 1344 rows take 6.0 us at a capacity of 1344, 9.7
    // at 33792 and 58 at 131072
    int cs = 1;
    while (cs < SEL_MAX_CLUSTER && (a.c.rows > cs * (long long)SEL_MAX_SLICE ||
                                    (units * cs * 2 <= sms && a.c.rows / cs >= SEL_LONG)))
        cs *= 2;
    if (a.c.rows > cs * (long long)SEL_MAX_SLICE) return launch_select_cs<SEL_MAX_CLUSTER, 1024, false>(a, dev, s);
    switch (cs) {
        case 1: return launch_select_rows<1>(a, dev, s);
        case 2: return launch_select_rows<2>(a, dev, s);
        case 4: return launch_select_rows<4>(a, dev, s);
        default: return launch_select_rows<8>(a, dev, s);
    }
}

// ---------------------------------------------------------------- eviction: moves
constexpr int APPLY_THREADS = 128;
constexpr int BATCH = 16;  // moves of a warp at a time
constexpr int APPLY_FLIGHT = 2;  // rows that a lane has under way

struct ApplyArgs {
    Cache c;
    int budget, max_moves;
    FastDiv by_warps;  // warps per unit
    int units;
    const int32_t* moves;
    const int32_t* n_moves;
};

// A warp takes BATCH moves: lane l looks up the page of move l's source, lane
// 16 + l that of its destination, so that the chain count -> moves -> page ids
// -> rows is walked once for all of them; then VPR lanes carry a row, 16 bytes
// of K and of V each, with APPLY_FLIGHT rows under way.
template <int VPR>
__global__ void __launch_bounds__(APPLY_THREADS) paged_apply_kernel(const __grid_constant__ ApplyArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    int first, h;
    const int u = a.by_warps.quot(blockIdx.x * (APPLY_THREADS / 32) + (threadIdx.x >> 5), &first);
    if (u >= a.units) return;
    const int s = a.c.by_heads.quot(u, &h);
    // the first moves are read together with their number, used or not
    const int32_t* mv = a.moves + (size_t)u * a.max_moves * 2;
    const bool is_dst = lane >= 16;
    auto move_at = [&](int k0) {
        const int k = k0 + (lane & 15);
        return k < a.max_moves ? mv[2 * k + is_dst] : -1;
    };
    int next = move_at(first * BATCH), n = a.n_moves[u];
    if (n < 0 || n > a.max_moves) {
        if (first == 0 && lane == 0) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        n = n < 0 ? 0 : a.max_moves;
    }
    const size_t o = (size_t)u * a.c.rows;
    constexpr int RP = 32 / VPR;  // rows at a time
    const int piece = (lane % VPR) * 16, sub = lane / VPR;
    for (int k0 = first * BATCH; k0 < n; k0 += (int)a.by_warps.d * BATCH) {
        int row = -1;
        if (k0 + (lane & 15) < n) {
            row = next;
            if (is_dst ? row < 0 || row >= a.budget || row >= a.c.rows : row < a.budget || row >= a.c.rows) {
                report(a.c.dev_err, CKV_DEV_BAD_INDEX);
                row = -1;
            }
        }
        next = move_at(k0 + (int)a.by_warps.d * BATCH);
        int slot = 0;
        const int pg = row < 0 ? -1 : page_of(a.c, s, row, &slot);
        const long long ko = pg * a.c.ks[0] + h * a.c.ks[1] + slot * a.c.ks[2];
        const long long vo = pg * a.c.vs[0] + h * a.c.vs[1] + slot * a.c.vs[2];
        const int dst = __shfl_sync(FULL, row, (lane & 15) + 16);
        const unsigned known = __ballot_sync(FULL, pg >= 0);
        const unsigned good = known & (known >> 16);  // bit l: move l
        if (lane < 16 && ((good >> lane) & 1)) {
            if (a.c.mass) a.c.mass[o + dst] = a.c.mass[o + row];
            if (a.c.pos) a.c.pos[o + dst] = a.c.pos[o + row];
        }
#pragma unroll
        for (int b = 0; b < BATCH; b += RP * APPLY_FLIGHT) {
            if (k0 + b >= n) break;
            uint4 kv[APPLY_FLIGHT], vv[APPLY_FLIGHT];
#pragma unroll
            for (int x = 0; x < APPLY_FLIGHT; ++x) {
                const int m = b + x * RP + sub;
                const long long ks = __shfl_sync(FULL, ko, m), vs = __shfl_sync(FULL, vo, m);
                if ((good >> m) & 1) {
                    kv[x] = *reinterpret_cast<const uint4*>(a.c.K + ks + piece);
                    vv[x] = *reinterpret_cast<const uint4*>(a.c.V + vs + piece);
                }
            }
#pragma unroll
            for (int x = 0; x < APPLY_FLIGHT; ++x) {
                const int m = b + x * RP + sub;
                const long long kd = __shfl_sync(FULL, ko, m + 16), vd = __shfl_sync(FULL, vo, m + 16);
                if ((good >> m) & 1) {
                    *reinterpret_cast<uint4*>(a.c.K + kd + piece) = kv[x];
                    *reinterpret_cast<uint4*>(a.c.V + vd + piece) = vv[x];
                }
            }
        }
    }
    // nothing in this kernel reads lens
    if (h == 0 && first == 0 && lane == 0 && a.c.lens[s] > a.budget) a.c.lens[s] = a.budget;
}

}  // namespace
}  // namespace paged
}  // namespace ckv

using namespace ckv;
using namespace ckv::paged;

extern "C" ckv_status ckv_paged_append(const ckv_paged_cache* cache, const void* k_src, const void* v_src,
                                       const int64_t* k_src_stride, const int64_t* v_src_stride, int32_t n,
                                       const int32_t* counts, const int32_t* start, const int32_t* first,
                                       void* stream) {
    CKV_TRACE("ckv_paged_append");
    AppendArgs a;
    const ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (!k_src || !v_src || !k_src_stride || !v_src_stride || n < 1) return CKV_ERR_ARG;
    const int elem = cache->kv_dtype == CKV_BF16 ? 2 : 4;
    const int32_t extent[3] = {cache->seqs, cache->heads, n};
    for (int i = 0; i < 3; ++i) {
        // sources are only read: a stride of 0 (one row for all) is allowed
        if (k_src_stride[i] < 0 || v_src_stride[i] < 0 || k_src_stride[i] > MAX_STRIDE ||
            v_src_stride[i] > MAX_STRIDE)
            return CKV_ERR_ARG;
        // the stride of a single extent is never multiplied by more than 0
        a.kst[i] = extent[i] > 1 ? k_src_stride[i] * elem : 0;
        a.vst[i] = extent[i] > 1 ? v_src_stride[i] * elem : 0;
    }
    if (!aligned16(k_src) || !aligned16(v_src) || !strides_aligned(a.kst, 3) || !strides_aligned(a.vst, 3))
        return CKV_ERR_ALIGN;
    a.k_src = static_cast<const unsigned char*>(k_src);
    a.v_src = static_cast<const unsigned char*>(v_src);
    a.counts = counts;
    a.start = start == a.c.lens ? nullptr : start;
    a.first = first == a.c.seen ? nullptr : first;
    a.n = n;
    const int vpr = D * elem / 16;
    const long long per_pass = APPEND_THREADS / vpr * IN_FLIGHT;
    long long blocks = ((long long)n * a.c.heads + per_pass - 1) / per_pass;
    if (blocks > 4096) blocks = 4096;
    while (blocks > 1 && blocks * a.c.seqs > 0x7fffffffLL) blocks = (blocks + 1) / 2;
    // a thread's item index plus a step stays below 2^31
    if ((long long)n * a.c.heads + (blocks + 1) * per_pass > 0x7fffffffLL) return CKV_ERR_ARG;
    a.by_blocks = FastDiv((uint32_t)blocks);
    // lens and seen may be advanced by the copying kernel where no other block
    // can still read the old values, whichever argument they are read through
    const int32_t* reads[3] = {a.start ? a.start : a.c.lens, a.first ? a.first : a.c.seen, counts};
    bool in_place = false;
    for (const int32_t* r : reads) {
        if (!same_or_apart(r, a.c.lens, a.c.seqs) || !same_or_apart(r, a.c.seen, a.c.seqs)) return CKV_ERR_ARG;
        if (r && (r == a.c.lens || r == a.c.seen)) in_place = true;
    }
    a.advance = !in_place || blocks == 1;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)(blocks * a.c.seqs)), block(APPEND_THREADS);
    cudaError_t e = vpr == 16 ? launch_dependent(paged_append_kernel<16>, grid, block, 0, s, a)
                              : launch_dependent(paged_append_kernel<32>, grid, block, 0, s, a);
    if (e == cudaSuccess && !a.advance)
        e = launch_dependent(paged_advance_kernel, dim3(ceil_div(a.c.seqs, 128)), dim3(128), 0, s, a);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}

namespace {
ckv_status check_evict(const Cache& c, int budget, int max_moves) {
    // the kernels count the words of a unit's moves in 32 bits; no eviction has more than 2^30 - 16
    if (budget < 1 || max_moves < 0 || max_moves > 1 << 30) return CKV_ERR_ARG;
    const int most = budget < c.rows - budget ? budget : c.rows - budget;  // negative if nothing can be over budget
    return max_moves < most ? CKV_ERR_CAPACITY : CKV_OK;
}
}  // namespace

extern "C" ckv_status ckv_paged_evict_select(const ckv_paged_cache* cache, int32_t budget, int32_t sinks,
                                             int32_t recent, int32_t max_moves, int32_t* moves, int32_t* n_moves,
                                             void* stream) {
    CKV_TRACE("ckv_paged_evict_select");
    SelectArgs a;
    ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (!a.c.mass || !a.c.pos || !a.c.seen || (!moves && max_moves > 0) || !n_moves) return CKV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(moves) & 7u) return CKV_ERR_ALIGN;
    if (sinks < 0 || recent < 0 || (long long)sinks + recent > budget) return CKV_ERR_ARG;
    st = check_evict(a.c, budget, max_moves);
    if (st != CKV_OK) return st;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.max_moves = max_moves;
    a.moves = moves;
    a.n_moves = n_moves;
    if ((long long)a.c.seqs * a.c.heads > 0x7fffffffLL / SEL_MAX_CLUSTER) return CKV_ERR_ARG;
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return CKV_ERR_CUDA;
    const cudaError_t e = launch_evict_select(a, sms, dev, (cudaStream_t)stream);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}

extern "C" ckv_status ckv_paged_evict_apply(const ckv_paged_cache* cache, int32_t budget, int32_t max_moves,
                                            const int32_t* moves, const int32_t* n_moves, void* stream) {
    CKV_TRACE("ckv_paged_evict_apply");
    ApplyArgs a;
    ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if ((!moves && max_moves > 0) || !n_moves) return CKV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(moves) & 7u) return CKV_ERR_ALIGN;
    st = check_evict(a.c, budget, max_moves);
    if (st != CKV_OK) return st;
    a.budget = budget;
    a.max_moves = max_moves;
    a.moves = moves;
    a.n_moves = n_moves;
    const int vpr = D * (cache->kv_dtype == CKV_BF16 ? 2 : 4) / 16;
    const long long units = (long long)a.c.seqs * a.c.heads;
    const int sms = sm_count(nullptr);
    if (sms < 1) return CKV_ERR_CUDA;
    // as many warps as the moves could keep busy, up to 32 to an SM in all
    long long warps = ceil_div(max_moves, BATCH);
    const long long most = (32LL * sms + units - 1) / units;
    if (warps > most) warps = most;
    if (warps < 1) warps = 1;
    a.by_warps = FastDiv((uint32_t)warps);
    a.units = (int)units;
    const long long blocks = (warps * units + APPLY_THREADS / 32 - 1) / (APPLY_THREADS / 32);
    if (blocks * (APPLY_THREADS / 32) > 0x7fffffffLL) return CKV_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)blocks), block(APPLY_THREADS);
    const cudaError_t e = vpr == 16 ? launch_dependent(paged_apply_kernel<16>, grid, block, 0, s, a)
                                    : launch_dependent(paged_apply_kernel<32>, grid, block, 0, s, a);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
