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
    if (!aligned16(c->K) || !aligned16(c->V) || !strides_aligned(o->ks, 3) || !strides_aligned(o->vs, 3))
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
    return CKV_OK;
}

namespace {

constexpr unsigned FULL = 0xffffffffu;

// ---------------------------------------------------------------- append
constexpr int APPEND_THREADS = 256;

struct AppendArgs {
    Cache c;
    const unsigned char* k_src;
    const unsigned char* v_src;
    long long kst[3], vst[3];  // byte strides: sequence, head, row
    const int32_t* counts;
    const int32_t* start;
    const int32_t* first;
    int n;
    int blocks_per_seq;
    int advance;  // this kernel writes lens and seen
};

// r0, p0 and the row count of sequence s; count -1 if it must be left alone
__device__ __forceinline__ int append_plan(const AppendArgs& a, int s, int* r0, int* p0) {
    *r0 = a.start ? a.start[s] : a.c.lens[s];
    *p0 = a.first ? a.first[s] : (a.c.seen ? a.c.seen[s] : 0);
    const int cnt = a.counts ? a.counts[s] : a.n;
    if (*r0 < 0 || cnt < 0 || cnt > a.n || (long long)*r0 + cnt > a.c.rows) return -1;
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
// threads take consecutive pieces of a row, then the KV heads of a token.
template <int VPR>
__global__ void __launch_bounds__(APPEND_THREADS) paged_append_kernel(const __grid_constant__ AppendArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int s = blockIdx.x / a.blocks_per_seq, b = blockIdx.x % a.blocks_per_seq;
    int r0, p0;
    const int cnt = append_plan(a, s, &r0, &p0);
    const int H = a.c.heads;
    const int piece = threadIdx.x % VPR;
    const long long items = cnt < 0 ? 0 : (long long)cnt * H;
    const long long step = (long long)a.blocks_per_seq * (APPEND_THREADS / VPR);
    for (long long i = (long long)b * (APPEND_THREADS / VPR) + threadIdx.x / VPR; i < items; i += step) {
        const int j = (int)(i / H), h = (int)(i % H), r = r0 + j;
        const int pg = page_of(a.c, s, r);
        if (pg < 0) continue;
        const int slot = r % a.c.page;
        const uint4 kv = *reinterpret_cast<const uint4*>(a.k_src + s * a.kst[0] + h * a.kst[1] + j * a.kst[2] + piece * 16);
        const uint4 vv = *reinterpret_cast<const uint4*>(a.v_src + s * a.vst[0] + h * a.vst[1] + j * a.vst[2] + piece * 16);
        *reinterpret_cast<uint4*>(a.c.K + pg * a.c.ks[0] + h * a.c.ks[1] + slot * a.c.ks[2] + piece * 16) = kv;
        *reinterpret_cast<uint4*>(a.c.V + pg * a.c.vs[0] + h * a.c.vs[1] + slot * a.c.vs[2] + piece * 16) = vv;
        if (piece == 0) {
            const size_t o = ((size_t)s * H + h) * a.c.rows + r;
            if (a.c.pos) a.c.pos[o] = p0 + j;
            if (a.c.mass) a.c.mass[o] = 0.f;
        }
    }
    if (a.advance) {
        // the plan was read by every thread of the sequence's only block
        // (advance in place), or from start and first, which nothing writes
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
constexpr int SEL_THREADS = 1024;

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

__device__ __forceinline__ int block_exclusive_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const int base = warp ? warp_sums[warp - 1] : 0;
    *total = warp_sums[31];
    __syncthreads();
    return base + x - v;
}

// One CTA per (sequence, KV head).  The key of the budget-th row by a radix
// select (8 bits a pass, histogram in shared memory), then one pass in row
// order: rows above that key are kept, of those equal to it the first ones
// that fit; movers and holes take their ranks from a scan.
__global__ void __launch_bounds__(SEL_THREADS) paged_select_kernel(const __grid_constant__ SelectArgs a) {
    __shared__ int hist[256];
    __shared__ int warp_sums[32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int u = blockIdx.x, s = u / a.c.heads, tid = threadIdx.x;
    if (tid == 0) check_len(a.c, s);
    const int len = rows_held(a.c, s);
    if (len <= a.budget) {
        if (tid == 0) a.n_moves[u] = 0;
        return;
    }
    const float* mass = a.c.mass + (size_t)u * a.c.rows;
    const int32_t* pos = a.c.pos + (size_t)u * a.c.rows;
    const int recent_from = a.c.seen[s] - a.recent;
    uint32_t prefix = 0, mask = 0;
    int need = a.budget;  // rows still to take among those whose key matches the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int r = tid; r < len; r += SEL_THREADS) {
            const uint32_t k = evict_key(mass[r], pos[r], a.sinks, recent_from);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, b = 255;
            while (b > 0 && left > hist[b]) left -= hist[b--];
            s_prefix = prefix | ((uint32_t)b << shift);
            s_need = left;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        mask |= 255u << shift;
    }
    int ties = 0, movers = 0, holes = 0;
    int32_t* out = a.moves + (size_t)u * a.max_moves * 2;
    for (int base = 0; base < len; base += SEL_THREADS) {
        const int r = base + tid;
        const uint32_t k = r < len ? evict_key(mass[r], pos[r], a.sinks, recent_from) : 0u;
        const int tie = r < len && k == prefix;
        int total;
        const int before = block_exclusive_scan(tie, warp_sums, &total);
        const bool kept = r < len && (k > prefix || (tie && ties + before < need));
        ties += total;
        const int mover = kept && r >= a.budget, hole = !kept && r < a.budget;
        const int m = block_exclusive_scan(mover, warp_sums, &total) + movers;
        movers += total;
        const int h = block_exclusive_scan(hole, warp_sums, &total) + holes;
        holes += total;
        if (mover && m < a.max_moves) out[2 * m] = r;
        if (hole && h < a.max_moves) out[2 * h + 1] = r;
    }
    if (tid == 0) a.n_moves[u] = movers;
}

// ---------------------------------------------------------------- eviction: moves
constexpr int APPLY_THREADS = 256;

struct ApplyArgs {
    Cache c;
    int budget, max_moves, blocks_per_unit;
    const int32_t* moves;
    const int32_t* n_moves;
};

template <int VPR>
__global__ void __launch_bounds__(APPLY_THREADS) paged_apply_kernel(const __grid_constant__ ApplyArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int u = blockIdx.x / a.blocks_per_unit, b = blockIdx.x % a.blocks_per_unit;
    const int s = u / a.c.heads, h = u % a.c.heads;
    int n = a.n_moves[u];
    if (n < 0 || n > a.max_moves) {
        if (b == 0 && threadIdx.x == 0) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        n = n < 0 ? 0 : a.max_moves;
    }
    const int32_t* mv = a.moves + (size_t)u * a.max_moves * 2;
    const int piece = threadIdx.x % VPR;
    for (int k = b * (APPLY_THREADS / VPR) + threadIdx.x / VPR; k < n;
         k += a.blocks_per_unit * (APPLY_THREADS / VPR)) {
        const int src = mv[2 * k], dst = mv[2 * k + 1];
        if (src < a.budget || src >= a.c.rows || dst < 0 || dst >= a.budget || dst >= a.c.rows) {
            report(a.c.dev_err, CKV_DEV_BAD_INDEX);
            continue;
        }
        const int p0 = page_of(a.c, s, src), p1 = page_of(a.c, s, dst);
        if (p0 < 0 || p1 < 0) continue;
        const int s0 = src % a.c.page, s1 = dst % a.c.page;
        const uint4 kv = *reinterpret_cast<const uint4*>(a.c.K + p0 * a.c.ks[0] + h * a.c.ks[1] + s0 * a.c.ks[2] + piece * 16);
        const uint4 vv = *reinterpret_cast<const uint4*>(a.c.V + p0 * a.c.vs[0] + h * a.c.vs[1] + s0 * a.c.vs[2] + piece * 16);
        *reinterpret_cast<uint4*>(a.c.K + p1 * a.c.ks[0] + h * a.c.ks[1] + s1 * a.c.ks[2] + piece * 16) = kv;
        *reinterpret_cast<uint4*>(a.c.V + p1 * a.c.vs[0] + h * a.c.vs[1] + s1 * a.c.vs[2] + piece * 16) = vv;
        if (piece == 0) {
            const size_t o = (size_t)u * a.c.rows;
            if (a.c.mass) a.c.mass[o + dst] = a.c.mass[o + src];
            if (a.c.pos) a.c.pos[o + dst] = a.c.pos[o + src];
        }
    }
    // nothing in this kernel reads lens
    if (h == 0 && b == 0 && threadIdx.x == 0 && a.c.lens[s] > a.budget) a.c.lens[s] = a.budget;
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
    for (int i = 0; i < 3; ++i) {
        // sources are only read: a stride of 0 (one row for all) is allowed
        if (k_src_stride[i] < 0 || v_src_stride[i] < 0 || k_src_stride[i] > MAX_STRIDE ||
            v_src_stride[i] > MAX_STRIDE)
            return CKV_ERR_ARG;
        a.kst[i] = k_src_stride[i] * elem;
        a.vst[i] = v_src_stride[i] * elem;
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
    const long long per_pass = APPEND_THREADS / vpr;
    long long blocks = ((long long)n * a.c.heads + 4 * per_pass - 1) / (4 * per_pass);
    if (blocks > 4096) blocks = 4096;
    while (blocks * a.c.seqs > 0x7fffffffLL) blocks = (blocks + 1) / 2;
    a.blocks_per_seq = (int)blocks;
    // lens and seen may be advanced by the copying kernel where no other
    // block can still read the old values
    const bool in_place = !a.start || (a.c.seen && !a.first);
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
    if (budget < 1 || max_moves < 0) return CKV_ERR_ARG;
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
    if (!a.c.mass || !a.c.pos || !a.c.seen || !moves || !n_moves) return CKV_ERR_ARG;
    if (sinks < 0 || recent < 0 || (long long)sinks + recent > budget) return CKV_ERR_ARG;
    st = check_evict(a.c, budget, max_moves);
    if (st != CKV_OK) return st;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.max_moves = max_moves;
    a.moves = moves;
    a.n_moves = n_moves;
    const cudaError_t e = launch_dependent(paged_select_kernel, dim3(a.c.seqs * a.c.heads), dim3(SEL_THREADS), 0,
                                           (cudaStream_t)stream, a);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}

extern "C" ckv_status ckv_paged_evict_apply(const ckv_paged_cache* cache, int32_t budget, int32_t max_moves,
                                            const int32_t* moves, const int32_t* n_moves, void* stream) {
    CKV_TRACE("ckv_paged_evict_apply");
    ApplyArgs a;
    ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (!moves || !n_moves) return CKV_ERR_ARG;
    st = check_evict(a.c, budget, max_moves);
    if (st != CKV_OK) return st;
    a.budget = budget;
    a.max_moves = max_moves;
    a.moves = moves;
    a.n_moves = n_moves;
    const int vpr = D * (cache->kv_dtype == CKV_BF16 ? 2 : 4) / 16;
    const int per_pass = APPLY_THREADS / vpr;
    long long blocks = ((long long)max_moves + 4 * per_pass - 1) / (4 * per_pass);
    if (blocks < 1) blocks = 1;
    const long long units = (long long)a.c.seqs * a.c.heads;
    while (blocks > 1 && blocks * units > (1 << 20)) blocks = (blocks + 1) / 2;
    a.blocks_per_unit = (int)blocks;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)(blocks * units)), block(APPLY_THREADS);
    const cudaError_t e = vpr == 16 ? launch_dependent(paged_apply_kernel<16>, grid, block, 0, s, a)
                                    : launch_dependent(paged_apply_kernel<32>, grid, block, 0, s, a);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
