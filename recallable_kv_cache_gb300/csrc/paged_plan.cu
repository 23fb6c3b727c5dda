// Paged cache: which pages the sequences get, and where each token of a step
// goes, from the sequences' lengths on the device.
//
// Three running sums over the sequences settle everything: of tokens (where a
// sequence's stand, and whether they fit), of pages wanted (which of the ring's
// free pages are whose, and from where on there are too few) and of pages handed
// back.  The state of a few hundred sequences is a few KB, so the call is bound
// by latency: one CTA keeps the sums in shared memory, and moves pages and
// writes the slot map by items (a page, a token), each finding its sequence in
// them by bisection, so that one long prompt is as spread out as many short
// ones (32 sequences of a token each: 2.9 us).  Where many pages change hands the
// bisections are what it takes (509 sequences that hand 10.7k pages back: 9.3 us,
// 60 % of the issue slots busy).  Slot maps of many tokens are left to a second
// kernel on all SMs (48 prompts of 46k tokens: 5.9 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace ckv {
namespace paged {
namespace {

constexpr unsigned FULL = 0xffffffffu;
// slot map entries up to which the planning CTA writes them itself
constexpr int SLOTS_HERE = 2048;
constexpr int SLOT_THREADS = 256;

struct PlanArgs {
    Cache c;
    int32_t* table;
    const int32_t* counts;
    const int32_t* start;  // never null: lens where the caller gave none
    const int32_t* first;  // seen where the caller gave none; null without seen: the rows
    const int32_t* shared;
    const int32_t* held_in;
    int32_t* held_out;
    int32_t* ring;
    const int32_t* span_in;
    int32_t* span_out;
    int32_t* granted;
    int32_t* starts;
    int4* slots;
    int cap, n_slots;
    int slots_here;
    FastDiv by_blocks;  // blocks per sequence of the slot map's kernel
};

// A sequence as the call finds it.
struct Seq {
    int start, count, first, held;
    int need;  // pages; held where the sequence is not to be touched
    bool ok;   // may take part: its numbers are in range
};
__device__ __forceinline__ Seq look(const PlanArgs& a, int s) {
    Seq q;
    q.start = a.start[s];
    q.count = a.counts[s];
    q.first = a.first ? a.first[s] : q.start;
    q.held = a.held_in[s];
    const int shared = a.shared ? a.shared[s] : 0;
    q.ok = q.start >= 0 && q.count >= 0 && q.first >= 0 && shared >= 0 && shared <= q.held && q.held <= a.c.max_pages &&
           (long long)q.start + q.count <= a.c.rows && (long long)q.first + q.count <= 0x7fffffffLL;
    q.need = q.held;
    if (q.ok) {
        int rem;
        const int pages = a.c.by_page.quot(q.start + q.count, &rem);
        q.need = max(pages + (rem > 0), shared);
    }
    return q;
}

// the sums that an item (a token, a page) is looked up in, one entry for the
// chunk of sequences of each thread
template <int NT>
struct Sums {
    long long tokens[NT + 1], takes[NT + 1], gives[NT + 1];  // before the chunk; [NT]: in all
};

// inclusive sums of v over the CTA's threads
template <int NT>
__device__ __forceinline__ long long scan(long long v, long long* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(FULL, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w)
        if (w < warp) v += warp_sum[w];
    __syncthreads();
    return v;
}
// place i of a ring whose first is `head` < cap, for i <= cap
__device__ __forceinline__ int ring_at(int head, long long i, int cap) {
    const long long x = head + i;
    return (int)(x >= cap ? x - cap : x);
}
// The sequence (or the chunk of them) that item i belongs to: the last of the NT
// whose items begin at i or before.
template <int NT, typename T>
__device__ __forceinline__ int owner_of(const T* begin, T i) {
    int lo = 0;
#pragma unroll
    for (int step = NT / 2; step > 0; step >>= 1)
        if (begin[lo + step] <= i) lo += step;
    return lo;
}

__device__ __forceinline__ int4 slot_entry(const PlanArgs& a, int s, int row, int position) {
    int slot;
    const int page = page_of(a.c, s, row, &slot);
    if (page < 0) return make_int4(-1, -1, -1, -1);
    return make_int4(page * a.c.page + slot, s, row, position);
}

// Sums that stop at `most`, below 2^31 (so that 32 bits do for whatever the inputs are):
// inclusive, of two values at a time.  `warp_sum` is not used again by a call
// that no barrier parts from this one.
template <int NT>
__device__ __forceinline__ uint2 sums_to(uint2 v, uint2 most, uint2* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto add = [&](uint2& x, int o, bool in) {
        const unsigned y = __shfl_up_sync(FULL, x.x, o), z = __shfl_up_sync(FULL, x.y, o);
        if (in) x = make_uint2(min(x.x + y, most.x), min(x.y + z, most.y));
    };
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) add(v, o, lane >= o);
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    uint2 w = lane < NT / 32 ? warp_sum[lane] : make_uint2(0, 0);
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) add(w, o, lane >= o);
    const unsigned x = __shfl_sync(FULL, w.x, max(warp, 1) - 1), y = __shfl_sync(FULL, w.y, max(warp, 1) - 1);
    return warp ? make_uint2(min(v.x + x, most.x), min(v.y + y, most.y)) : v;
}

// Up to NT sequences, one CTA, a thread a sequence.
template <int NT>
__global__ void __launch_bounds__(NT) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
    constexpr int AT_A_TIME = 4;  // pages that a thread has under way
    __shared__ uint2 warp_sum[2][NT / 32];
    __shared__ unsigned tokens_from[NT + 1], takes_from[NT + 1], gives_from[NT + 1];  // [NT]: in all
    __shared__ int4 seq[NT];  // start, first, pages in hand, pages to have
    __shared__ unsigned taken_here;  // pages really taken
    const int s = threadIdx.x;
    if (s == 0) taken_here = tokens_from[0] = takes_from[0] = gives_from[0] = 0;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    int head = a.span_in[0], avail = a.span_in[1];
    Seq q{0, 0, 0, 0, 0, true};
    if (s < a.c.seqs) q = look(a, s);
    if (head < 0 || head >= a.cap || avail < 0 || avail > a.cap) {
        if (s == 0) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        head = avail = 0;
    }
    const unsigned n = max(0, q.count), most = (unsigned)a.n_slots + 1;
    const unsigned tokens_end = sums_to<NT>(make_uint2(min(n, most), 0), make_uint2(most, 0), warp_sum[0]).x;
    if (tokens_end > (unsigned)a.n_slots && n) q.ok = false;
    if (!q.ok) {
        q.need = q.held;
        report(a.c.dev_err, CKV_DEV_BAD_COUNT);
    }
    const unsigned take = max(0, q.need - q.held), give = max(0, q.held - q.need);
    const uint2 end = sums_to<NT>(make_uint2(min(take, avail + 1u), min(give, a.cap + 1u)),
                                  make_uint2(avail + 1u, a.cap + 1u), warp_sum[1]);
    // served in order while the pages last: of the takes, those served are the first
    const bool served = q.ok && (take == 0 || end.x <= (unsigned)avail);
    if (served && take) atomicMax(&taken_here, end.x);
    // (a sum that has stopped is of items that are not served, or have no place)
    tokens_from[s + 1] = tokens_end;
    takes_from[s + 1] = end.x;
    gives_from[s + 1] = end.y;
    seq[s] = make_int4(served ? q.start : -1, q.first, q.held, q.need);
    __syncthreads();
    const unsigned taken = taken_here, given = min(gives_from[NT], (unsigned)(a.cap - avail));
    if (s == 0 && given < gives_from[NT]) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
    // the pages: the first `taken` from the ring's head, then those handed back
    for (unsigned i0 = s; i0 < taken + given; i0 += NT * AT_A_TIME) {
        int32_t* to[AT_A_TIME];
        int32_t page[AT_A_TIME];
#pragma unroll
        for (int k = 0; k < AT_A_TIME; ++k) {
            const unsigned i = i0 + k * NT;
            to[k] = nullptr;
            if (i < taken + given) {
                const bool takes = i < taken;
                const unsigned item = takes ? i : i - taken;
                const unsigned* from = takes ? takes_from : gives_from;
                const int o = owner_of<NT>(from, item);
                int32_t* row = a.table + (size_t)o * a.c.max_pages + (takes ? seq[o].z : seq[o].w) + (item - from[o]);
                int32_t* ring = a.ring + ring_at(head, takes ? item : (long long)avail + item, a.cap);
                page[k] = takes ? *ring : *row;
                to[k] = takes ? row : ring;
            }
        }
#pragma unroll
        for (int k = 0; k < AT_A_TIME; ++k)
            if (to[k]) *to[k] = page[k];
    }
    if (a.slots_here) {
        __syncthreads();  // the table is whole
        for (int t = s; t < a.n_slots; t += NT) {
            int4 e = make_int4(-1, -1, -1, -1);
            if (t < (int)tokens_from[NT]) {
                const int o = owner_of<NT>(tokens_from, (unsigned)t), j = t - (int)tokens_from[o];
                const int4 v = seq[o];
                if (v.x >= 0) e = slot_entry(a, o, v.x + j, v.y + j);
            }
            a.slots[t] = e;
        }
    }
    // The outputs: a thread wrote what only it has read, and read it before the barriers.
    if (s < a.c.seqs) {
        const int got = served ? q.count : 0;
        a.starts[s] = (int)min(tokens_from[s], (unsigned)a.n_slots);
        a.granted[s] = got;
        a.held_out[s] = served ? q.need : q.held;
        if (q.ok) {
            a.c.lens[s] = q.start + got;
            if (a.c.seen) a.c.seen[s] = q.first + got;
        }
    }
    if (s == 0) {
        a.starts[a.c.seqs] = (int)min(tokens_from[NT], (unsigned)a.n_slots);
        a.span_out[0] = ring_at(head, taken, a.cap);
        a.span_out[1] = avail - (int)taken + (int)given;
    }
}

// More sequences.  One CTA; a thread has a chunk of neighbouring sequences and
// looks at them three times, the later times in the first-level cache, and an item
// that has found its chunk walks through it (1500 / 4096 sequences of a token each
// 14 / 22 us, and 47 / 144 where they hand 31 / 84 thousand pages back).
template <int NT>
__global__ void __launch_bounds__(NT) paged_plan_many_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ Sums<NT> sums;
    __shared__ long long warp_sum[NT / 32], taken_sum[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int chunk = (a.c.seqs + NT - 1) / NT;
    const int s0 = min(a.c.seqs, tid * chunk), s1 = min(a.c.seqs, s0 + chunk);
    int head = a.span_in[0], avail = a.span_in[1];
    if (head < 0 || head >= a.cap || avail < 0 || avail > a.cap) {
        if (tid == 0) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        head = avail = 0;
    }
    long long tokens = 0;
    for (int s = s0; s < s1; ++s) tokens += max(0, a.counts[s]);
    const long long tokens_end = scan<NT>(tokens, warp_sum);
    sums.tokens[tid] = tokens_end - tokens;
    if (tid == NT - 1) sums.tokens[NT] = tokens_end;
    // f(sequence, its numbers, pages it wants, pages it hands back, its first token)
    auto each = [&](auto f) {
        long long at = tokens_end - tokens;
        for (int s = s0; s < s1; ++s) {
            Seq q = look(a, s);
            const long long t = at;
            at += max(0, q.count);
            if (at > a.n_slots && q.count > 0) q.ok = false;
            if (!q.ok) q.need = q.held;
            f(s, q, max(0, q.need - q.held), max(0, q.held - q.need), t);
        }
    };
    long long takes = 0, gives = 0;
    each([&](int, const Seq& q, int take, int give, long long) {
        if (!q.ok) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
        takes += take;
        gives += give;
    });
    const long long takes_end = scan<NT>(takes, warp_sum), gives_end = scan<NT>(gives, warp_sum);
    sums.takes[tid] = takes_end - takes;
    sums.gives[tid] = gives_end - gives;
    if (tid == NT - 1) {
        sums.takes[NT] = takes_end;
        sums.gives[NT] = gives_end;
    }
    // pages really taken: those of the sequences that are not refused
    long long taken = 0, run = takes_end - takes;
    each([&](int, const Seq&, int take, int, long long) {
        run += take;
        if (run <= avail) taken += take;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) taken += __shfl_xor_sync(FULL, taken, o);
    if (lane == 0) taken_sum[warp] = taken;
    __syncthreads();
    taken = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) taken += taken_sum[w];

    // the pages, one a thread.  Refused sequences come after all that are served,
    // but for those that take nothing, so the pages taken are the first `taken`.
    const long long given = min(sums.gives[NT], (long long)a.cap - avail);
    if (tid == 0 && given < sums.gives[NT]) report(a.c.dev_err, CKV_DEV_BAD_COUNT);
    for (long long i = tid; i < taken + given; i += NT) {
        const bool takes_page = i < taken;
        const long long item = takes_page ? i : i - taken;
        const long long* list = takes_page ? sums.takes : sums.gives;
        const int c = owner_of<NT>(list, item);
        long long left = item - list[c];
        int s = c * chunk;
        Seq q = look(a, s);
        // which sequences have no place for their tokens is settled by the running sum
        long long at = sums.tokens[c];
        for (;;) {
            at += max(0, q.count);
            if (at > a.n_slots && q.count > 0) q.need = q.held;
            const int n = max(0, takes_page ? q.need - q.held : q.held - q.need);
            if (left < n) break;
            left -= n;
            q = look(a, ++s);
        }
        int32_t* row = a.table + (size_t)s * a.c.max_pages;
        if (takes_page) {
            row[q.held + left] = a.ring[ring_at(head, item, a.cap)];
        } else {
            a.ring[ring_at(head, avail + item, a.cap)] = row[q.need + left];
        }
    }
    __syncthreads();  // the table is whole, and nobody reads the inputs' table rows any more
    if (a.slots_here) {
        for (int t = tid; t < a.n_slots; t += NT) {
            int4 e = make_int4(-1, -1, -1, -1);
            if (t < sums.tokens[NT]) {
                const int c = owner_of<NT>(sums.tokens, (long long)t);
                long long left = t - sums.tokens[c], before = sums.takes[c], at = sums.tokens[c];
                int s = c * chunk;
                Seq q = look(a, s);
                for (;;) {
                    at += max(0, q.count);
                    if (at > a.n_slots && q.count > 0) q.ok = false;
                    if (q.ok) before += max(0, q.need - q.held);
                    if (left < max(0, q.count)) break;
                    left -= max(0, q.count);
                    q = look(a, ++s);
                }
                if (q.ok && (q.need <= q.held || before <= avail))
                    e = slot_entry(a, s, q.start + (int)left, q.first + (int)left);
            }
            a.slots[t] = e;
        }
        __syncthreads();
    }
    // the outputs last: inputs may be the same arrays
    run = takes_end - takes;
    each([&](int s, const Seq& q, int take, int, long long t) {
        run += take;
        const bool served = q.ok && (take == 0 || run <= avail);
        const int n = served ? q.count : 0;
        a.starts[s] = (int)min(t, (long long)a.n_slots);
        a.granted[s] = n;
        a.held_out[s] = served ? q.need : q.held;
        if (q.ok) {
            a.c.lens[s] = q.start + n;
            if (a.c.seen) a.c.seen[s] = q.first + n;
        }
    });
    if (tid == 0) {
        a.starts[a.c.seqs] = (int)min(sums.tokens[NT], (long long)a.n_slots);
        a.span_out[0] = ring_at(head, taken, a.cap);
        a.span_out[1] = (int)(avail - taken + given);
    }
}

// The slot map of many tokens, from what the plan has left: a few blocks to a
// sequence, which stride over its tokens.
__global__ void __launch_bounds__(SLOT_THREADS) paged_slots_kernel(const __grid_constant__ PlanArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    int b;
    const int s = a.by_blocks.quot(blockIdx.x, &b);
    const int t0 = a.starts[s], t1 = a.starts[s + 1], n = a.granted[s];
    const int row = a.c.lens[s] - n;
    // first may be lens, which the plan has moved on (start is lens then, too)
    const int position = a.c.seen ? a.c.seen[s] - n : (a.first && a.first != a.c.lens ? a.first[s] : row);
    const int step = a.by_blocks.d * SLOT_THREADS;
    for (int j = b * SLOT_THREADS + threadIdx.x; j < t1 - t0; j += step)
        a.slots[t0 + j] = n ? slot_entry(a, s, row + j, position + j) : make_int4(-1, -1, -1, -1);
    const long long all = (long long)gridDim.x * SLOT_THREADS;
    for (long long t = a.starts[a.c.seqs] + (long long)blockIdx.x * SLOT_THREADS + threadIdx.x; t < a.n_slots; t += all)
        a.slots[t] = make_int4(-1, -1, -1, -1);
}

}  // namespace
}  // namespace paged
}  // namespace ckv

using namespace ckv;
using namespace ckv::paged;

extern "C" ckv_status ckv_paged_plan(const ckv_paged_cache* cache, const int32_t* counts, const int32_t* start,
                                     const int32_t* first, const int32_t* shared, const int32_t* held_in,
                                     int32_t* held_out, int32_t* free_pages, int32_t free_cap, const int32_t* span_in,
                                     int32_t* span_out, int32_t* granted, int32_t* starts, int32_t* slots,
                                     int32_t n_slots, void* stream) {
    CKV_TRACE("ckv_paged_plan");
    PlanArgs a;
    const ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (!counts || !held_in || !held_out || !free_pages || !span_in || !span_out || !granted || !starts || !slots ||
        free_cap < 1 || n_slots < 1 || (long long)a.c.n_pages * a.c.page > 0x7fffffffLL)
        return CKV_ERR_ARG;
    if (n_slots > 0x7fffffff - (1 << 24)) return CKV_ERR_ARG;  // indices plus a grid's step stay below 2^31
    if (free_cap == 0x7fffffff) return CKV_ERR_ARG;  // sums of pages stop at free_cap + 1, and two of them stay below 2^32
    if (!aligned16(slots)) return CKV_ERR_ALIGN;
    a.start = start ? start : a.c.lens;
    a.first = first ? first : a.c.seen;
    a.shared = shared;
    a.counts = counts;
    a.held_in = held_in;
    a.held_out = held_out;
    a.table = const_cast<int32_t*>(a.c.table);
    a.ring = free_pages;
    a.span_in = span_in;
    a.span_out = span_out;
    a.granted = granted;
    a.starts = starts;
    a.slots = reinterpret_cast<int4*>(slots);
    a.cap = free_cap;
    a.n_slots = n_slots;
    // every array written against every other array: apart, but for the pairs
    // whose elements are read before they are written
    struct Range {
        const void* p;
        long long n;
    };
    const long long S = a.c.seqs;
    const Range writes[9] = {{a.c.lens, S}, {a.c.seen, S}, {held_out, S}, {span_out, 2}, {granted, S},
                             {starts, S + 1}, {slots, 4LL * n_slots}, {free_pages, free_cap},
                             {a.table, S * a.c.max_pages}};
    const Range reads[6] = {{counts, S}, {a.start, S}, {a.first, S}, {shared, S}, {held_in, S}, {span_in, 2}};
    auto apart = [](const Range& x, const Range& y) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(x.p), q = reinterpret_cast<uintptr_t>(y.p);
        return !p || !q || p + 4 * (uintptr_t)x.n <= q || q + 4 * (uintptr_t)y.n <= p;
    };
    for (int i = 0; i < 9; ++i) {
        for (int j = 0; j < i; ++j)
            if (!apart(writes[i], writes[j])) return CKV_ERR_ARG;
        for (int j = 0; j < 6; ++j) {
            // lens and seen: counts, start and first; held_out: held_in; span_out: span_in
            const bool may_be_same = (i < 2 && j < 3) || (i == 2 && j == 4) || (i == 3 && j == 5);
            if (!apart(writes[i], reads[j]) && !(may_be_same && writes[i].p == reads[j].p)) return CKV_ERR_ARG;
        }
    }
    // (positions that count from the old lens, rows from other numbers, and no
    // seen: after the plan nothing holds them any more, so it writes the map)
    a.slots_here = n_slots <= SLOTS_HERE || (!a.c.seen && a.first == a.c.lens && a.start != a.c.lens);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (S <= 256 && (n_slots <= 512 || !a.slots_here))
        e = launch_dependent(paged_plan_kernel<256>, dim3(1), dim3(256), 0, s, a);
    else if (S <= 1024)
        e = launch_dependent(paged_plan_kernel<1024>, dim3(1), dim3(1024), 0, s, a);
    else
        e = launch_dependent(paged_plan_many_kernel<1024>, dim3(1), dim3(1024), 0, s, a);
    if (e == cudaSuccess && !a.slots_here) {
        // about one token a thread where the sequences are alike
        const long long share = ((long long)n_slots + S - 1) / S;
        long long blocks = (share + SLOT_THREADS - 1) / SLOT_THREADS;
        if (blocks > 64) blocks = 64;
        while (blocks > 1 && blocks * S > (1 << 16)) blocks = (blocks + 1) / 2;
        a.by_blocks = FastDiv((uint32_t)blocks);
        e = launch_dependent(paged_slots_kernel, dim3((unsigned)(blocks * S)), dim3(SLOT_THREADS), 0, s, a);
    }
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
