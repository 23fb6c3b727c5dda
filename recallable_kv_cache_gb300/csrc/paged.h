// Declarations shared by the paged cache's kernel files.
#pragma once
#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace ckv {
namespace paged {

constexpr int TILE = 16;         // pages are multiples of this many rows
constexpr int MAX_G = 16;        // query heads per KV head
constexpr int MAX_DEVICES = 64;
constexpr int MAX_GRID = 256;    // CTAs a workspace is laid out for (a GB300 has 152 SMs)
constexpr long long MAX_STRIDE = 1LL << 37;  // elements; a tensor map's strides stay below 2^40 bytes

// Quotient by a divisor fixed at launch, for dividends below 2^31: with s =
// ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, n / d = (hi32(m n) + n) >> s
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994; n below 2^31 keeps the sum inside 32 bits).
struct FastDiv {
    uint32_t d, m, s;
    __host__ __device__ FastDiv() : d(1), m(1), s(0) {}
    __host__ explicit FastDiv(uint32_t div) : d(div), s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)((((1ull << s) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ int quot(int n) const { return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s); }
    __device__ __forceinline__ int quot(int n, int* rem) const {
        const int q = quot(n);
        *rem = n - q * (int)d;
        return q;
    }
};

// What the kernels take of a ckv_paged_cache.
struct Cache {
    unsigned char* K;
    unsigned char* V;
    long long ks[3], vs[3];  // byte strides: page, head, row
    const int32_t* table;
    int32_t* lens;
    float* mass;
    int32_t* pos;
    int32_t* seen;
    int32_t* dev_err;
    int n_pages, heads, page, seqs, max_pages;
    int rows;  // max_pages * page
    FastDiv by_page, by_heads;
};

// The deal: `total` tiles to the warps of n_cta CTAs, in order, as evenly as
// they go (shares of q + 1 tiles, then of q).
struct Deal {
    int total, n_cta, warps, q, r;
    __device__ __forceinline__ Deal(int total_, int n_cta_, int warps_) : total(total_), n_cta(n_cta_), warps(warps_) {
        q = total / (n_cta * warps);
        r = total - q * (n_cta * warps);
    }
    static __device__ __forceinline__ int ctas(int total, int warps, int grid) {
        return max(1, min(grid, (total + warps - 1) / warps));
    }
    __device__ __forceinline__ int begin_warp(int w) const { return w * q + min(w, r); }  // w: across CTAs
    __device__ __forceinline__ int begin_cta(int c) const { return begin_warp(c * warps); }
    // the CTA whose share holds tile t
    __device__ __forceinline__ int cta_of(int t) const {
        const int w = t < (q + 1) * r ? t / (q + 1) : r + (t - (q + 1) * r) / q;
        return w / warps;
    }
};

ckv_status check_cache(const ckv_paged_cache* c, Cache* out);
// SM count of the current device (looked up once per device); 0 on failure
int sm_count(int* dev);

bool encode_pool(CUtensorMap* m, const Cache& c, const void* base, const long long* st, bool bf16, bool swizzled,
                 int tile_rows, int pieces_a_box = 0);
// what ckv_paged_set_wait_limit has set
void waits(long long* limit, int* stall);
// bytes of the decode attention's workspace without weights, and where the lse
// (base 2, [seqs][heads * g]) and the parts of its calls stand
size_t attn_workspace(const Cache& c, int g, float** lse2, float** part, void* workspace);
// A partial result of g heads: unnormalised outputs [g][D], maxima [g] (base 2), sums [g].
__host__ __device__ __forceinline__ size_t part_floats(int g) { return ((size_t)g * (D + 2) + 3) / 4 * 4; }
// Decode attention over the rows of each sequence from skip[s] on (device int32,
// multiples of TILE) by *ctas CTAs, bf16.  To follow, as a dependent launch, a kernel that has
// waited for its own predecessor and that writes nothing this one reads; a
// kernel behind it that waits for it has waited for both.  It finds the units of
// up to JOINED_PARTS CTAs as their parts: CTA c's is part 2 c, 2 c + 1 where the
// unit begins in it (left[unit] says which, above its use).
constexpr int JOINED_PARTS = 8;
cudaError_t launch_attn_own_rows(const Cache& c, const int32_t* skip, const int32_t* ctas, int32_t* left, const void* q,
                                 const long long* q_stride, int g, float qscale, float* out, float* lse, void* workspace,
                                 cudaStream_t s);

// Groups of sequences with leading rows in common, as ckv_paged_shared_attn takes them.
struct Groups {
    const int32_t* starts;
    const int32_t* prefix;
    int n;
};
// Up to this many groups and sequences a CTA looks them up by itself, a lane a group.
constexpr int FEW_GROUPS = 32, FEW_SEQS = 1024;
// Decode attention, fp32, of few groups: a sequence attends its own number of rows, or
// its group's where that is more.
cudaError_t launch_attn_in_groups(const Cache& c, const Groups& groups, const void* q, const long long* q_stride, int g,
                                  float qscale, float* out, float* lse, void* workspace, cudaStream_t s);

// two arrays of n 32-bit elements that are one and the same (an element is read
// before it is written) or do not overlap; no array overlaps nothing
inline bool same_or_apart(const void* x, const void* y, long long n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return !x || !y || a == b || (a < b ? b - a : a - b) >= (uintptr_t)n * 4;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ void report(int32_t* dev_err, int code) {
    if (dev_err) atomicCAS(dev_err, 0, code);
}
// rows held by sequence s, clamped to [0, rows]
__device__ __forceinline__ int rows_held(const Cache& c, int s) {
    const int n = c.lens[s];
    return n < 0 ? 0 : (n > c.rows ? c.rows : n);
}
__device__ __forceinline__ void check_len(const Cache& c, int s) {
    const int n = c.lens[s];
    if (n < 0 || n > c.rows) report(c.dev_err, CKV_DEV_BAD_COUNT);
}
// page holding row r of sequence s, -1 (and the error word) if the id is bad
__device__ __forceinline__ int page_of(const Cache& c, int s, int r, int* slot) {
    const int p = c.table[(size_t)s * c.max_pages + c.by_page.quot(r, slot)];
    if (p >= 0 && p < c.n_pages) return p;
    report(c.dev_err, CKV_DEV_BAD_INDEX);
    return -1;
}

}  // namespace paged
}  // namespace ckv
