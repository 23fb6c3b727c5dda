// Declarations shared by the paged cache's kernel files.
#pragma once
#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace ckv {
namespace paged {

constexpr int TILE = 16;         // pages are multiples of this many rows
constexpr int MAX_G = 16;        // query heads per KV head
constexpr int MAX_DEVICES = 64;
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

ckv_status check_cache(const ckv_paged_cache* c, Cache* out);
// SM count of the current device (looked up once per device); 0 on failure
int sm_count(int* dev);

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
