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
};

ckv_status check_cache(const ckv_paged_cache* c, Cache* out);
// SM count of the current device (looked up once per device); 0 on failure
int sm_count(int* dev);

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
__device__ __forceinline__ int page_of(const Cache& c, int s, int r) {
    const int p = c.table[(size_t)s * c.max_pages + r / c.page];
    if (p >= 0 && p < c.n_pages) return p;
    report(c.dev_err, CKV_DEV_BAD_INDEX);
    return -1;
}

}  // namespace paged
}  // namespace ckv
