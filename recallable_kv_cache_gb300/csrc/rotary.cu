// Norms and rotary positions of queries and keys, in one pass: on their own
// (ckv_rotate) or with the keys and values going into a paged cache
// (ckv_paged_append_rotated).
//
//   y = x w / sqrt(mean x^2 + eps),  (y_a, y_b) := A (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//
// Every row is read and written once, so long inputs are bound by HBM (32k tokens
// of 40 rows, bf16: 101 us, 98 % of the copy rate) or, with norms, by issue slots
// (124 us, 80 %), and a step's few rows by latency.  Sixteen lanes have a row, eight channels a lane in
// two pieces of four that hold both channels of its four pairs, whichever way
// they are paired: nothing is exchanged but the sum of squares.  A lane works out
// the angles of its pairs once for all rows of a token that its group has, with
// the first rows under way meanwhile; no block waits for another thread.
//
// The angle of pair i at position p is p turns_i / 2^64 of a turn: the product of
// two integers, whose wrap at 2^64 is the angle's own, so that the angle is as
// exact at position 10^9 as at 1, to 2^-28 of a turn (p w_i in fp32 would be off by
// 0.06 at 10^6).
// The quarter turn nearest to it is taken off before the sine is looked up.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mma_sync.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace ckv {
namespace paged {
namespace {

constexpr int THREADS = 256;
constexpr int LANES = 16;               // lanes of a row
constexpr int GROUPS = THREADS / LANES; // rows that a block has in hand at a time
constexpr int FLIGHT = 4;               // rows that a lane group has under way

struct RotArgs {
    Cache c;  // where PAGED
    const unsigned char* src[3];  // q, k, v
    unsigned char* dst[2];        // q_out, k_out (not where PAGED)
    long long sst[3][2], dst_st[2][2];  // byte strides: token, head
    int rows[3];                  // heads of q, k and v
    int tokens;
    int per_token;                // lane groups to a token: a power of two
    const int32_t* positions;
    const int4* slots;
    const unsigned long long* turns;
    const float* weight[2];
    float eps, amplitude;
    int rot, interleaved;
    long long slots_held;         // n_pages * page
};

// cos and sin of phase / 2^64 of a turn
__device__ __forceinline__ float2 unit_circle(unsigned long long phase) {
    const uint32_t hi = (uint32_t)(phase >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    // what is left is within an eighth of a turn, exact as a float to 2^-24 of itself
    const float x = (float)(int32_t)(hi - (quarter << 30)) * 0x1p-31f;  // in half turns
    float s, c;
    sincospif(x, &s, &c);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

// a lane's eight channels as they are in memory; TOGETHER: its two pieces follow one another
template <typename T, bool TOGETHER>
struct Raw;
template <bool TOGETHER>
struct Raw<__nv_bfloat16, TOGETHER> {
    uint2 v[2];
    __device__ __forceinline__ void load(const unsigned char* p, int a, int b) {
        if (TOGETHER) {
            const uint4 x = *reinterpret_cast<const uint4*>(p + a);
            v[0] = make_uint2(x.x, x.y);
            v[1] = make_uint2(x.z, x.w);
        } else {
            v[0] = *reinterpret_cast<const uint2*>(p + a);
            v[1] = *reinterpret_cast<const uint2*>(p + b);
        }
    }
    __device__ __forceinline__ void store(unsigned char* p, int a, int b) const {
        if (TOGETHER) {
            *reinterpret_cast<uint4*>(p + a) = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
        } else {
            *reinterpret_cast<uint2*>(p + a) = v[0];
            *reinterpret_cast<uint2*>(p + b) = v[1];
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * i] = __uint_as_float(v[i].x << 16);
            x[4 * i + 1] = __uint_as_float(v[i].x & 0xffff0000u);
            x[4 * i + 2] = __uint_as_float(v[i].y << 16);
            x[4 * i + 3] = __uint_as_float(v[i].y & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = make_uint2(mmas::pack2(x[4 * i], x[4 * i + 1]), mmas::pack2(x[4 * i + 2], x[4 * i + 3]));
    }
};
template <bool TOGETHER>
struct Raw<float, TOGETHER> {
    float4 v[2];
    __device__ __forceinline__ void load(const unsigned char* p, int a, int b) {
        v[0] = *reinterpret_cast<const float4*>(p + a);
        v[1] = *reinterpret_cast<const float4*>(p + b);
    }
    __device__ __forceinline__ void store(unsigned char* p, int a, int b) const {
        *reinterpret_cast<float4*>(p + a) = v[0];
        *reinterpret_cast<float4*>(p + b) = v[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) x[4 * i] = v[i].x, x[4 * i + 1] = v[i].y, x[4 * i + 2] = v[i].z, x[4 * i + 3] = v[i].w;
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
};

// A block has GROUPS / per_token tokens, a lane group every per_token-th row of
// its token: queries, then keys, then values (PAGED).
template <typename T, bool PAGED, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const __grid_constant__ RotArgs a) {
    const int tid = threadIdx.x, lane = tid & (LANES - 1), group = tid / LANES;
    const int sub = group & (a.per_token - 1);
    const long long t = (long long)blockIdx.x * (GROUPS / a.per_token) + group / a.per_token;
    // the lane's channels: pairs 4 lane .. 4 lane + 3, or eight behind the rotated ones
    const int reach = a.rot / 8;  // lanes that have pairs
    const bool turns = lane < reach;
    const int at0 = (INTERLEAVED || !turns ? 8 : 4) * lane * (int)sizeof(T);
    const int at1 = at0 + (INTERLEAVED || !turns ? 4 : a.rot / 2) * (int)sizeof(T);
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    if (t >= a.tokens) return;
    int4 place = make_int4(0, 0, 0, 0);
    if (PAGED) {
        place = a.slots[t];
        if (place.x == -1) return;
        if (place.x < 0 || place.x >= a.slots_held ||
            ((a.c.pos || a.c.mass) && (place.y < 0 || place.y >= a.c.seqs || place.z < 0 || place.z >= a.c.rows))) {
            if (lane == 0 && sub == 0) report(a.c.dev_err, CKV_DEV_BAD_INDEX);
            return;
        }
    } else {
        place.w = a.positions[t];
    }
    const unsigned half_warp = 0xffffu << (tid & LANES);
    // row r of the token: whether it is of q, k or v, and its head
    const int all = a.rows[0] + a.rows[1] + (PAGED ? a.rows[2] : 0), first_v = a.rows[0] + a.rows[1];
    auto kind_of = [&](int r, int* h) {
        const int kind = (r >= a.rows[0]) + (PAGED && r >= first_v);
        *h = r - (kind == 0 ? 0 : kind == 1 ? a.rows[0] : first_v);
        return kind;
    };
    Raw<T, INTERLEAVED> raw[FLIGHT];
    auto ask = [&](Raw<T, INTERLEAVED>& to, int r) {
        int h;
        const int kind = kind_of(r, &h);
        to.load(a.src[kind] + t * a.sst[kind][0] + h * a.sst[kind][1], at0, at1);
    };
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i)
        if (sub + i * a.per_token < all) ask(raw[i], sub + i * a.per_token);
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
    if (turns) {
        const ulonglong2* w = reinterpret_cast<const ulonglong2*>(a.turns + 4 * lane);
        const ulonglong2 w0 = w[0], w1 = w[1];
        const unsigned long long f[4] = {w0.x, w0.y, w1.x, w1.y}, p = (unsigned long long)(long long)place.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 cs = unit_circle(p * f[i]);
            c[i] = cs.x * a.amplitude;
            s[i] = cs.y * a.amplitude;
        }
    }
    int slot = 0;
    const long long page = PAGED ? a.c.by_page.quot(place.x, &slot) : 0;
    // each row's registers take the row FLIGHT further on as soon as it is done
#pragma unroll 1
    for (int r0 = sub; r0 < all; r0 += FLIGHT * a.per_token) {
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            const int r = r0 + i * a.per_token;
            if (r >= all) break;  // the same for the group's lanes
            int h;
            const int kind = kind_of(r, &h);
            if (!PAGED || kind < 2) {
                float x[8];
                raw[i].get(x);
                const float* weight = a.weight[kind];
                if (weight) {
                    float sq = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(half_warp, sq, o, LANES);
                    const float scale = rsqrtf(sq * (1.f / D) + a.eps);
                    const float4 u = *reinterpret_cast<const float4*>(weight + at0 / (int)sizeof(T));
                    const float4 v = *reinterpret_cast<const float4*>(weight + at1 / (int)sizeof(T));
                    const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= scale * w[e];
                }
                if (turns) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // pair e: neighbours, or the two pieces' e-th channels
                        float& u = x[INTERLEAVED ? 2 * e : e];
                        float& v = x[INTERLEAVED ? 2 * e + 1 : e + 4];
                        const float y = u * c[e] - v * s[e];
                        v = v * c[e] + u * s[e];
                        u = y;
                    }
                }
                raw[i].put(x);
            }
            unsigned char* to;
            if (PAGED && kind > 0) {
                const long long* st = kind == 1 ? a.c.ks : a.c.vs;
                to = (kind == 1 ? a.c.K : a.c.V) + page * st[0] + slot * st[2] + h * st[1];
            } else {
                to = a.dst[kind & 1] + t * a.dst_st[kind & 1][0] + h * a.dst_st[kind & 1][1];
            }
            raw[i].store(to, at0, at1);
            if (PAGED && kind == 1 && lane == 0) {
                const size_t o = ((size_t)place.y * a.c.heads + h) * a.c.rows + place.z;
                if (a.c.pos) a.c.pos[o] = place.w;
                if (a.c.mass) a.c.mass[o] = 0.f;
            }
            if (r + FLIGHT * a.per_token < all) ask(raw[i], r + FLIGHT * a.per_token);
        }
    }
}

bool rotary_ok(const ckv_rotary* r) {
    return r && r->rot >= 0 && r->rot <= D && r->rot % 16 == 0 && (r->rot == 0 || r->turns) && r->eps >= 0.f &&
           isfinite(r->eps) && isfinite(r->amplitude) && (r->interleaved == 0 || r->interleaved == 1);
}

// its arrays are read 16 bytes at a time
bool rotary_aligned(const ckv_rotary* r) { return aligned16(r->turns) && aligned16(r->q_weight) && aligned16(r->k_weight); }

// byte strides (token, head) of an operand; sources may stand still
ckv_status operand(const int64_t* st, int tokens, int heads, int elem, bool output, long long* out) {
    if (!st) return CKV_ERR_ARG;
    const int extent[2] = {tokens, heads};
    for (int i = 0; i < 2; ++i) {
        if (extent[i] <= 1) {
            out[i] = 0;  // never multiplied by more than 0
            continue;
        }
        if (st[i] < (output ? D : 0) || st[i] > MAX_STRIDE) return CKV_ERR_ARG;
        out[i] = (long long)st[i] * elem;
    }
    return ((out[0] | out[1]) & 15) ? CKV_ERR_ALIGN : CKV_OK;
}

// Rows of `width` bytes, n[0] tokens by n[1] heads, at byte strides st (where an
// extent is one its stride is 0, and the other way round).
struct Rows {
    const unsigned char* p;
    long long st[2];
    int n[2];
    long long width;
};
using Wide = __int128;  // extents times strides, whatever the arguments are
Rows rows_of(const void* p, const long long* st, int tokens, int heads, int elem) {
    return Rows{static_cast<const unsigned char*>(p), {st[0], st[1]}, {st[0] ? tokens : 1, st[1] ? heads : 1}, (long long)D * elem};
}
Rows array_of(const void* p, long long bytes) { return Rows{static_cast<const unsigned char*>(p), {0, 0}, {1, 1}, bytes}; }
// bytes from the first row along dimension i to the end of the last
Wide span(const Rows& r, int i) { return (Wide)(r.n[i] - 1) * r.st[i] + r.width; }
// whether some k in [lo, hi] has x - before < k step < x + behind
bool multiple_near(Wide x, Wide before, Wide behind, long long step, long long lo, long long hi) {
    if (step == 0) return x < before && -x < behind;
    const Wide from = x - before;
    Wide k = from / step - (from % step < 0) + 1;  // the first above x - before
    if (k < lo) k = lo;
    return k <= hi && k * step < x + behind;
}
// whether two of the rows overlap
bool rows_overlap(const Rows& r) {
    const int a = r.n[0] <= r.n[1] ? 0 : 1, b = 1 - a;
    const int inner = r.st[0] <= r.st[1] ? 0 : 1;
    if (r.n[1 - inner] == 1 || r.st[1 - inner] >= span(r, inner)) return r.n[inner] > 1 && r.st[inner] < r.width;
    if ((r.n[0] > 1 && r.st[0] < r.width) || (r.n[1] > 1 && r.st[1] < r.width)) return true;
    for (int i = 1; i < r.n[a]; ++i)
        if (multiple_near((Wide)i * r.st[a], r.width, r.width, r.st[b], 0, r.n[b] - 1)) return true;
    return false;
}
// Whether a row of x overlaps a row of y.  Rows side by side in one tensor are
// found apart by the first tests; what these leave is tried row by row, and taken
// to overlap where that would be long.
bool rows_meet(const Rows& x, const Rows& y) {
    const Wide apart = (Wide)(reinterpret_cast<uintptr_t>(y.p)) - (Wide)(reinterpret_cast<uintptr_t>(x.p));
    if (apart >= span(x, 0) + span(x, 1) - x.width || -apart >= span(y, 0) + span(y, 1) - y.width) return false;
    for (int i = 0; i < 2; ++i) {
        const long long step = x.st[i];
        if (step == 0 || step != y.st[i]) continue;
        // places modulo the step, which a stride of several steps does not change
        const Wide at = apart % step + (apart % step < 0 ? step : 0);
        const Wide long_x = x.st[1 - i] % step ? span(x, 1 - i) : x.width, long_y = y.st[1 - i] % step ? span(y, 1 - i) : y.width;
        if (at >= long_x && at + long_y <= step) return false;
    }
    // Numbers of a dimension come in by their difference where the strides are one,
    // else y's are gone through: heads h - g, then g, then tokens t - u, then u.
    auto one = [&](int i) { return x.n[i] == 1 || y.n[i] == 1 || x.st[i] == y.st[i]; };
    auto step = [&](int i) { return x.n[i] == 1 ? y.st[i] : x.st[i]; };
    auto least = [&](int i) { return one(i) ? 1 - (long long)y.n[i] : 0; };
    const int us = one(0) ? 1 : y.n[0], gs = one(1) ? 1 : y.n[1];
    if ((Wide)(x.n[1] - least(1)) * gs * us > 1 << 16) return true;
    for (int u = 0; u < us; ++u)
        for (int g = 0; g < gs; ++g)
            for (long long h = least(1); h < x.n[1]; ++h)
                if (multiple_near(apart + (Wide)u * y.st[0] + (Wide)g * y.st[1] - (Wide)h * step(1), x.width, y.width, step(0),
                                  least(0), x.n[0] - 1))
                    return true;
    return false;
}
// Whether outputs (out[i] is of the rows in[i], which it may be itself) overlap
// themselves, one another, another input or what the call reads besides.
template <int N, int M, int L>
bool outputs_overlap(const Rows (&out)[N], const Rows (&in)[M], const Rows (&read)[L]) {
    for (int i = 0; i < N; ++i) {
        if (!out[i].p) continue;
        if (rows_overlap(out[i])) return true;
        for (int j = 0; j < i; ++j)
            if (out[j].p && rows_meet(out[i], out[j])) return true;
        for (int j = 0; j < M; ++j)
            if (in[j].p && !(i == j && out[i].p == in[j].p) && rows_meet(out[i], in[j])) return true;
        for (int j = 0; j < L; ++j)
            if (read[j].p && rows_meet(out[i], read[j])) return true;
    }
    return false;
}

template <typename T, bool PAGED>
cudaError_t launch(RotArgs& a, cudaStream_t s) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int all = a.rows[0] + a.rows[1] + a.rows[2];
    // Lane groups to a token: few, so that one goes through 12 to 24 rows with the
    // angles of one token (32k tokens of 40 rows: 101 us with 20 rows to a group,
    // 107 with 10); more while there are fewer blocks than SMs, where latency counts.
    int per = 1;
    while (per < GROUPS && per * FLIGHT * 6 < all) per *= 2;
    while (per < GROUPS && per < all && (long long)a.tokens * per / GROUPS < sms) per *= 2;
    a.per_token = per;
    const int mine = GROUPS / per;
    const long long blocks = ((long long)a.tokens + mine - 1) / mine;
    return a.interleaved
               ? launch_dependent(rotary_kernel<T, PAGED, true>, dim3((unsigned)blocks), dim3(THREADS), 0, s, a)
               : launch_dependent(rotary_kernel<T, PAGED, false>, dim3((unsigned)blocks), dim3(THREADS), 0, s, a);
}

void take_rotary(const ckv_rotary* r, RotArgs* a) {
    a->turns = reinterpret_cast<const unsigned long long*>(r->turns);
    a->weight[0] = r->q_weight;
    a->weight[1] = r->k_weight;
    a->eps = r->eps;
    a->amplitude = r->amplitude;
    a->rot = r->rot;
    a->interleaved = r->interleaved;
}
constexpr long long MAX_ROWS = 0x7fff0000LL;

}  // namespace
}  // namespace paged
}  // namespace ckv

using namespace ckv;
using namespace ckv::paged;

extern "C" ckv_status ckv_rotate(const ckv_rotary* rotary, const void* q, const int64_t* q_stride, void* q_out,
                                 const int64_t* q_out_stride, int32_t heads_q, const void* k, const int64_t* k_stride,
                                 void* k_out, const int64_t* k_out_stride, int32_t heads_k, const int32_t* positions,
                                 int32_t tokens, int32_t d, int32_t dtype, void* stream) {
    CKV_TRACE("ckv_rotate");
    if (!rotary_ok(rotary) || d != D || tokens < 1 || heads_q < 0 || heads_k < 0 || (long long)heads_q + heads_k < 1 ||
        !positions)
        return CKV_ERR_ARG;
    if (dtype != CKV_F32 && dtype != CKV_BF16) return CKV_ERR_DTYPE;
    if (!rotary_aligned(rotary)) return CKV_ERR_ALIGN;
    if (((long long)heads_q + heads_k) * tokens > MAX_ROWS) return CKV_ERR_ARG;
    const int elem = dtype == CKV_BF16 ? 2 : 4;
    RotArgs a = {};
    take_rotary(rotary, &a);
    a.tokens = tokens;
    a.positions = positions;
    const void* src[2] = {q, k};
    void* dst[2] = {q_out, k_out};
    const int64_t *sst[2] = {q_stride, k_stride}, *dstst[2] = {q_out_stride, k_out_stride};
    a.rows[0] = heads_q;
    a.rows[1] = heads_k;
    for (int i = 0; i < 2; ++i) {
        if (a.rows[i] == 0) continue;
        if (!src[i] || !dst[i]) return CKV_ERR_ARG;
        ckv_status st = operand(sst[i], tokens, a.rows[i], elem, false, a.sst[i]);
        if (st == CKV_OK) st = operand(dstst[i], tokens, a.rows[i], elem, true, a.dst_st[i]);
        if (st != CKV_OK) return st;
        if (!aligned16(src[i]) || !aligned16(dst[i])) return CKV_ERR_ALIGN;
        if (src[i] == dst[i] && (a.sst[i][0] != a.dst_st[i][0] || a.sst[i][1] != a.dst_st[i][1])) return CKV_ERR_ARG;
        a.src[i] = static_cast<const unsigned char*>(src[i]);
        a.dst[i] = static_cast<unsigned char*>(dst[i]);
    }
    Rows out[2] = {}, in[2] = {};
    for (int i = 0; i < 2; ++i) {
        if (a.rows[i] == 0) continue;
        out[i] = rows_of(dst[i], a.dst_st[i], tokens, a.rows[i], elem);
        in[i] = rows_of(src[i], a.sst[i], tokens, a.rows[i], elem);
    }
    const Rows read[4] = {array_of(positions, 4LL * tokens), array_of(rotary->turns, 4LL * rotary->rot),
                          array_of(rotary->q_weight, 4 * D), array_of(rotary->k_weight, 4 * D)};
    if (outputs_overlap(out, in, read)) return CKV_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = elem == 2 ? launch<__nv_bfloat16, false>(a, s) : launch<float, false>(a, s);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}

extern "C" ckv_status ckv_paged_append_rotated(const ckv_paged_cache* cache, const ckv_rotary* rotary, const void* q,
                                               const int64_t* q_stride, int32_t g, void* q_out,
                                               const int64_t* q_out_stride, const void* k, const int64_t* k_stride,
                                               const void* v, const int64_t* v_stride, const int32_t* slots,
                                               int32_t tokens, void* stream) {
    CKV_TRACE("ckv_paged_append_rotated");
    RotArgs a = {};
    ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    a.slots_held = (long long)a.c.n_pages * a.c.page;
    if (!rotary_ok(rotary) || g < 0 || tokens < 1 || !k || !v || !slots || a.slots_held > 0x7fffffffLL ||
        (long long)a.c.heads * g > MAX_ROWS || ((long long)a.c.heads * g + 2LL * a.c.heads) * tokens > MAX_ROWS)
        return CKV_ERR_ARG;
    if (!rotary_aligned(rotary)) return CKV_ERR_ALIGN;
    const int elem = cache->kv_dtype == CKV_BF16 ? 2 : 4;
    take_rotary(rotary, &a);
    a.tokens = tokens;
    a.rows[0] = a.c.heads * g;
    a.rows[1] = a.rows[2] = a.c.heads;
    a.src[0] = static_cast<const unsigned char*>(q);
    a.src[1] = static_cast<const unsigned char*>(k);
    a.src[2] = static_cast<const unsigned char*>(v);
    a.dst[0] = static_cast<unsigned char*>(q_out);
    if (g > 0) {
        if (!q || !q_out) return CKV_ERR_ARG;
        st = operand(q_stride, tokens, a.rows[0], elem, false, a.sst[0]);
        if (st == CKV_OK) st = operand(q_out_stride, tokens, a.rows[0], elem, true, a.dst_st[0]);
        if (st != CKV_OK) return st;
        if (!aligned16(q) || !aligned16(q_out)) return CKV_ERR_ALIGN;
        if (q == q_out && (a.sst[0][0] != a.dst_st[0][0] || a.sst[0][1] != a.dst_st[0][1])) return CKV_ERR_ARG;
    }
    st = operand(k_stride, tokens, a.rows[1], elem, false, a.sst[1]);
    if (st == CKV_OK) st = operand(v_stride, tokens, a.rows[2], elem, false, a.sst[2]);
    if (st != CKV_OK) return st;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots)) return CKV_ERR_ALIGN;
    a.slots = reinterpret_cast<const int4*>(slots);
    if (g > 0) {
        const Rows out[1] = {rows_of(q_out, a.dst_st[0], tokens, a.rows[0], elem)};
        const Rows in[3] = {rows_of(q, a.sst[0], tokens, a.rows[0], elem), rows_of(k, a.sst[1], tokens, a.rows[1], elem),
                            rows_of(v, a.sst[2], tokens, a.rows[2], elem)};
        const Rows read[4] = {array_of(slots, 16LL * tokens), array_of(rotary->turns, 4LL * rotary->rot),
                              array_of(rotary->q_weight, 4 * D), array_of(rotary->k_weight, 4 * D)};
        if (outputs_overlap(out, in, read)) return CKV_ERR_ARG;
    }
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = elem == 2 ? launch<__nv_bfloat16, true>(a, s) : launch<float, true>(a, s);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
