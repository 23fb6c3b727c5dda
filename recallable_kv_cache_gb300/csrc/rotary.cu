// Norms and rotary positions of queries and keys, in one pass: on their own
// (ckv_rotate) or with the keys and values going into a paged cache
// (ckv_paged_append_rotated).
//
//   y = x w / sqrt(mean x^2 + eps),  (y_a, y_b) := A (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//
// Every row is read and written once, so long inputs are bound by HBM.  What a
// row costs besides is kept small: sixteen lanes have a row, eight channels a
// lane (16 bytes of bf16), the sum of squares and the other half of a pair come
// by shuffles, and the angles of a token are worked out once for all its heads:
// the block leaves cos and sin in shared memory, and a lane keeps those of its
// channels in registers while it goes through rows of one token.
//
// The angle of pair i at position p is p turns_i / 2^64 of a turn: the product of
// two integers, whose wrap at 2^64 is the angle's own, so that the angle is as
// exact at position 10^9 as at 1 (p w_i in fp32 would be off by 0.06 at 10^6).
// The quarter turn nearest to it is taken off before the sine is looked up.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

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

template <typename T>
struct Raw;  // eight channels as they are in memory
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const unsigned char* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(unsigned char* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const unsigned char* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(unsigned char* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// A block has GROUPS / per_token tokens, a lane group every per_token-th row of
// its token: queries, then keys, then values (PAGED).
template <typename T, bool PAGED, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const __grid_constant__ RotArgs a) {
    constexpr int CS = INTERLEAVED ? 4 : 8;  // pairs that a lane has channels of
    constexpr int ROW = 8 * sizeof(T);       // bytes of a lane's channels
    extern __shared__ float2 turned[];       // [tokens of the block][rot / 2]
    __shared__ __align__(16) float weight[2][D];
    const int tid = threadIdx.x, lane = tid & (LANES - 1), group = tid / LANES;
    const int half = a.rot / 2;
    const int mine = GROUPS / a.per_token;  // tokens of a block
    const long long t0 = (long long)blockIdx.x * mine;
    const int local = group / a.per_token, sub = group % a.per_token;
    const long long t = t0 + local;
    const int all = a.rows[0] + a.rows[1] + a.rows[2];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    int4 place = make_int4(0, 0, 0, 0);
    bool live = t < a.tokens;
    if (PAGED && live) {
        place = a.slots[t];
        live = place.x != -1;
        const bool bad = place.x < -1 || place.x >= a.slots_held ||
                         ((a.c.pos || a.c.mass) && (place.y < 0 || place.y >= a.c.seqs || place.z < 0 || place.z >= a.c.rows));
        if (live && bad) {
            if (lane == 0 && sub == 0) report(a.c.dev_err, CKV_DEV_BAD_INDEX);
            live = false;
        }
    }
    // row r of the token: which of q, k, v, and its head
    auto kind_of = [&](int r, int* h) {
        const int kind = (r >= a.rows[0]) + (r >= a.rows[0] + a.rows[1]);
        *h = r - (kind > 0 ? a.rows[0] : 0) - (kind > 1 ? a.rows[1] : 0);
        return kind;
    };
    Raw<T> raw[FLIGHT];
    auto ask = [&](int r0) {
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            const int r = r0 + i * a.per_token;
            if (live && r < all) {
                int h;
                const int kind = kind_of(r, &h);
                raw[i].load(a.src[kind] + t * a.sst[kind][0] + h * a.sst[kind][1] + lane * ROW);
            }
        }
    };
    ask(sub);
    // the angles, and the weights
    for (int i = tid; i < 2 * D; i += THREADS) {
        const float* w = a.weight[i / D];
        weight[i / D][i % D] = w ? w[i % D] : 1.f;
    }
    for (int i = tid; i < mine * half; i += THREADS) {
        const int token = i / half, pair = i - token * half;
        float2 cs = make_float2(0.f, 0.f);
        if (t0 + token < a.tokens) {
            const int p = PAGED ? a.slots[t0 + token].w : a.positions[t0 + token];
            cs = unit_circle((unsigned long long)(long long)p * a.turns[pair]);
        }
        turned[i] = make_float2(cs.x * a.amplitude, cs.y * a.amplitude);
    }
    __syncthreads();
    // this lane's pairs; channels from rot on keep their value
    float c[CS], s[CS];
    const int reach = a.rot / 8;  // lanes that have rotated channels
    const bool turns = lane < reach;
    // the other channel of a pair is `reach / 2` lanes on or back
    const bool low = lane < reach / 2;
    const int other = INTERLEAVED || !turns ? lane : (low ? lane + reach / 2 : lane - reach / 2);
#pragma unroll
    for (int i = 0; i < CS; ++i) {
        const int pair = INTERLEAVED ? lane * 4 + i : (low ? lane : lane - reach / 2) * 8 + i;
        const float2 cs = turns ? turned[local * half + pair] : make_float2(1.f, 0.f);
        c[i] = cs.x;
        s[i] = INTERLEAVED || !low ? cs.y : -cs.y;
    }
    const int page = PAGED && live ? a.c.by_page.quot(place.x, &place.x) : 0;
    // the two groups of a warp may be at rows of different kinds
    const unsigned half_warp = 0xffffu << (tid & LANES);
    for (int r0 = sub; r0 < all; r0 += FLIGHT * a.per_token) {
        if (r0 != sub) ask(r0);
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            const int r = r0 + i * a.per_token;
            int h;
            const int kind = kind_of(r, &h);
            const bool there = live && r < all;
            if (!PAGED || kind < 2) {
                float x[8];
                raw[i].get(x);
                if (a.weight[kind & 1]) {
                    float sq = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(half_warp, sq, o, LANES);
                    const float scale = rsqrtf(sq * (1.f / D) + a.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= scale * weight[kind & 1][8 * lane + e];
                }
                if (INTERLEAVED) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float u = x[2 * e], v = x[2 * e + 1];
                        x[2 * e] = turns ? u * c[e] - v * s[e] : u;
                        x[2 * e + 1] = turns ? v * c[e] + u * s[e] : v;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = __shfl_sync(half_warp, x[e], other, LANES);
                        x[e] = turns ? x[e] * c[e] + y * s[e] : x[e];
                    }
                }
                raw[i].put(x);
            }
            if (!there) continue;
            unsigned char* to;
            if (PAGED && kind > 0) {
                const long long* st = kind == 1 ? a.c.ks : a.c.vs;
                to = (kind == 1 ? a.c.K : a.c.V) + page * st[0] + h * st[1] + place.x * st[2];
                if (kind == 1 && lane == 0) {
                    const size_t o = ((size_t)place.y * a.c.heads + h) * a.c.rows + place.z;
                    if (a.c.pos) a.c.pos[o] = place.w;
                    if (a.c.mass) a.c.mass[o] = 0.f;
                }
            } else {
                to = a.dst[kind & 1] + t * a.dst_st[kind & 1][0] + h * a.dst_st[kind & 1][1];
            }
            raw[i].store(to + lane * ROW);
        }
    }
}

bool rotary_ok(const ckv_rotary* r) {
    return r && r->rot >= 0 && r->rot <= D && r->rot % 16 == 0 && (r->rot == 0 || r->turns) && r->eps >= 0.f &&
           isfinite(r->eps) && isfinite(r->amplitude) && (r->interleaved == 0 || r->interleaved == 1);
}

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

template <typename T, bool PAGED>
cudaError_t launch(RotArgs& a, cudaStream_t s) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int all = a.rows[0] + a.rows[1] + a.rows[2];
    // Lane groups to a token: enough that one has FLIGHT rows at a time and no
    // more than a few turns of them, as the angles cost as much as some ten rows;
    // more while there are fewer blocks than SMs, where latency counts.
    int per = 1;
    while (per < GROUPS && per * FLIGHT * 3 < all) per *= 2;
    while (per < GROUPS && per < all && (long long)a.tokens * per / GROUPS < sms) per *= 2;
    a.per_token = per;
    const int mine = GROUPS / per;
    const long long blocks = ((long long)a.tokens + mine - 1) / mine;
    const size_t smem = (size_t)mine * (a.rot / 2) * sizeof(float2);
    return a.interleaved
               ? launch_dependent(rotary_kernel<T, PAGED, true>, dim3((unsigned)blocks), dim3(THREADS), smem, s, a)
               : launch_dependent(rotary_kernel<T, PAGED, false>, dim3((unsigned)blocks), dim3(THREADS), smem, s, a);
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
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = elem == 2 ? launch<__nv_bfloat16, true>(a, s) : launch<float, true>(a, s);
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
