// Decode attention of one new token per sequence over a paged cache.
//
//   s_jr = scale q_j . K_r,  lse_j = ln sum_r e^{s_jr},  o_j = sum_r e^{s_jr - lse_j} V_r
//
// for the g query heads j that share a KV head, over its rows r < lens[s].
// The rows are cut into blocks of SPLIT; a CTA computes one block's maximum,
// sum and weighted V (and, where the accumulated weights are wanted, leaves
// the scores in the workspace); the join merges the blocks of a (sequence, KV
// head) and a last kernel adds e^{s - lse} to the accumulated weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace ckv {
namespace paged {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int SPLIT = 256;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct AttnArgs {
    Cache c;
    const void* q;
    long long qst[2];  // element strides: sequence, query head
    int g;
    float qscale;  // scale * log2(e): scores are kept in base 2
    float* out;
    float* lse;
    const float* mass_in;
    float* mass_out;
    float* part;    // [units][splits][g][D + 2]
    float* scores;  // [units][g][rows], base 2
    float* lse2;    // [units][g]
    int splits;
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(w.x << 16);
    f[1] = __uint_as_float(w.x & 0xffff0000u);
    f[2] = __uint_as_float(w.y << 16);
    f[3] = __uint_as_float(w.y & 0xffff0000u);
}
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
}

template <typename T>
__global__ void __launch_bounds__(D) paged_attn_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ float sc[MAX_G][SPLIT];
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int u = blockIdx.x / a.splits, b = blockIdx.x % a.splits;
    const int s = u / a.c.heads, h = u % a.c.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (h == 0 && b == 0 && tid == 0) check_len(a.c, s);
    const int len = rows_held(a.c, s), r0 = b * SPLIT;
    if (r0 >= len) return;
    const int n = min(SPLIT, len - r0);
    for (int j = 0; j < a.g; ++j) {
        float q[4];
        load4(static_cast<const T*>(a.q) + s * a.qst[0] + (h * a.g + j) * a.qst[1] + 4 * lane, q);
        for (int i = warp; i < n; i += 4) {
            const int r = r0 + i, pg = page_of(a.c, s, r);
            float x = -INFINITY;
            if (pg >= 0) {
                float k[4];
                load4(reinterpret_cast<const T*>(a.c.K + pg * a.c.ks[0] + h * a.c.ks[1] + (r % a.c.page) * a.c.ks[2]) +
                          4 * lane, k);
                x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
                x *= a.qscale;
            }
            if (lane == 0) {
                sc[j][i] = x;
                if (a.scores) a.scores[((size_t)u * a.g + j) * a.c.rows + r] = x;
            }
        }
    }
    __syncthreads();
    float* pp = a.part + ((size_t)u * a.splits + b) * a.g * (D + 2);
    for (int j = warp; j < a.g; j += 4) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, sc[j][i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        const float ms = m == -INFINITY ? 0.f : m;
        for (int i = lane; i < n; i += 32) {
            const float p = exp2f(sc[j][i] - ms);
            sc[j][i] = p;
            l += p;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
        if (lane == 0) {
            pp[j * (D + 2) + D] = m;
            pp[j * (D + 2) + D + 1] = l;
        }
    }
    __syncthreads();
    float o[MAX_G];
#pragma unroll
    for (int j = 0; j < MAX_G; ++j) o[j] = 0.f;
    for (int i = 0; i < n; ++i) {
        const int r = r0 + i, pg = page_of(a.c, s, r);
        if (pg < 0) continue;
        const float v = static_cast<float>(
            reinterpret_cast<const T*>(a.c.V + pg * a.c.vs[0] + h * a.c.vs[1] + (r % a.c.page) * a.c.vs[2])[tid]);
#pragma unroll
        for (int j = 0; j < MAX_G; ++j)
            if (j < a.g) o[j] += sc[j][i] * v;
    }
#pragma unroll
    for (int j = 0; j < MAX_G; ++j)
        if (j < a.g) pp[j * (D + 2) + tid] = o[j];
}

__global__ void __launch_bounds__(D) paged_join_kernel(const __grid_constant__ AttnArgs a) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int u = blockIdx.x / a.g, j = blockIdx.x % a.g, tid = threadIdx.x;
    const int len = rows_held(a.c, u / a.c.heads);
    const int ns = (len + SPLIT - 1) / SPLIT;
    const float* pp = a.part + ((size_t)u * a.splits * a.g + j) * (D + 2);
    const size_t step = (size_t)a.g * (D + 2);
    float m = -INFINITY;
    for (int i = 0; i < ns; ++i) m = fmaxf(m, pp[i * step + D]);
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f, o = 0.f;
    for (int i = 0; i < ns; ++i) {
        const float w = exp2f(pp[i * step + D] - ms);
        l += w * pp[i * step + D + 1];
        o += w * pp[i * step + tid];
    }
    a.out[((size_t)u * a.g + j) * D + tid] = l > 0.f ? o / l : (l == 0.f ? 0.f : l);
    if (tid == 0) {
        const float x = l == 0.f ? -INFINITY : ms + log2f(l);
        if (a.lse) a.lse[(size_t)u * a.g + j] = x * LN2;
        a.lse2[(size_t)u * a.g + j] = x;
    }
}

__global__ void __launch_bounds__(256) paged_mass_kernel(const __grid_constant__ AttnArgs a, int blocks) {
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int u = blockIdx.x / blocks, b = blockIdx.x % blocks;
    const int len = rows_held(a.c, u / a.c.heads);
    for (int r = b * 256 + threadIdx.x; r < len; r += blocks * 256) {
        float w = 0.f;
        for (int j = 0; j < a.g; ++j) {
            const float x = a.scores[((size_t)u * a.g + j) * a.c.rows + r], z = a.lse2[(size_t)u * a.g + j];
            w += z == -INFINITY ? 0.f : exp2f(x - z);
        }
        const size_t o = (size_t)u * a.c.rows + r;
        a.mass_out[o] = (a.mass_in ? a.mass_in[o] : 0.f) + w;
    }
}

struct Layout {
    int splits;
    size_t part, lse2, scores, total;  // byte offsets
};
Layout layout_of(const Cache& c, int g, bool with_mass) {
    Layout l;
    const size_t units = (size_t)c.seqs * c.heads;
    l.splits = ceil_div(c.rows, SPLIT);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.part = 0;
    l.lse2 = up(units * l.splits * g * (D + 2) * sizeof(float));
    l.scores = l.lse2 + up(units * g * sizeof(float));
    l.total = l.scores + (with_mass ? up(units * g * (size_t)c.rows * sizeof(float)) : 0);
    return l;
}

}  // namespace
}  // namespace paged
}  // namespace ckv

using namespace ckv;
using namespace ckv::paged;

extern "C" ckv_status ckv_paged_attn_workspace(const ckv_paged_cache* cache, int32_t g, int32_t with_mass,
                                               int64_t* bytes) {
    Cache c;
    const ckv_status st = check_cache(cache, &c);
    if (st != CKV_OK) return st;
    if (!bytes || g < 1 || g > MAX_G) return CKV_ERR_ARG;
    *bytes = (int64_t)layout_of(c, g, with_mass != 0).total;
    return CKV_OK;
}

extern "C" ckv_status ckv_paged_decode_attn(const ckv_paged_cache* cache, const void* q, int32_t q_dtype,
                                            const int64_t* q_stride, int32_t g, float scale, float* out, float* lse,
                                            const float* mass_in, float* mass_out, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
    CKV_TRACE("ckv_paged_decode_attn");
    AttnArgs a;
    const ckv_status st = check_cache(cache, &a.c);
    if (st != CKV_OK) return st;
    if (!q || !q_stride || !out || !workspace) return CKV_ERR_ARG;
    if (q_dtype != cache->kv_dtype) return CKV_ERR_DTYPE;
    if (g < 1 || g > MAX_G || !isfinite(scale) || (mass_in && !mass_out)) return CKV_ERR_ARG;
    const int elem = q_dtype == CKV_BF16 ? 2 : 4;
    for (int i = 0; i < 2; ++i) {
        if (q_stride[i] < 0 || q_stride[i] > (1LL << 38)) return CKV_ERR_ARG;
        if (q_stride[i] * elem & 15) return CKV_ERR_ALIGN;
        a.qst[i] = q_stride[i];
    }
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return CKV_ERR_ALIGN;
    const Layout l = layout_of(a.c, g, mass_out != nullptr);
    if (workspace_bytes < (int64_t)l.total) return CKV_ERR_CAPACITY;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    a.q = q;
    a.g = g;
    a.qscale = scale * LOG2E;
    a.out = out;
    a.lse = lse;
    a.mass_in = mass_in;
    a.mass_out = mass_out;
    a.part = reinterpret_cast<float*>(w + l.part);
    a.lse2 = reinterpret_cast<float*>(w + l.lse2);
    a.scores = mass_out ? reinterpret_cast<float*>(w + l.scores) : nullptr;
    a.splits = l.splits;
    const long long units = (long long)a.c.seqs * a.c.heads;
    if (units * l.splits > 0x7fffffffLL || units * g > 0x7fffffffLL) return CKV_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)(units * l.splits));
    cudaError_t e = q_dtype == CKV_BF16 ? launch_dependent(paged_attn_kernel<__nv_bfloat16>, grid, dim3(D), 0, s, a)
                                        : launch_dependent(paged_attn_kernel<float>, grid, dim3(D), 0, s, a);
    if (e == cudaSuccess) e = launch_dependent(paged_join_kernel, dim3((unsigned)(units * g)), dim3(D), 0, s, a);
    if (e == cudaSuccess && mass_out) {
        const int blocks = ceil_div(a.c.rows, 4096);
        e = launch_dependent(paged_mass_kernel, dim3((unsigned)(units * blocks)), dim3(256), 0, s, a, blocks);
    }
    return e == cudaSuccess ? CKV_OK : CKV_ERR_CUDA;
}
