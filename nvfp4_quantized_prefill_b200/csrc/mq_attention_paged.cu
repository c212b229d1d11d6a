// mq_attention_paged.cu -- attention of a serving step over many sequences at
// once: packed prompts (keys and values in the batch itself) and new tokens
// over a paged KV cache.
//
//   o[t, h, :] = sum_{j <= pos(t)} softmax_j( q[t,h,:] . k[j,g,:] / sqrt(D) ) v[j,g,:],
//   g = h / (H / Hkv), j over the positions of t's own sequence.
//
// One warp per (token, query head): each lane holds four of the 128
// dimensions, keys are taken one after the other with a running maximum and
// sum in FP32.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "mq_internal.h"
#include "mq_ptx.cuh"

namespace mq {

namespace {

constexpr int kD = 128;
// log2(e) / sqrt(128): scores in the base-2 exponent domain
constexpr float kScaleLog2 = 0.12751743082459868f;

__device__ __forceinline__ int seq_of(const int *cu, int B, int t) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
}

// The new tokens' K and V rows to their slots (one warp per token and KV head:
// 16 lanes for K, 16 for V).
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedAttnArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t n_slots = p.n_pages << p.ps_shift;
    const int64_t total = static_cast<int64_t>(min(p.T, p.cu[p.B])) * p.Hkv;
    const int lane = threadIdx.x & 31;
    for (int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < total;
         w += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
        const int64_t t = w / p.Hkv, g = w % p.Hkv;
        const int64_t slot = p.slots[t];
        if (slot < 0 || slot >= n_slots) continue;
        const int64_t dst = ((((slot >> p.ps_shift) * p.Hkv + g) << p.ps_shift) + (slot & ((1 << p.ps_shift) - 1))) * kD;
        const __nv_bfloat16 *row = p.qkv + t * p.ldqkv + (p.H + g) * kD + (lane < 16 ? 0 : p.Hkv * kD);
        reinterpret_cast<uint4 *>((lane < 16 ? p.k_pages : p.v_pages) + dst)[lane & 15] =
            reinterpret_cast<const uint4 *>(row)[lane & 15];
    }
}

__global__ void __launch_bounds__(256) paged_rows_kernel(const PagedAttnArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int total = max(min(p.T, p.cu[p.B]), 0);
    const int group = p.H / p.Hkv, ps = 1 << p.ps_shift;
    float amax = 0.0f;
    for (int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         w < static_cast<int64_t>(total) * p.H; w += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
        const int t = static_cast<int>(w / p.H), h = static_cast<int>(w % p.H), g = h / group;
        const int b = seq_of(p.cu, p.B, t);
        const int start = max(p.cu[b], 0);
        int64_t n = t - start + 1;           // keys of this row
        if (p.table) n = min(n + max(p.ctx[b], 0), static_cast<int64_t>(p.max_pages) << p.ps_shift);
        const float4 q = load4(p.qkv + t * p.ldqkv + h * kD + lane * 4);
        float m = -INFINITY, l = 0.0f, a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t j = 0; j < n; ++j) {
            const __nv_bfloat16 *k, *v;
            if (p.table) {
                const int id = p.table[static_cast<int64_t>(b) * p.max_pages + (j >> p.ps_shift)];
                if (id < 0 || id >= p.n_pages) continue;
                const int64_t off = (((static_cast<int64_t>(id) * p.Hkv + g) << p.ps_shift) + (j & (ps - 1))) * kD;
                k = p.k_pages + off;
                v = p.v_pages + off;
            } else {
                k = p.qkv + (start + j) * p.ldqkv + (p.H + g) * kD;
                v = k + p.Hkv * kD;
            }
            const float4 kk = load4(k + lane * 4);
            float s = q.x * kk.x + q.y * kk.y + q.z * kk.z + q.w * kk.w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            s *= kScaleLog2;
            const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
            const float4 vv = load4(v + lane * 4);
            l = l * f + e;
            a[0] = a[0] * f + e * vv.x;
            a[1] = a[1] * f + e * vv.y;
            a[2] = a[2] * f + e * vv.z;
            a[3] = a[3] * f + e * vv.w;
            m = mn;
        }
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // a row without keys: zeros; NaN stays
        __nv_bfloat162 r[2] = {__floats2bfloat162_rn(a[0] * inv, a[1] * inv), __floats2bfloat162_rn(a[2] * inv, a[3] * inv)};
        *reinterpret_cast<uint2 *>(p.o + t * p.ldo + h * kD + lane * 4) = *reinterpret_cast<uint2 *>(r);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(__bfloat162float(r[i].x)), fabsf(__bfloat162float(r[i].y))));
    }
    if (p.o_amax) {
        const unsigned u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));
        if (lane == 0 && u) atomicMax(reinterpret_cast<unsigned *>(p.o_amax), u);
    }
}

}  // namespace

size_t attention_paged_workspace_bytes(int64_t T, int64_t B, int64_t max_new, int64_t H, int64_t Hkv, bool paged) {
    return 256;
}

cudaError_t launch_attention_paged(const PagedAttnArgs &a, void *ws, unsigned *err, int num_sms, cudaStream_t s) {
    cudaError_t e;
    if (a.o_amax && (e = cudaMemsetAsync(a.o_amax, 0, sizeof(float), s)) != cudaSuccess) return e;
    if (a.slots && (e = launch_pdl(paged_append_kernel, dim3(4 * num_sms), dim3(256), 0, s, a)) != cudaSuccess) return e;
    const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(a.T) * a.H + 7) / 8, 1 << 16);
    e = launch_pdl(paged_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mq
