// mq_paged_plan.cu -- the page plan of a serving step: which pages of the KV
// cache the step's new tokens take, and the cache slot of each of them.
//
//   cu[b + 1]        = min(T, sum_{i <= b} new_i)           (rows of the batch)
//   held_b           = ceil(ctx_b / ps),  need_b = ceil((ctx_b + n_b) / ps) - held_b
//   table[b][held_b + j] = free[sum_{i < b} need_i + j]       (j < need_b)
//   slot(t)          = table[b][pos / ps] * ps + pos % ps,  pos = ctx_b + t - cu[b]
//
// At most about 1 MB is read and written, so the launch is what it costs.  One
// kernel does it all: every block takes both prefix sums over the requests by
// itself (the lengths are a few KB, in L2 after the first block) and keeps
// them in shared memory, then fills its own token rows, so no block waits for
// another.  A new page's table entry is written by the thread of the page's
// first token.
#include <algorithm>

#include "mq_internal.h"

namespace mq {

namespace {

constexpr int kPlanThreads = 512;

struct PlanParams {
    const int *ctx, *nw, *free_pages;
    int *table, *cu, *info;
    int64_t *slots;
    int B, T, n_free, max_pages, ps_shift;
};

// Exclusive prefix sum of one value per thread over the block; *total gets the
// sum.  red: one value per warp plus the total.
__device__ __forceinline__ int64_t block_exclusive_scan(int64_t v, int64_t *red, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t s = lane < kPlanThreads / 32 ? red[lane] : 0;
#pragma unroll
        for (int o = 1; o < kPlanThreads / 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < kPlanThreads / 32) red[lane] = s;
    }
    __syncthreads();
    *total = red[kPlanThreads / 32 - 1];
    const int64_t r = x - v + (warp ? red[warp - 1] : 0);
    __syncthreads();           // red may be written again
    return r;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p) {
    extern __shared__ int psm[];
    int *ctx_s = psm;                 // [B] cached tokens
    int *cu_s = ctx_s + p.B;          // [B + 1] first: new tokens asked; then the clipped prefix
    int *base_s = cu_s + p.B + 1;     // [B] new pages of the requests before
    __shared__ int64_t red[kPlanThreads / 32];
    __shared__ int lost_s, longest_s;
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    for (int b = tid; b < p.B; b += kPlanThreads) {
        ctx_s[b] = max(p.ctx[b], 0);
        cu_s[b] = max(p.nw[b], 0);
    }
    if (tid == 0) {
        lost_s = 0;
        longest_s = 0;
    }
    __syncthreads();
    // each thread owns a run of consecutive requests
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int64_t sum = 0, asked;
    for (int b = b0; b < b1; ++b) sum += cu_s[b];
    int64_t at = block_exclusive_scan(sum, red, &asked);
    const int ps = 1 << p.ps_shift;
    int64_t need = 0, pages;
    int longest = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t lo = min(at, static_cast<int64_t>(p.T));
        at += cu_s[b];
        cu_s[b] = static_cast<int>(lo);
        const int64_t end = ctx_s[b] + (min(at, static_cast<int64_t>(p.T)) - lo);
        longest = max(longest, static_cast<int>(min(end, static_cast<int64_t>(INT32_MAX))));
        const int64_t held = min((static_cast<int64_t>(ctx_s[b]) + ps - 1) >> p.ps_shift,
                                 static_cast<int64_t>(p.max_pages));
        const int64_t all = min((end + ps - 1) >> p.ps_shift, static_cast<int64_t>(p.max_pages));
        base_s[b] = static_cast<int>(all - held);
        need += all - held;
    }
    if (tid == 0) cu_s[p.B] = static_cast<int>(min(asked, static_cast<int64_t>(p.T)));
    int64_t pbase = block_exclusive_scan(need, red, &pages);
    for (int b = b0; b < b1; ++b) {
        const int n = base_s[b];
        base_s[b] = static_cast<int>(pbase);
        pbase += n;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        // the prefix of rows, and what the caller has to know of the step
        int lost = 0;
        for (int b = b0; b < b1; ++b) {
            const int64_t ctx = ctx_s[b], end = ctx + (cu_s[b + 1] - cu_s[b]);
            const int64_t held = min((ctx + ps - 1) >> p.ps_shift, static_cast<int64_t>(p.max_pages));
            const int64_t all = min((end + ps - 1) >> p.ps_shift, static_cast<int64_t>(p.max_pages));
            const int64_t got = min(all - held, max(static_cast<int64_t>(p.n_free) - base_s[b], static_cast<int64_t>(0)));
            lost += static_cast<int>(end - min(end, max(ctx, (held + got) << p.ps_shift)));
        }
        if (lost) atomicAdd(&lost_s, lost);
        atomicMax(&longest_s, longest);
        for (int b = tid; b <= p.B; b += kPlanThreads) p.cu[b] = cu_s[b];
        __syncthreads();
        if (tid == 0) {
            const int64_t cap = INT32_MAX;
            p.info[0] = static_cast<int>(min(asked, cap));
            p.info[1] = static_cast<int>(min(pages, cap));
            p.info[2] = static_cast<int>(min(asked - cu_s[p.B] + lost_s, cap));
            p.info[3] = longest_s;
        }
    }
    const int total = cu_s[p.B];
    for (int t = blockIdx.x * kPlanThreads + tid; t < p.T; t += gridDim.x * kPlanThreads) {
        int64_t slot = -1;
        if (t < total) {
            int lo = 0, hi = p.B;          // the last request with cu[b] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu_s[mid] <= t) lo = mid; else hi = mid;
            }
            const int64_t pos = static_cast<int64_t>(ctx_s[lo]) + (t - cu_s[lo]);
            const int64_t page = pos >> p.ps_shift, off = pos & (ps - 1);
            if (page < p.max_pages) {
                const int64_t held = (static_cast<int64_t>(ctx_s[lo]) + ps - 1) >> p.ps_shift;
                int *entry = p.table + static_cast<int64_t>(lo) * p.max_pages + page;
                int id;
                if (page >= held) {
                    const int64_t k = base_s[lo] + (page - held);
                    id = k < p.n_free ? p.free_pages[k] : -1;
                    if (off == 0) *entry = id;
                } else {
                    id = *entry;
                }
                if (id >= 0) slot = (static_cast<int64_t>(id) << p.ps_shift) + off;
            }
        }
        p.slots[t] = slot;
    }
}

}  // namespace

cudaError_t launch_paged_plan(const int *ctx, const int *nw, int64_t B, int64_t page_size, const int *free_pages,
                              int64_t n_free, int *table, int64_t max_pages, int64_t T, int *cu, int64_t *slots,
                              int *info, int num_sms, cudaStream_t s) {
    PlanParams p;
    p.ctx = ctx;
    p.nw = nw;
    p.free_pages = free_pages;
    p.table = table;
    p.cu = cu;
    p.info = info;
    p.slots = slots;
    p.B = static_cast<int>(B);
    p.T = static_cast<int>(T);
    p.n_free = static_cast<int>(n_free);
    p.max_pages = static_cast<int>(max_pages);
    p.ps_shift = 0;
    while ((1 << p.ps_shift) < page_size) ++p.ps_shift;
    const size_t smem = (3 * static_cast<size_t>(B) + 1) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(std::max<size_t>(smem, 48 * 1024)));
    if (e != cudaSuccess) return e;
    const int64_t want = (T + kPlanThreads - 1) / kPlanThreads;
    const int grid = static_cast<int>(std::min<int64_t>(want, num_sms));
    e = launch_pdl(paged_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mq
