// mq_paged_plan.cu -- the page plan of a serving step: which pages of the KV
// cache the step's new tokens take, and the cache slot of each of them.
//
//   cu[b + 1]        = min(T, sum_{i <= b} new_i)           (rows of the batch)
//   held_b           = ceil(ctx_b / ps),  need_b = ceil((ctx_b + n_b) / ps) - held_b
//   table[b][held_b + j] = free[sum_{i < b} need_i + j]       (j < need_b)
//   slot(t)          = table[b][pos / ps] * ps + pos % ps,  pos = ctx_b + t - cu[b]
//
// 8 bytes are written per row and little else is moved (1.0 MB for 4096 requests
// with 114009 rows), so the launch is what it costs.  One kernel does it all:
// every block takes both prefix sums over the requests by itself (the lengths are
// a few KB, in L2 after the first block; a thread keeps its run of consecutive
// requests in registers) and leaves them in shared memory, then fills its own
// token rows, so no block waits for another.  Where there are several, the first
// block fills none: it looks for negative ids in the table and the free list and
// counts the tokens without a slot (16 loads a thread in flight: with 4, 262144
// pages of one step took it 86 us, twice the others' time).  A new page's table
// entry is written by the thread of the page's first token.
// Measured, us a call among 40 in a graph: 2.3 for 8 requests, 3.5 for 257, 6.9
// for 4096 with 114009 rows, 34 for 16384, 43 for 2.1 million rows in pages of 8.
#include <algorithm>

#include "mq_internal.h"

namespace mq {

namespace {

struct PlanParams {
    const int *ctx, *nw, *free_pages;
    int *table, *cu, *info;
    int64_t *slots;
    int B, T, n_free, max_pages, ps_shift;
};

// Exclusive prefix sums of two values per thread over the block, and the totals.
template <int kThreads>
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t (*red)[kThreads / 32], int64_t &total_a,
                                            int64_t &total_b) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) {
        red[0][warp] = x;
        red[1][warp] = y;
    }
    __syncthreads();
    if (warp < 2) {
        int64_t s = lane < kWarps ? red[warp][lane] : 0;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += u;
        }
        if (lane < kWarps) red[warp][lane] = s;
    }
    __syncthreads();
    total_a = red[0][kWarps - 1];
    total_b = red[1][kWarps - 1];
    a = x - a + (warp ? red[0][warp - 1] : 0);
    b = y - b + (warp ? red[1][warp - 1] : 0);
    __syncthreads();           // red may be written again
}

// kPer: consecutive requests a thread holds (kThreads x kPer >= B)
template <int kThreads, int kPer>
__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PlanParams p) {
    extern __shared__ int psm[];
    int *ctx_s = psm;                 // [B] cached tokens
    int *base_s = ctx_s + p.B;        // [B] new pages of the requests before
    int *cu_s = base_s + p.B;         // [B + 1] first row
    __shared__ int64_t red[2][kThreads / 32];
    __shared__ int lost_s, longest_s;
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    const int b0 = min(tid * kPer, p.B), nb = min(kPer, p.B - b0);
    const int ps = 1 << p.ps_shift;
    const int64_t T = p.T;
    int ctx[kPer], nw[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        ctx[i] = i < nb ? max(p.ctx[b0 + i], 0) : 0;
        nw[i] = i < nb ? max(p.nw[b0 + i], 0) : 0;
    }
    if (tid == 0) {
        lost_s = 0;
        longest_s = 0;
    }
    // (unsigned 32 bits hold a length cut at T: below 2^31 + 2^22)
    const unsigned most = p.max_pages;
    auto pages_of = [&](unsigned n) { return (n + ps - 1) >> p.ps_shift; };
    auto pages_to = [&](unsigned n) { return min(pages_of(n), most); };         // that a table row can hold
    // both sums at once, as if no row were cut at T; the pages again if some are
    int64_t at = 0, base = 0, asked, pages;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        at += nw[i];
        base += pages_to(static_cast<unsigned>(ctx[i]) + nw[i]) - pages_to(ctx[i]);
    }
    block_scan2<kThreads>(at, base, red, asked, pages);
    if (asked > T) {
        int64_t a = at, none = 0, zero;
        base = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int lo = static_cast<int>(min(a, T)), hi = static_cast<int>(min(a + nw[i], T));
            a += nw[i];
            base += pages_to(static_cast<unsigned>(ctx[i]) + (hi - lo)) - pages_to(ctx[i]);
        }
        block_scan2<kThreads>(none, base, red, zero, pages);
    }
    // tokens past the pages that a request has and gets have no slot
    int lost = 0;
    unsigned longest = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= nb) break;
        const int lo = static_cast<int>(min(at, T)), hi = static_cast<int>(min(at + nw[i], T));
        const unsigned c = ctx[i], end = c + (hi - lo), held = pages_to(c), need = pages_to(end) - held;
        ctx_s[b0 + i] = ctx[i];
        cu_s[b0 + i] = lo;
        base_s[b0 + i] = static_cast<int>(base);
        const unsigned have = held + static_cast<unsigned>(min(static_cast<int64_t>(need), max(p.n_free - base, static_cast<int64_t>(0))));
        if (have < pages_of(end)) lost += end - max(c, have << p.ps_shift);
        base += need;
        at += nw[i];
        longest = max(longest, end);
    }
    if (tid == 0) cu_s[p.B] = static_cast<int>(min(asked, T));
    __syncthreads();
    if (blockIdx.x == 0) {
        // the prefix of rows, and what the caller has to know of the step: also
        // without a slot are tokens whose page has a negative id, in the table
        // (the last page held, if it is not full) or in the free list
        constexpr int kFlight = 16;            // loads in flight
        for (int j0 = tid; j0 < p.B; j0 += kFlight * kThreads) {
            int id[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int b = j0 + u * kThreads;
                id[u] = 0;
                if (u < kPer && b < p.B) {
                    const unsigned c = ctx_s[b], page = c >> p.ps_shift;
                    if (cu_s[b + 1] > cu_s[b] && (c & (ps - 1)) && page < most) id[u] = p.table[static_cast<int64_t>(b) * most + page];
                }
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (id[u] < 0) {
                    const int b = j0 + u * kThreads;
                    lost += min(cu_s[b + 1] - cu_s[b], ps - (ctx_s[b] & (ps - 1)));
                }
        }
        const int taken = static_cast<int>(min(pages, static_cast<int64_t>(p.n_free)));
        for (int k0 = tid; k0 < taken; k0 += kFlight * kThreads) {
            int id[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) id[u] = u * kThreads < taken - k0 ? p.free_pages[k0 + u * kThreads] : 0;
            unsigned neg = 0;
#pragma unroll
            for (int u = 0; u < kFlight; ++u) neg |= (id[u] < 0 ? 1u : 0u) << u;
            for (; neg; neg &= neg - 1) {
                const int k = k0 + (__ffs(neg) - 1) * kThreads;
                int lo = 0, hi = p.B;          // the last request with base[b] <= k
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (base_s[mid] <= k) lo = mid; else hi = mid;
                }
                const unsigned end = static_cast<unsigned>(ctx_s[lo]) + (cu_s[lo + 1] - cu_s[lo]);
                const unsigned start = (pages_to(ctx_s[lo]) + (k - base_s[lo])) << p.ps_shift;
                lost += min(end - start, static_cast<unsigned>(ps));
            }
        }
        if (lost) atomicAdd(&lost_s, lost);
        atomicMax(&longest_s, static_cast<int>(min(longest, static_cast<unsigned>(INT32_MAX))));
        for (int b = tid; b <= p.B; b += kThreads) p.cu[b] = cu_s[b];
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
    const int first = gridDim.x > 1 ? 1 : 0;       // block 0 only counts where there are others to fill the rows
    if (static_cast<int>(blockIdx.x) < first) return;
    for (int t = (blockIdx.x - first) * kThreads + tid; t < p.T; t += (gridDim.x - first) * kThreads) {
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

template <int kThreads, int kPer>
cudaError_t launch_plan(const PlanParams &p, int num_sms, cudaStream_t s) {
    const size_t smem = (3 * static_cast<size_t>(p.B) + 1) * sizeof(int);
    if (smem > 48 * 1024) {
        // the same value on every call: concurrent callers cannot undo each other
        constexpr int kMost = (3 * kThreads * kPer + 1) * sizeof(int);
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel<kThreads, kPer>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
    }
    const int rows = (p.T + kThreads - 1) / kThreads, grid = rows == 1 ? 1 : std::max(std::min(rows + 1, num_sms), 2);
    const cudaError_t e = launch_pdl(paged_plan_kernel<kThreads, kPer>, dim3(grid), dim3(kThreads), smem, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
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
    if (B <= 256) return launch_plan<256, 1>(p, num_sms, s);
    if (B <= 1024) return launch_plan<1024, 1>(p, num_sms, s);
    if (B <= 4096) return launch_plan<1024, 4>(p, num_sms, s);
    return launch_plan<1024, 16>(p, num_sms, s);
}

}  // namespace mq
