// The page plan of a serving step: from the requests' cached and new token counts to the
// packed offsets, the used lengths, each token's position and cache slot, and the new
// block-table entries (include/fa.h, fa_page_plan).
//
//   cu[b]    = sum of n_r over r < b                      used[b] = c_b + n_b
//   pages of request b: old = ceil(c_b / P), total = ceil((c_b + n_b) / P); its new page j
//     (old <= j < total) is free[head + (new pages of the requests before it) + j - old]
//   token t of request b: position c_b + t - cu[b], slot = page(position / P) * P + position % P
//
// Two prefix sums over the requests and one lookup per token: a few hundred kilobytes at
// most, so the launch and its chain of dependent loads set the time, not bytes.  It is one
// launch without any exchange between CTAs: every CTA takes a run of tokens and scans the
// requests itself (they are few and stay in L2), a block of kThreads at a time.  The requests'
// own outputs (offsets, lengths, table entries) are written block by block by the CTAs in turn.
// (2048 requests, 139000 tokens: 11.5 us, 13.9 with 2048 tokens to a CTA and no loads ahead, 18.3
// with four requests to a thread; 32 requests of a decode step 3.2.)
#include "kernels.h"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kTokensPerCta = 1024;

struct PlanSmem {
    long long start[kThreads];  // first token of each request of the block
    long long warp_n[kThreads / 32], warp_p[kThreads / 32];
    long long first[kThreads];  // new pages of all requests before it
    int cached[kThreads], old[kThreads];
};

// Pages that n tokens take (n and the page below 2^31: their sum fits 32 bits without a sign).
__device__ __forceinline__ int pages_of(int n, int page) { return (int)(((unsigned)n + (unsigned)page - 1u) / (unsigned)page); }

// A page of the free list, or -1 past its end or outside the pool.
__device__ __forceinline__ int free_page(const PagePlanArgs& a, long long at, bool& bad) {
    const int pg = at >= 0 && at < a.n_free ? a.free_pages[at] : -1;
    if (pg >= 0 && pg < a.num_pages) return pg;
    bad = true;
    return -1;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const PagePlanArgs a) {
    __shared__ PlanSmem s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long t0 = (long long)blockIdx.x * kTokensPerCta;
    const long long t1 = min(t0 + (long long)kTokensPerCta, (long long)a.T);
    const int cap = a.max_blocks * a.page_size;  // tokens a table row can hold (fits: checked on the host)
    const long long head = a.free_head ? *a.free_head : 0;
    long long run_n = 0, run_p = 0;  // totals of the blocks before this one
    bool bad = head < 0;
    int next_c = tid < a.B ? a.cached[tid] : 0, next_n = tid < a.B ? a.fresh[tid] : 0;
    for (int base = 0; base < a.B || base == 0; base += kThreads) {
        const int b = base + tid;
        int c = next_c, n = next_n;
        // (the next block's are on their way meanwhile)
        next_c = b < a.B - kThreads ? a.cached[b + kThreads] : 0;
        next_n = b < a.B - kThreads ? a.fresh[b + kThreads] : 0;
        if (b < a.B) {
            if (c < 0 || n < 0 || (long long)c + n > cap) bad = true;
            c = min(max(c, 0), cap);
            n = max(n, 0);
        }
        const int used = (int)min((long long)c + n, (long long)cap);
        const int old = pages_of(c, a.page_size), np = pages_of(used, a.page_size) - old;
        // inclusive scans of the token and page counts
        long long sn = n, sp = np;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long xn = __shfl_up_sync(0xffffffffu, sn, o), xp = __shfl_up_sync(0xffffffffu, sp, o);
            if (lane >= o) {
                sn += xn;
                sp += xp;
            }
        }
        __syncthreads();  // the previous block's arrays are no longer read
        if (lane == 31) {
            s.warp_n[warp] = sn;
            s.warp_p[warp] = sp;
        }
        __syncthreads();
        long long before_n = run_n, before_p = run_p, all_n = run_n, all_p = run_p;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) {
                before_n += s.warp_n[w];
                before_p += s.warp_p[w];
            }
            all_n += s.warp_n[w];
            all_p += s.warp_p[w];
        }
        const long long start = before_n + sn - n, first = before_p + sp - np;
        s.start[tid] = start;
        s.cached[tid] = c;
        s.old[tid] = old;
        s.first[tid] = first;
        // the block's per-request outputs
        if ((base / kThreads) % gridDim.x == blockIdx.x) {
            if (b < a.B) {
                if (start + n > a.T) bad = true;
                a.cu[b + 1] = (int)min(start + n, (long long)a.T);
                if (b == 0) a.cu[0] = 0;
                a.used[b] = used;
                if (b == a.B - 1) *a.head_out = (int)min(head + all_p, 0x7fffffffLL);
            } else if (a.B == 0 && tid == 0) {
                a.cu[0] = 0;
                *a.head_out = (int)head;
            }
            // new table entries: one or two by the request's own thread, longer runs by the warp
            int* row = b < a.B ? a.table + (long long)b * a.max_blocks + old : a.table;
            if (np <= 2)
                for (int j = 0; j < np; ++j) row[j] = free_page(a, head + first + j, bad);
            for (unsigned m = __ballot_sync(0xffffffffu, np > 2); m; m &= m - 1) {
                const int src = __ffs(m) - 1;
                const int cnt = __shfl_sync(0xffffffffu, np, src);
                const long long f = __shfl_sync(0xffffffffu, first, src);
                int* to = reinterpret_cast<int*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), src));
                for (int j = lane; j < cnt; j += 32) to[j] = free_page(a, head + f + j, bad);
            }
        }
        __syncthreads();
        // this CTA's tokens among the block's requests
        const long long lo = max(t0, run_n), hi = min(t1, all_n);
        for (long long t = lo + tid; t < hi; t += kThreads) {
            int l = 0, r = kThreads - 1;  // the last request that starts at or before t
            while (l < r) {
                const int m = (l + r + 1) >> 1;
                if (s.start[m] <= t) l = m;
                else r = m - 1;
            }
            const long long at = s.cached[l] + (t - s.start[l]);
            int slot = -1;
            if (at < cap) {
                const int pos = (int)at, pg = pos / a.page_size, q = base + l;
                int page;
                if (pg < s.old[l]) {
                    page = a.table[(long long)q * a.max_blocks + pg];
                    if (page < 0 || page >= a.num_pages) {
                        page = -1;
                        bad = true;
                    }
                } else {
                    page = free_page(a, head + s.first[l] + pg - s.old[l], bad);
                }
                if (page >= 0) slot = page * a.page_size + pos % a.page_size;
            }
            a.positions[t] = at < cap ? (int)at : -1;
            a.slots[t] = slot;
        }
        run_n = all_n;
        run_p = all_p;
    }
    for (long long t = max(t0, run_n) + tid; t < t1; t += kThreads) {  // rows behind the last request
        a.positions[t] = -1;
        a.slots[t] = -1;
    }
    if (bad && a.status) atomicCAS(a.status, 0, FA_ERR_DEVICE_CHECK);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t st) {
    const int ctas = a.T > 0 ? cdiv(a.T, kTokensPerCta) : 1;
    page_plan_kernel<<<ctas, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
