// Packed queries over a paged cache: what the schedule, the kernels and the combine share.
//
// Work is counted in (row tile, key tile) units.  A sequence's query rows (position, head of
// the group) of one key/value head are cut into row tiles; each row tile and key/value head
// is an item of as many units as it has key tiles in its band (one if it has none: its rows
// still have to be written).  All units form one line, sequence by sequence, row tile by row
// tile, head by head, and each of n CTAs takes an equal stretch of it: every CTA streams the
// same number of key tiles whatever the lengths are.  An item cut by a stretch's end leaves
// fp32 partials (at most two per CTA, so the workspace does not depend on the lengths), which
// the combine merges in the order of the keys.
#pragma once
#include "common.cuh"

namespace fa {

constexpr int kKeyTile = 128;

struct PagedSeq {
    int q0, nq, nk;
};

// Offsets and lengths are kept within the tensors whatever the arrays hold.
__device__ __forceinline__ PagedSeq paged_seq(const Problem& p, int b) {
    PagedSeq s;
    s.q0 = min(max(p.cu_q[b], 0), p.T_q);
    s.nq = min(max(p.cu_q[b + 1], s.q0), p.T_q) - s.q0;
    if (p.seqused_q) s.nq = min(s.nq, max(0, p.seqused_q[b]));
    s.nk = min(max(p.seqused_k[b], 0), p.s_kv);
    return s;
}

// Key tiles [t0, t1) of the rows [r0, r0 + rows) (numbered position * G + head of the group; r0 is
// one of them, rows * G in all fit 32 bits), and the units they cost.
__device__ __forceinline__ int paged_tiles(const Problem& p, const PagedSeq& s, int r0, int rows, int& t0, int& t1) {
    const Band bd{s.nk - s.nq, p.left, p.right, s.nk};
    const unsigned G = (unsigned)p.G;
    const int i0 = (int)((unsigned)r0 / G), i1 = min(s.nq - 1, (int)((unsigned)(r0 + rows - 1) / G));
    kv_tile_range(bd, i0, i1, kKeyTile, t0, t1);
    return max(t1 - t0, 1);
}

// The line of one kernel's units as the preparation leaves it: n CTAs take part, CTA c's stretch
// is [start(c), start(c + 1)), the first `more` stretches one unit longer than `each`.
struct PagedLine {
    long long units;
    int n, more;
    long long each;
    __device__ __forceinline__ long long start(int c) const { return c * each + min(c, more); }
    // the CTA that holds unit u
    __device__ __forceinline__ int owner(long long u) const {
        const long long head = more * (each + 1);
        return u < head ? (int)(u / (each + 1)) : more + (int)((u - head) / each);
    }
};
// Each CTA has kMinUnits units at least.
constexpr int kMinUnits = 2;
__device__ __forceinline__ PagedLine paged_line(long long units, int n_ctas) {
    PagedLine x;
    x.units = units;
    x.n = (int)min((long long)n_ctas, (units + kMinUnits - 1) / kMinUnits);
    x.each = x.n > 0 ? units / x.n : 0;
    x.more = x.n > 0 ? (int)(units % x.n) : 0;
    return x;
}

// The largest b in [0, B) with pre[b] <= u (warp-wide; pre is non-decreasing, pre[0] = 0).
__device__ __forceinline__ int find_sequence(const long long* pre, int B, long long u) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B - 1;
#pragma unroll 1
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool le = at <= hi && pre[at] <= u;
        lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// Unit `rem` of a sequence: its item (row tile, head) and the unit of the item.  Warp-wide: a
// lane to a row tile, 32 at a time.
struct PagedUnit {
    int rt, g, k, cost, t0, t1;
};
__device__ __forceinline__ PagedUnit paged_unit(const Problem& p, const PagedSeq& s, int rows, long long rem) {
    const int lane = threadIdx.x & 31;
    const int tiles = (s.nq * p.G + rows - 1) / rows;
    PagedUnit x;
    int base = 0, src = 0, sum = 0, cost = 0, t0 = 0, t1 = 0;
#pragma unroll 1
    for (;; base += 32) {
        t0 = t1 = cost = 0;
        if (base + lane < tiles) cost = paged_tiles(p, s, (base + lane) * rows, rows, t0, t1);
        sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, rem < (long long)sum * p.h_kv);
        src = past ? __ffs(past) - 1 : 31;
        if (past || base + 32 >= tiles) break;  // (no lane is past only for a unit outside the sequence)
        rem -= (long long)__shfl_sync(0xffffffffu, sum, 31) * p.h_kv;
    }
    x.rt = base + src;
    x.cost = max(__shfl_sync(0xffffffffu, cost, src), 1);
    x.t0 = __shfl_sync(0xffffffffu, t0, src);
    x.t1 = __shfl_sync(0xffffffffu, t1, src);
    rem -= (long long)(__shfl_sync(0xffffffffu, sum, src) - x.cost) * p.h_kv;
    // rem < cost h_kv, which fits 32 bits
    x.g = (int)((unsigned)rem / (unsigned)x.cost);
    x.k = (int)((unsigned)rem - (unsigned)(x.g * x.cost));
    return x;
}

}  // namespace fa
