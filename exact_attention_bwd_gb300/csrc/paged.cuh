// Packed queries over a paged cache: what the schedule, the kernels and the combine share.
//
// Work is counted in key tiles of a row tile.  A sequence's query rows (position, head of the
// group) of one key/value head are cut into row tiles; each head and row tile is an item of
// a few units for its prologue and epilogue, which cost about as much as so many tiles (`lead`),
// and one unit for each key tile in its band (one if it has none: its rows still have to be
// written).  All units form one line, sequence by sequence, head by head, row tile by row tile,
// and each of n CTAs takes an equal stretch of it, so the CTAs finish together whatever the
// lengths are; neighbours on the line, which run at the same time, share a head's keys in L2.
// A stretch's end among an item's tiles cuts it (one among its lead stands for the item's start):
// the pieces leave fp32 partials, at most two per CTA, so the workspace does not depend on the
// lengths, and the combine merges them in the order of the keys.
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

// The lead of an item in tiles: flat from 1 to 4 for both kernels (8 chunks of 1024 tokens 707 / 703 /
// 705 / 707 us, a mixed batch at d = 64 65 / 65 / 64 / 66).
constexpr int kLead = 2;
// Few rows over a cache in 8 bits: a tile takes half of the time, and an item's ends join 8 or 16 warps.
// (Decode of 64 requests over 2k to 32k keys with a lead of 2 / 4 / 6 / 10: 254 / 241 / 235 / 239 us; the chunks' kernels
// prefer 2 there as well.)
constexpr int kLeadFew8 = 6;

// Key tiles [t0, t1) of the rows [r0, r0 + rows) (numbered position * G + head of the group; r0 is
// one of them, nq * G fits 32 bits), and the units of the item.
template <int LEAD = kLead>
__device__ __forceinline__ int paged_tiles(const Problem& p, const PagedSeq& s, int r0, int rows, int& t0, int& t1) {
    const Band bd{s.nk - s.nq, p.left, p.right, s.nk};
    const unsigned G = (unsigned)p.G;
    const int i0 = (int)((unsigned)r0 / G), i1 = min(s.nq - 1, (int)((unsigned)(r0 + rows - 1) / G));
    kv_tile_range(bd, i0, i1, kKeyTile, t0, t1);
    return LEAD + max(t1 - t0, 1);
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
// With more than one CTA a stretch has LEAD / 2 + 1 units at least (two CTAs; at a lead of 2 4 units are two of 2, at one
// of 6 8 units two of 4).  One that ends among the lead of an item passes the item on, to the CTA that
// holds the lead's end, so a CTA may be left without a tile.
template <int LEAD = kLead>
__device__ __forceinline__ PagedLine paged_line(long long units, int n_ctas) {
    PagedLine x;
    x.units = units;
    x.n = (int)min((long long)n_ctas, (units + LEAD) / (LEAD + 1));
    x.each = x.n > 0 ? units / x.n : 0;
    x.more = x.n > 0 ? (int)(units % x.n) : 0;
    return x;
}

// The sequence of unit u: the largest b in [0, B) with pre[b] h_kv <= u, where pre[b] counts the
// units of one head ahead of sequence b (warp-wide; pre is non-decreasing, pre[0] = 0).
__device__ __forceinline__ int find_sequence(const long long* pre, int B, int h_kv, long long u) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B - 1;
#pragma unroll 1
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool le = at <= hi && pre[at] * h_kv <= u;
        lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// Unit `rem` of a sequence with `per_head` units to a head: its item (head, row tile), the unit of
// the item and the item's units and key tiles.  Warp-wide: a lane to a row tile, 32 at a time, from
// where the last look at the same head ended (units only move forward).
struct PagedUnit {
    int rt, g, k, cost, t0, t1;
};
struct PagedLook {
    int g = -1, base = 0;  // head, first of the 32 row tiles
    long long units = 0;   // of the head ahead of them
};
template <int LEAD = kLead>
__device__ __forceinline__ PagedUnit paged_unit(const Problem& p, const PagedSeq& s, int rows, long long rem, long long per_head,
                                                PagedLook& look) {
    const int lane = threadIdx.x & 31;
    const int tiles = (s.nq * p.G + rows - 1) / rows;
    PagedUnit x;
    x.g = rem < per_head ? 0 : (int)(rem / per_head);
    if (look.g != x.g) look = PagedLook{x.g, 0, 0};
    rem -= x.g * per_head + look.units;
    int base = look.base, src = 0, sum = 0, cost = 0, t0 = 0, t1 = 0;
#pragma unroll 1
    for (;; base += 32) {
        t0 = t1 = cost = 0;
        if (base + lane < tiles) cost = paged_tiles<LEAD>(p, s, (base + lane) * rows, rows, t0, t1);
        sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, rem < sum);
        src = past ? __ffs(past) - 1 : 31;
        if (past || base + 32 >= tiles) break;  // (no lane is past only for a unit outside the sequence)
        const int skipped = __shfl_sync(0xffffffffu, sum, 31);
        rem -= skipped;
        look.units += skipped;
    }
    look.base = base;
    x.rt = base + src;
    x.cost = __shfl_sync(0xffffffffu, cost, src);
    x.t0 = __shfl_sync(0xffffffffu, t0, src);
    x.t1 = __shfl_sync(0xffffffffu, t1, src);
    x.k = (int)rem - (__shfl_sync(0xffffffffu, sum, src) - x.cost);
    return x;
}

// An item cut behind its start: the CTA that holds the start leaves this for the combine.
struct PagedCut {
    int q0, g;        // first query row of the sequence, key/value head
    int r0, rows;     // first row and rows (0: the CTA's stretch cuts no item behind its start)
    int pieces;       // its CTAs, this one and the next ones
};

// The walk of one warp over its CTA's stretch, piece by piece.  Up to 32 sequences are held a lane
// each from the start, when line, units, offsets and lengths are read side by side; more are looked up one
// after another (decode of 32 sequences over 4000 keys 56.2 us, 57.2 with lookups).
template <int LEAD>
struct PagedWalkOf {
    long long u = 0, end = 0;  // next unit, end of the stretch
    bool held = false;
    long long my_pre = 0, my_units = 0;  // held: the units of a head ahead of the lane's sequence and its own
    PagedSeq mine{};
    long long before = 0, per_head = 0, after = 0;  // the sequence's: units ahead of it, of a head, up to its end
    int b = 0;
    PagedSeq seq{};
    PagedLook look;
    __device__ __forceinline__ void start(const Problem& p, const long long* pre, const PagedLine* line, int cta) {
        const int lane = threadIdx.x & 31;
        held = p.B <= 32;
        if (held && lane < p.B) {
            my_pre = pre[lane];
            my_units = pre[lane + 1] - my_pre;
            mine = paged_seq(p, lane);
        }
        u = line->start(cta);
        end = line->start(cta + 1);
    }
    PagedUnit x;               // the piece's item
    int t0 = 0, t1 = 0;        // its key tiles
    bool from_start = true, to_end = true;  // whether it is the item's start and end
    PagedCut cut{0, 0, 0, 0, 0};
    // Moves to the next piece; false: the stretch is done
    __device__ __forceinline__ bool next(const Problem& p, const long long* pre, const PagedLine& line, int cta, int rows, bool no_split) {
        while (u < end) {
            if (u >= after) {
                if (held) {
                    b = 31 - __clz(__ballot_sync(0xffffffffu, (threadIdx.x & 31) < p.B && my_pre * p.h_kv <= u));
                    before = __shfl_sync(0xffffffffu, my_pre, b) * p.h_kv;
                    per_head = __shfl_sync(0xffffffffu, my_units, b);
                    seq = PagedSeq{__shfl_sync(0xffffffffu, mine.q0, b), __shfl_sync(0xffffffffu, mine.nq, b), __shfl_sync(0xffffffffu, mine.nk, b)};
                } else {
                    b = find_sequence(pre, p.B, p.h_kv, u);
                    before = pre[b] * p.h_kv;
                    per_head = pre[b + 1] - pre[b];
                    seq = paged_seq(p, b);
                }
                after = before + per_head * p.h_kv;
                look.g = -1;
            }
            x = paged_unit<LEAD>(p, seq, rows, u - before, per_head, look);
            if (no_split && x.k > LEAD) {  // the item is the CTA's that holds its start
                u += x.cost - x.k;
                continue;
            }
            const long long start = u - x.k;
            if (end - start <= LEAD) break;  // the item's start counts for the next CTA
            from_start = x.k <= LEAD;
            to_end = no_split || end - start >= x.cost;
            t0 = x.t0 + (from_start ? 0 : x.k - LEAD);
            t1 = to_end ? x.t1 : x.t0 + (int)(end - start) - LEAD;
            u = to_end ? start + x.cost : end;
            if (from_start && !to_end) {
                const int r0 = x.rt * rows;
                cut = PagedCut{seq.q0, x.g, r0, min(rows, seq.nq * p.G - r0), line.owner(start + x.cost - 1) - cta + 1};
            }
            return true;
        }
        return false;
    }
};

using PagedWalk = PagedWalkOf<kLead>;
using PagedWalkFew8 = PagedWalkOf<kLeadFew8>;

// A warp's own copy of a value that all its lanes hold.  Where the warp groups split the registers
// between them, the walk needs more than its group has, and what other roles share with it would be
// spilled for it and loaded again in their loops; what comes out of a shuffle is a value of its own.
// (8 chunks of 1024 tokens 776 / 706 us; decode of 32 x 16000 keys at d = 64 and 40 rows 151 / 140.)
__device__ __forceinline__ int own_copy(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t own_copy(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
template <class T>
__device__ __forceinline__ T& own_shared(T& shared) {
    return *reinterpret_cast<T*>(__cvta_shared_to_generic(own_copy(smem_u32(&shared))));
}

}  // namespace fa
