// Attention of packed queries over a paged cache, few query rows per key/value head (decode,
// verification of drafted tokens, short chunks), with its schedule and combine.
//
// With few rows the work is a stream over the cache, so the tensor cores take the keys as the
// long side: S^T = K Q^T (128 keys x NR rows) and O^T = V^T P^T (d x NR rows), both with the
// cache tile as the 128-row operand straight from the swizzled tile that TMA wrote, and NR = 16,
// 32 or 64 columns.  A key is a TMEM lane, so each of 128 threads does the softmax of one key
// for all rows.  The online softmax's reference maximum is only moved when some score passes it
// by more than 2^8 (one vote per tile), so the cross-lane maxima are formed rarely.  A tile's way
// through the softmax is a chain of latencies, at 32 and 64 rows longer than its keys take to
// arrive where they are few bytes: there (d = 64) two groups of four warps take the tiles in turn, each an
// online softmax of its own with its own accumulator, joined at the end.  (Decode of 32 x 16000
// keys, 4 heads, one group against two: d = 64 116 / 95 us at 32 rows and 158 / 110 at 64, none
// gained at 16; d = 128 179 / 181 at 64; with 2 heads d = 256 175 / 193 at 64.)
//
// Warp roles (one CTA per SM):
//   warp 0       TMA producer: K and V tiles, page by page, through a ring of [128 keys] units
//   warp 1       MMA issuer (one thread; of P V where warp 2 has S)
//   warp 2       owns the TMEM allocation; with two issuers the one of S (one thread)
//   warp 3       scheduler: finds the CTA's pieces of work, stages each item's Q rows
//   warps 4..7   softmax (thread = key) and epilogue (thread = column of O, then warp = row)
//   warps 8..11  with two groups: the softmax of the odd tiles of the CTA's stream (warps 4..7 then
//                have the even ones) and the epilogue of the second half of the rows
#include "cache8.cuh"
#include "paged.cuh"

namespace fa {
namespace {

// ------------------------------------------------------------------------------------------
// schedule: the line of units
// ------------------------------------------------------------------------------------------
constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
// row tiles that a thread counts by itself; longer sequences are counted by all threads together (one
// of 262144 tokens, four heads a group, by one thread: 273 us)
constexpr int kPrepAlone = 32;

template <int FEW, int MANY>  // the leads
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(const PagedArgs a) {
    __shared__ long long warp_sum[2][kPrepWarps];
    __shared__ unsigned long long units_of[kPrepThreads];
    __shared__ int bad_any, n_long, long_ones[kPrepThreads];
    const Problem& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    allow_next_kernel();
    long long run0 = 0, run1 = 0;
    bool bad = false;
    if (tid == 0) bad_any = 0;
    __syncthreads();
    for (int base = 0; base < p.B; base += kPrepThreads) {
        const int b = base + tid;
        long long w0 = 0, w1 = 0;
        bool is_long = false, few = false;
        if (tid == 0) n_long = 0;
        __syncthreads();
        if (b < p.B) {
            if (a.validate) {
                bad = bad || (b == 0 && p.cu_q[0] != 0) || p.cu_q[b + 1] < p.cu_q[b] || p.cu_q[b + 1] > p.T_q ||
                      p.seqused_k[b] < 0 || p.seqused_k[b] > p.s_kv;
            }
            const PagedSeq s = paged_seq(p, b);
            const long rows = (long)s.nq * p.G;
            if (rows > 0) {
                few = rows <= a.few_max;
                const int step = few ? a.few_rows : a.many_rows;
                is_long = rows > (long)kPrepAlone * step;
                long long w = 0;
                if (is_long) {
                    units_of[tid] = 0;
                    long_ones[atomicAdd(&n_long, 1)] = b;
                } else {
#pragma unroll 1
                    for (int r = 0; r < (int)rows; r += step) {
                        int t0, t1;
                        w += few ? paged_tiles<FEW>(p, s, r, step, t0, t1) : paged_tiles<MANY>(p, s, r, step, t0, t1);
                    }
                }
                (few ? w0 : w1) = w;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int e = 0; e < n_long; ++e) {
            const int bl = long_ones[e];
            const PagedSeq s = paged_seq(p, bl);
            const long rows = (long)s.nq * p.G;
            const int step = rows <= a.few_max ? a.few_rows : a.many_rows;
            long long w = 0;
#pragma unroll 1
            for (long r = (long)tid * step; r < rows; r += (long)kPrepThreads * step) {
                int t0, t1;
                w += rows <= a.few_max ? paged_tiles<FEW>(p, s, (int)r, step, t0, t1) : paged_tiles<MANY>(p, s, (int)r, step, t0, t1);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            if (lane == 0) atomicAdd(&units_of[bl - base], (unsigned long long)w);
        }
        __syncthreads();
        if (is_long) (few ? w0 : w1) = (long long)units_of[tid];
        long long s0 = w0, s1 = w1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x0 = __shfl_up_sync(0xffffffffu, s0, o), x1 = __shfl_up_sync(0xffffffffu, s1, o);
            if (lane >= o) {
                s0 += x0;
                s1 += x1;
            }
        }
        if (lane == 31) {
            warp_sum[0][warp] = s0;
            warp_sum[1][warp] = s1;
        }
        __syncthreads();
        long long b0 = run0, b1 = run1;
#pragma unroll
        for (int w = 0; w < kPrepWarps; ++w) {
            if (w < warp) {
                b0 += warp_sum[0][w];
                b1 += warp_sum[1][w];
            }
            run0 += warp_sum[0][w];
            run1 += warp_sum[1][w];
        }
        if (b < p.B) {
            a.pre[b + 1] = b0 + s0;
            a.pre[p.B + 1 + b + 1] = b1 + s1;
        }
        __syncthreads();
    }
    if (bad) bad_any = 1;
    __syncthreads();
    if (tid == 0) {
        a.pre[0] = 0;
        a.pre[p.B + 1] = 0;
        *a.status = bad_any ? kStatusDeviceCheck : kStatusOk;
        a.line[0] = paged_line<FEW>(run0 * p.h_kv, a.few_ctas);
    } else if (tid == 32) {
        a.line[1] = paged_line<MANY>(run1 * p.h_kv, a.many_ctas);
    }
}

// ------------------------------------------------------------------------------------------
// few-row kernel
// ------------------------------------------------------------------------------------------
// registers after setmaxnreg with two softmax groups: 128 x 72 + 256 x 216 = the launch's 384 x 168
constexpr int kFewRegLow = 72, kFewRegHigh = 216;
constexpr int kItems = 4;
constexpr int kSmemMax = 227 * 1024;

constexpr int pow2_at_least(int x) { return x <= 32 ? 32 : x <= 64 ? 64 : x <= 128 ? 128 : x <= 256 ? 256 : 512; }

template <int D, int NR>
struct FewCfg {
    static constexpr int UC = D == 256 ? 128 : D;      // columns of a ring unit
    static constexpr int KU = D / UC;                  // units of a K (or V) tile
    static constexpr int CHUNK = kKeyTile * 128;       // [128 keys][64 columns]
    static constexpr int UNIT = kKeyTile * UC * 2;
    static constexpr int Q_BYTES = NR * D * 2, P_BYTES = NR * kKeyTile * 2;
    static constexpr int Q_BUFS = Q_BYTES <= 16384 ? 2 : 1;
    static constexpr int FIT = (kSmemMax - 1024 - 4096 - Q_BUFS * Q_BYTES - 2 * P_BYTES) / UNIT;
    // MMA issuers.  With two, one thread issues S and another P V, which one thread could not do as fast as
    // small tiles arrive (16000 keys, 4 heads: d = 64 at 16 / 32 / 64 rows 111 / 117 / 128 us with one, 92 / 95 /
    // 110 with two, d = 128 at 64 rows 182 / 178; but 164 / 167 at 16).  Each waits for its own units by
    // the parity of their slots' phases, so K and V must have slots of their own: one unit to a tile
    // and an even ring (a phase that a thread has not waited for would pass for the one after it).
    static constexpr int ISSUERS = D == 64 || (D == 128 && NR >= 32) ? 2 : 1;
    static constexpr int MOST = D == 64 ? 12 : 6;
    static constexpr int RING = ISSUERS == 2 ? (FIT > MOST ? MOST : FIT / 2 * 2) : (FIT > MOST ? MOST : FIT);
    static_assert(ISSUERS == 1 || (KU == 1 && RING % 2 == 0), "slots of their own");
    static_assert(RING >= 3 && RING >= 2 * KU, "a K and a V tile have to fit");
    // Some unit of a tile's V takes the slot of a unit of the V before it (d = 256 at 32 and 64 rows,
    // rings of 5 and 4 units): by parity, a wait for its arrival would also pass while the
    // one before has not arrived yet.
    static constexpr bool V_AFTER_V = RING < 3 * KU;
    static constexpr int OH = D > 128 ? 2 : 1;         // 128-lane accumulators of O^T
    // P^T in shared memory: 64 rows are a whole swizzle row per key, which a thread writes with
    // eight 16-byte stores (rows innermost); fewer rows lie [row][key], a 2-byte store each
    static constexpr bool P_MN = NR == 64;
    static constexpr int NG = D == 64 && NR >= 32 ? 2 : 1;  // softmax groups
    static constexpr int THREADS = 128 + 128 * NG;
    // scores held at a time; with two groups (fewer registers) 64 rows are read twice, 32 at a time
    static constexpr int HR = NG == 2 && NR > 32 ? 32 : NR;
    static constexpr int TMEM_COLS = pow2_at_least(2 * NR + NG * OH * NR);
    // Unit n of the stream: K and V tiles in turn.  At d = 64 the 128-row V^T operand takes the
    // slot behind V's as its second 64 rows (their products, lanes 64 .. 127, are not read): K and V
    // swap slots so that this is the K of the same tile, which is held until then.
    __device__ static __forceinline__ int slot_of(uint32_t n) { return D == 64 ? (int)(n % RING) ^ 1 : (int)(n % RING); }
};

struct FewItem {
    int end;
    int b, q0, nq, nk, g;
    int r0, rows;      // first row of the sequence's (position, head) rows, rows held
    int t0, t1;        // key tiles
    int lo, hi;        // keys that any row of the item may see
    int part;          // partial slot, or -1: the item is whole
};

template <int D, int NR>
struct __align__(1024) FewSmem {
    using C = FewCfg<D, NR>;
    uint8_t ring[C::RING][C::UNIT];
    uint8_t q[C::Q_BUFS][C::Q_BYTES];
    uint8_t p[2][C::P_BYTES];
    // Of each softmax group: reference maxima m of the item's rows (log2 units; -inf: no key so
    // far); what the exponent adds, -m (0 for -inf); minus the score (unscaled) past which m
    // moves, (m + 8) / scale; the last change of m as a factor, in the epilogue the factor of O; sums
    float mref[C::NG][NR];
    alignas(16) float negm[C::NG][NR];
    alignas(16) float limit[C::NG][NR];
    alignas(16) float alpha[C::NG][NR];
    float lsum[C::NG][NR];
    uint64_t full[C::RING], empty[C::RING];
    uint64_t q_full[C::Q_BUFS], q_empty[C::Q_BUFS];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free, drain[2];
    uint64_t item_full[kItems], item_empty[kItems];
    FewItem item[kItems];
    uint32_t tmem_base;
    int abort_flag;
};

// NR consecutive fp32 TMEM columns of the warp's 32 lanes.
template <int NR>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t* r) {
    if constexpr (NR == 8) tmem_ld_32x32b_x8(addr, r);
    else if constexpr (NR == 16) tmem_ld_32x32b_x16(addr, r);
    else if constexpr (NR == 32) tmem_ld_32x32b_x32(addr, r);
    else tmem_ld_32x32b_x64(addr, r);
}
template <int NR>
__device__ __forceinline__ void tmem_st_cols(uint32_t addr, const uint32_t* r) {
    if constexpr (NR == 16) tmem_st_32x32b_x16(addr, r);
    else if constexpr (NR == 32) tmem_st_32x32b_x32(addr, r);
    else tmem_st_32x32b_x64(addr, r);
}

// Votes of softmax threads (named barriers: 1 + group for a group's four warps, 3 for both
// groups): what one of them decides all decide, so no warp is left waiting for another that gave
// up.  The barriers' numbers are immediates.
template <int BAR, int THREADS>
__device__ __forceinline__ bool vote_at(bool x) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbarrier.cta.red.or.pred q, %2, %3, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(BAR), "n"(THREADS)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ bool group_or(int grp, bool x) { return grp ? vote_at<2, 128>(x) : vote_at<1, 128>(x); }
__device__ __forceinline__ void group_sync(int grp) {
    if (grp) asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
    else asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}

template <int D, int NR>
__global__ void __launch_bounds__(FewCfg<D, NR>::THREADS, 1)
    paged_few_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = FewCfg<D, NR>;
    constexpr int RING = C::RING, KU = C::KU;
    extern __shared__ uint8_t smem_raw[];
    FewSmem<D, NR>& smem = *reinterpret_cast<FewSmem<D, NR>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    FewSmem<D, NR>& s = smem;
    const Problem& p = a.p;
    const bool f16 = p.dtype == FA_DTYPE_F16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    allow_next_kernel();

    Abort ab{&s.abort_flag, a.status, p.wait_ns};
    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < RING; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < C::Q_BUFS; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.pv_done[i], 1);
        }
        mbar_init(&s.o_free, 4 * C::NG);
        mbar_init(&s.drain[0], 1);
        mbar_init(&s.drain[1], 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], 1 + C::ISSUERS + 4 * C::NG);  // producer, MMA issuers, softmax warps
        }
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(&s.tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    // the schedule is there; a CTA without work, or one of a call that already failed, leaves
    wait_previous_kernel();
    PagedWalk walk;
    if (warp == 3) walk.start(p, a.pre, a.line, cta);
    // (one thread looks, so that all leave or none)
    tc_fence_before();
    const bool leave = __syncthreads_or(tid == 0 && (cta >= a.line->n || *reinterpret_cast<volatile int*>(a.status) != 0));
    tc_fence_after();
    if (leave) {
        if (warp == 2) tmem_dealloc(s.tmem_base, C::TMEM_COLS);
        return;
    }
    const uint32_t tmem_base = s.tmem_base, tmem = tmem_base;
    // TMEM columns: the two S buffers (tile g's is g & 1), group x's O^T at cO + OH NR x
    constexpr uint32_t cS = 0, cO = 2 * NR;

    if (warp < 4) {
    if constexpr (C::NG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kFewRegLow) : "memory");
    if (warp == 0) {
        // ================= TMA producer =================
        FewSmem<D, NR>& s = C::NG == 2 ? own_shared(smem) : smem;
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        const int boxes = kKeyTile / a.box;
        uint32_t n = 0;  // units issued
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it % kItems;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s.item_full[slot], (it / kItems) & 1, ab)))) break;
            const int end = s.item[slot].end, b = s.item[slot].b, lo = s.item[slot].lo, hi = s.item[slot].hi, g = s.item[slot].g;
            const int t0 = s.item[slot].t0, t1 = s.item[slot].t1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.item_empty[slot]);
            if (end) break;
            const int32_t* table = p.block_table + (long)b * p.max_blocks;
            // lane x takes box x of a tile: its page, or the pool's end (zero fill) past the keys that any
            // row sees or for a table entry outside the pool, which is an error where some row sees a key of
            // the box.  The entry of the next tile is on its way while this one waits for its slots.
            auto entry = [&](int t) {
                const int j = t * kKeyTile + lane * a.box;
                return lane < boxes && t < t1 && j <= hi ? table[j / p.page_size] : a.num_pages;
            };
            int next = entry(t0);
            for (int t = t0; ok && t < t1; ++t) {
                int page = next;
                next = entry(t + 1);
                const int j = t * kKeyTile + lane * a.box, row = j % p.page_size;
                if (lane < boxes && (unsigned)page >= (unsigned)a.num_pages) {
                    if (j <= hi && j + a.box > lo) atomicCAS(a.status, 0, kStatusDeviceCheck);
                    page = a.num_pages;
                }
#pragma unroll
                for (int x = 0; x < 2 * KU; ++x, ++n) {
                    const int sl = C::slot_of(n);
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s.empty[sl], ((n / RING) & 1) ^ 1, ab)))) break;
                    if (lane == 0) mbar_expect_tx(&s.full[sl], C::UNIT);
                    __syncwarp();
                    if (lane < boxes) {
#pragma unroll
                        for (int c = 0; c < C::UC / 64; ++c)
                            tma_load_4d(&s.ring[sl][c * C::CHUNK + lane * a.box * 128], x < KU ? &tmk : &tmv, &s.full[sl],
                                        (x % KU) * C::UC + c * 64, g, row, page);
                    }
                }
            }
        }
        // every copy still in flight lands before the CTA may exit
        for (uint32_t back = 1; back <= (uint32_t)RING && back <= n; ++back)
            mbar_wait_quiet(&s.full[C::slot_of(n - back)], ((n - back) / RING) & 1);
    } else if (warp == 1 || (C::ISSUERS == 2 && warp == 2)) {
        // ================= MMA issuer (of two: warp 2 S, warp 1 P V) =================
        FewSmem<D, NR>& s = C::NG == 2 ? own_shared(smem) : smem;
        const uint32_t tmem = C::NG == 2 ? own_copy(tmem_base) : tmem_base;
        if (lane == 0) {
            const uint32_t idS = idesc_16(128, NR, false, false, f16);
            const uint32_t idO = idesc_16(128, NR, true, C::P_MN, f16);
            uint32_t gt = 0, qi = 0;  // tiles of the CTA's stream before the item, items with keys
            bool ok = true;
            // the KU units from n on have arrived
            auto arrived = [&](uint32_t n) {
                bool y = true;
#pragma unroll
                for (int h = 0; h < KU; ++h) y = y && mbar_test(&s.full[C::slot_of(n + h)], ((n + h) / RING) & 1);
                return y;
            };
            auto issue_s = [&](uint32_t g, uint32_t q_addr) {
#pragma unroll
                for (int h = 0; h < KU; ++h) {
                    const int sl = C::slot_of(2 * KU * g + h);
                    const uint64_t kd = sdesc_sw128(smem_u32(s.ring[sl]), 16, 1024);
                    const uint64_t qd = sdesc_sw128(q_addr + h * (C::UC / 64) * NR * 128, 16, 1024);
#pragma unroll
                    for (int c = 0; c < C::UC / 64; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_ss(tmem + cS + NR * (g & 1), kd + c * (C::CHUNK >> 4) + 2 * x, qd + c * (NR * 8) + 2 * x, idS,
                                   h > 0 || c > 0 || x > 0 ? 1u : 0u);
                    if (D != 64) tc_commit(&s.empty[sl]);
                }
                tc_commit(&s.s_full[g & 1]);
            };
            auto issue_pv = [&](uint32_t g, bool start) {
                const uint64_t pd = sdesc_sw128(smem_u32(s.p[g & 1]), 16, 1024);
                auto product = [&](uint32_t o_col, uint32_t v_addr) {
                    const uint64_t vd = sdesc_sw128(v_addr, C::CHUNK, 1024);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        mma_ss(tmem + o_col, vd + 128 * x, pd + (C::P_MN ? 128 * x : (x / 4) * (NR * 8) + 2 * (x % 4)), idO,
                               !start || x > 0 ? 1u : 0u);
                };
                const uint32_t o_col = cO + (C::NG == 2 ? C::OH * NR * (g & 1) : 0);
#pragma unroll
                for (int h = 0; h < KU; ++h) {
                    const int sl = C::slot_of(2 * KU * g + KU + h);
                    product(o_col + NR * h, smem_u32(s.ring[sl]));
                    // d = 192: columns 64 .. 191 again as the second accumulator
                    if (D == 192) product(o_col + NR, smem_u32(s.ring[sl]) + C::CHUNK);
                    tc_commit(&s.empty[sl]);
                }
                if (D == 64) tc_commit(&s.empty[C::slot_of(2 * g)]);
                tc_commit(&s.pv_done[g & 1]);
            };
            for (int it = 0; ok; ++it) {
                const int slot = it % kItems;
                if (!(ok = mbar_wait(&s.item_full[slot], (it / kItems) & 1, ab))) break;
                const int end = s.item[slot].end, nt = s.item[slot].t1 - s.item[slot].t0;
                mbar_arrive(&s.item_empty[slot]);
                if (end) break;
                if (nt <= 0) continue;
                const int qb = (int)(qi % C::Q_BUFS);
                const uint32_t q_addr = smem_u32(s.q[qb]);
                // the K or the V unit n of a tile of one unit has arrived
                auto wait_unit = [&](uint32_t n) {
                    const bool y = mbar_wait(&s.full[C::slot_of(n)], (n / RING) & 1, ab);
                    tc_fence_after();
                    return y;
                };
                if constexpr (D > 128) {
                    if (!(ok = mbar_wait(&s.q_full[qb], (qi / C::Q_BUFS) & 1, ab))) break;
                    // The ring holds two tiles at most, so either product's operands may come first:
                    // whichever has them goes, P V before S (tile j's S goes into the buffer whose scores
                    // were tile j - 2's, so it may run two tiles ahead).  A fixed order
                    // takes 15 % longer (16000 keys, 2 heads, 64 rows, d = 256 and d = 192).  (S of tile j
                    // comes behind P V of tile j - 2, so every earlier phase of its slots has been seen.)
                    int js = 0, jv = 0;  // tiles whose S, whose P V was issued
                    uint32_t idle = 0;
                    unsigned long long since = 0;
                    while (jv < nt) {
                        const uint32_t gv = gt + jv, gs = gt + js;
                        if (jv < js && mbar_test(&s.p_full[gv & 1], (gv >> 1) & 1) && arrived(2 * KU * gv + KU) &&
                            (jv > 0 || qi == 0 || mbar_test(&s.o_free, (qi - 1) & 1))) {  // (the previous item's O has been read)
                            tc_fence_after();
                            issue_pv(gv, jv < C::NG);
                            ++jv;
                            idle = 0;
                            since = 0;
                        } else if (js < nt && js <= jv + 1 && arrived(2 * KU * gs)) {
                            tc_fence_after();
                            issue_s(gs, q_addr);
                            if (++js == nt) tc_commit(&s.q_empty[qb]);
                            idle = 0;
                            since = 0;
                        } else {
                            // nothing yet; the bound on all of it (the clock every 32 rounds)
                            if ((++idle & 31) == 0) {
                                const unsigned long long now = globaltimer();
                                if (since == 0) since = now;
                                if (ab.raised() || now - since > ab.limit) {
                                    ab.raise(kStatusTimeout);
                                    ok = false;
                                    break;
                                }
                            }
                        }
                    }
                } else if constexpr (C::ISSUERS == 1) {
                    // S two tiles ahead, in a fixed order (a deep ring: looking for what is ready costs more
                    // than it finds, 400 against 393 us for 64 requests at d = 128)
                    if (!(ok = mbar_wait(&s.q_full[qb], (qi / C::Q_BUFS) & 1, ab))) break;
                    for (int t = -2; t < nt; ++t) {
                        if (t >= 0) {
                            const uint32_t g = gt + t;
                            if (!(ok = mbar_wait(&s.p_full[g & 1], (g >> 1) & 1, ab))) break;
                            // the previous item's O has been read
                            if (t == 0 && qi > 0 && !(ok = mbar_wait(&s.o_free, (qi - 1) & 1, ab))) break;
                            if (!(ok = wait_unit(2 * g + 1))) break;
                            issue_pv(g, t < C::NG);
                        }
                        if (t + 2 < nt) {
                            if (!(ok = wait_unit(2 * (gt + t + 2)))) break;
                            issue_s(gt + t + 2, q_addr);
                            if (t + 3 == nt) tc_commit(&s.q_empty[qb]);
                        }
                    }
                } else {
                    if (warp == 2) {
                        if (!(ok = mbar_wait(&s.q_full[qb], (qi / C::Q_BUFS) & 1, ab))) break;
                        for (int t = 0; t < nt; ++t) {
                            const uint32_t g = gt + t;
                            // (the buffer's last scores, two tiles ago, have become P)
                            if (g >= 2 && !(ok = mbar_wait(&s.p_full[g & 1], ((g - 2) >> 1) & 1, ab))) break;
                            if (!(ok = wait_unit(2 * g))) break;
                            issue_s(g, q_addr);
                        }
                        if (ok) tc_commit(&s.q_empty[qb]);
                    } else {
                        for (int t = 0; t < nt; ++t) {
                            const uint32_t g = gt + t;
                            if (!(ok = mbar_wait(&s.p_full[g & 1], (g >> 1) & 1, ab))) break;
                            // the previous item's O has been read
                            if (t == 0 && qi > 0 && !(ok = mbar_wait(&s.o_free, (qi - 1) & 1, ab))) break;
                            if (!(ok = wait_unit(2 * g + 1))) break;
                            issue_pv(g, t < C::NG);
                        }
                    }
                }
                gt += nt;
                ++qi;
            }
            tc_commit(&s.drain[warp - 1]);
            mbar_wait_quiet(&s.drain[warp - 1], 0);
        }
    } else if (warp == 3) {
        // ================= scheduler =================
        const PagedLine line = *a.line;
        int it = 0;
        uint32_t qi = 0;
        bool ok = true;
        // Q rows: a lane takes a 16-byte unit of every ROWS-th row; from one to the next the head moves by
        // step_h in the group, with the tokens in between and one more where it wraps
        constexpr int ROWS = D == 192 ? 1 : 256 / D, LANES = ROWS * (D / 8);
        const int row = D == 192 ? 0 : lane / (D / 8), col = lane - row * (D / 8);
        const unsigned step_h = (unsigned)ROWS % (unsigned)p.G;
        const long step = ((long)(ROWS / p.G) * p.h_q + step_h) * D;
        while (ok && walk.next(p, a.pre, line, cta, NR, a.no_split)) {
            const PagedUnit& x = walk.x;
            const int t0 = walk.t0, t1 = walk.t1;
            const PagedSeq& sq = walk.seq;
            const int r0 = x.rt * NR, rows = min(NR, sq.nq * p.G - r0);
            const int slot = it % kItems;
            if (it >= kItems && !(ok = __all_sync(0xffffffffu, mbar_wait(&s.item_empty[slot], ((it / kItems) - 1) & 1, ab)))) break;
            if (lane == 0) {
                const Band bd{sq.nk - sq.nq, p.left, p.right, sq.nk};
                FewItem& w = s.item[slot];
                w.end = 0;
                w.b = walk.b;
                w.q0 = sq.q0;
                w.nq = sq.nq;
                w.nk = sq.nk;
                w.g = x.g;
                w.r0 = r0;
                w.rows = rows;
                w.t0 = t0;
                w.t1 = t1;
                w.lo = bd.lo(r0 / p.G);
                w.hi = bd.hi((r0 + rows - 1) / p.G);
                w.part = walk.from_start && walk.to_end ? -1 : 2 * cta + (walk.from_start ? 1 : 0);
                mbar_arrive(&s.item_full[slot]);
            }
            ++it;
            if (t1 <= t0) continue;
            // Q rows of the item, in the 128-byte-swizzled layout the MMA reads; zeros past them
            const int qb = (int)(qi % C::Q_BUFS);
            if (qi >= (uint32_t)C::Q_BUFS &&
                !(ok = __all_sync(0xffffffffu, mbar_wait(&s.q_empty[qb], ((qi / C::Q_BUFS) - 1) & 1, ab))))
                break;
            // (asynchronous copies, all of them in flight at once: through registers, four at a time,
            // the 64 rows of d = 256 took 16 round trips, and verifying 5 tokens of 16 / 2 heads in 32
            // sequences 73 us against 62)
            if (lane < LANES) {
                unsigned i = (unsigned)(r0 + row) / (unsigned)p.G, h = (unsigned)(r0 + row) - i * p.G;
                const uint16_t* src = a.q + (((long)sq.q0 + i) * p.h_q + x.g * p.G + h) * D + 8 * col;
                uint8_t* to = &s.q[qb][(col >> 3) * NR * 128];
#pragma unroll 4
                for (int r = row; r < NR; r += ROWS) {
                    copy16_async(to + r * 128 + (((col ^ r) & 7) << 4), r < rows ? src : a.q, r < rows);
                    h += step_h;
                    src += step;
                    if (h >= (unsigned)p.G) {
                        h -= p.G;
                        src += (long)(p.h_q - p.G) * D;
                    }
                }
            }
            copies_wait();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.q_full[qb]);
            ++qi;
        }
        if (lane == 0) a.cut[cta] = walk.cut;
        if (ok) {
            const int slot = it % kItems;
            if (it < kItems || __all_sync(0xffffffffu, mbar_wait(&s.item_empty[slot], ((it / kItems) - 1) & 1, ab))) {
                if (lane == 0) {
                    s.item[slot].end = 1;
                    mbar_arrive(&s.item_full[slot]);
                }
            }
        }
    }
    } else {
        if constexpr (C::NG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kFewRegHigh) : "memory");
        // ================= softmax: one thread per key =================
        FewSmem<D, NR>& s = C::NG == 2 ? own_shared(smem) : smem;
        const uint32_t tmem = C::NG == 2 ? own_copy(tmem_base) : tmem_base;
        const int warp = C::NG == 2 ? own_copy(tid >> 5) : tid >> 5;
        constexpr int HR = C::HR, NG = C::NG;
        const int grp = NG == 2 ? (warp - 4) >> 2 : 0, key = tid & 127, sub = warp & 3;
        const uint32_t lane_base = (uint32_t)(sub * 32) << 16;
        const uint32_t tO = tmem + lane_base + cO + C::OH * NR * grp;
        const float c = p.scale_log2;
        // byte offset of this key in row r of a [row][key] P buffer: p_at[r & 7] + 128 r
        uint32_t p_at[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            p_at[x] = (key >> 6) * (NR * 128) + (((((key & 63) >> 3) ^ x) & 7) << 4) + (key & 7) * 2;
        // The group's P buffer, while none of its P V is in flight: [warp][row] of what is joined across the
        // keys (thread `key` then takes row `key`), [row][key] of the output on its way to rows.
        float* grid = reinterpret_cast<float*>(s.p[grp]);
        constexpr int GR = NR / NG;  // rows that the group finishes
        auto joined = [&](auto op, int row) {  // of the four warps' values of a row
            return op(op(grid[row], grid[NR + row]), op(grid[2 * NR + row], grid[3 * NR + row]));
        };
        uint32_t gt = 0;  // tiles of the CTA's stream before the item
        bool ok = true;
        for (int it = 0;; ++it) {
            const int slot = it % kItems;
            ok = __all_sync(0xffffffffu, mbar_wait(&s.item_full[slot], (it / kItems) & 1, ab)) && ok;
            if (vote_at<3, 128 * NG>(!ok)) break;
            if (s.item[slot].end) break;
            const FewItem& w = s.item[slot];
            const int t0 = w.t0, t1 = w.t1, off = w.nk - w.nq, nk = w.nk, lo = w.lo, hi = w.hi, r0 = w.r0;
            // a tile inside [in_lo, in_hi] is seen by every row
            const unsigned G = (unsigned)p.G;
            const int in_lo = p.left >= 0 ? (int)((unsigned)(r0 + w.rows - 1) / G) + off - p.left : 0;
            const int in_hi = p.right >= 0 ? min(nk - 1, (int)((unsigned)r0 / G) + off + p.right) : nk - 1;
            float2 l[NR / 2];  // sums of the rows 2 r, 2 r + 1 over this key's tiles
#pragma unroll
            for (int r = 0; r < NR / 2; ++r) l[r] = make_float2(0.f, 0.f);
            const int first = t0 + (NG == 2 ? (gt ^ grp) & 1 : 0);  // the group's tiles: first, first + NG, ...
            uint32_t g = gt + (first - t0);           // index of the tile in the CTA's stream
            for (int t = first; t < t1; t += NG, g += NG) {
                const int buf = NG == 2 ? grp : g & 1;
                const uint32_t tS = tmem + lane_base + cS + NR * buf;
                uint8_t* pbuf = s.p[buf];
                const int j0 = t * kKeyTile, j = j0 + key;
                const bool edge = j0 < in_lo || j0 + kKeyTile - 1 > in_hi;
                // rows [ra, rb] see key j: positions j - off - right <= i <= j - off + left
                int ra = 0, rb = NR - 1;
                if (edge) {
                    if (p.right >= 0) ra = (int)max(min(((long)j - off - p.right) * p.G - r0, (long)NR), 0l);
                    if (p.left >= 0) rb = (int)min(max(((long)j - off + p.left + 1) * p.G - 1 - r0, -1l), (long)NR);
                    if (j >= nk) ra = NR;
                }
                // HR scores of this key from row r0 on, masked
                auto scores = [&](int h, uint32_t* sr) {
                    tmem_ld_cols<HR>(tS + h, sr);
                    if (edge) {
#pragma unroll
                        for (int r = 0; r < HR; ++r)
                            if (h + r < ra || h + r > rb) sr[r] = __float_as_uint(-INFINITY);
                    }
                };
                ok = __all_sync(0xffffffffu, mbar_wait(&s.s_full[buf], (g >> 1) & 1, ab)) && ok;
                tc_fence_after();
                uint32_t sr[HR];
                // (a maximum rather than a chain of comparisons, which took a quarter longer at d = 64 and 64 rows)
                float past[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // largest score - limit
#pragma unroll
                for (int h = 0; h < NR; h += HR) {
                    scores(h, sr);
#pragma unroll
                    for (int r = 0; r < HR; r += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(&s.limit[grp][h + r]);
                        const float2 x = __fadd2_rn(make_float2(__uint_as_float(sr[r]), __uint_as_float(sr[r + 1])), make_float2(m.x, m.y));
                        const float2 y = __fadd2_rn(make_float2(__uint_as_float(sr[r + 2]), __uint_as_float(sr[r + 3])), make_float2(m.z, m.w));
                        past[(r >> 2) & 3] = max3(past[(r >> 2) & 3], fmaxf(x.x, x.y), fmaxf(y.x, y.y));
                    }
                }
                // (the item's first tile sets the references)
                const bool over = t == first || fmaxf(fmaxf(past[0], past[1]), fmaxf(past[2], past[3])) > 0.f;
                if (group_or(grp, over || !ok)) {
                    if (group_or(grp, !ok)) break;
                    // some score passes its row's reference by more than 2^8: the references move to the
                    // maxima so far, sums and O follow
                    if (t > first) {  // O holds P V of the group's tile before, its P buffers are free
                        ok = __all_sync(0xffffffffu, mbar_wait(&s.pv_done[(g - NG) & 1], ((g - NG) >> 1) & 1, ab)) && ok;
                        tc_fence_after();
                    }
                    // (a loop, 16 rows at a time: this comes once or twice an item, and straight-line code
                    // for 64 rows took 2.2 us, most of it instruction fetches)
#pragma unroll 1
                    for (int h = 0; h < NR; h += 16) {
                        uint32_t x[16];
                        tmem_ld_cols<16>(tS + h, x);
                        float top = -INFINITY;  // lane r: row h + r, over the warp's keys
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float m = warp_max(edge && (h + r < ra || h + r > rb) ? -INFINITY : __uint_as_float(x[r]));
                            if (lane == r) top = m;
                        }
                        if (lane < 16) grid[NR * sub + h + lane] = top;
                    }
                    group_sync(grp);
                    if (key < NR) {
                        const float x = joined([](float a, float b) { return fmaxf(a, b); }, key);
                        const float m = t == first ? -INFINITY : s.mref[grp][key], mn = fmaxf(m, x * c);
                        s.alpha[grp][key] = m == mn ? 1.f : ex2(m - mn);  // m = -inf: 0
                        s.mref[grp][key] = mn;
                        s.negm[grp][key] = mn == -INFINITY ? 0.f : -mn;
                        // (no key so far: any finite score passes)
                        s.limit[grp][key] = mn == -INFINITY ? INFINITY : -(mn + 8.f) / c;
                    }
                    group_sync(grp);
                    if (t > first) {
#pragma unroll
                        for (int r = 0; r < NR; r += 4) {
                            const float4 al = *reinterpret_cast<const float4*>(&s.alpha[grp][r]);
                            l[r / 2] = __fmul2_rn(l[r / 2], make_float2(al.x, al.y));
                            l[r / 2 + 1] = __fmul2_rn(l[r / 2 + 1], make_float2(al.z, al.w));
                        }
                        constexpr int OC = NR < 32 ? NR : 32;  // columns of O at a time
#pragma unroll 1
                        for (int h = 0; h < C::OH * NR; h += OC) {
                            uint32_t o[OC];
                            tmem_ld_cols<OC>(tO + h, o);
                            const float* al = &s.alpha[grp][h % NR];
#pragma unroll
                            for (int r = 0; r < OC; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * al[r]);
                            tmem_st_cols<OC>(tO + h, o);
                        }
                    }
                }
                // P^T of this key: 16-bit (the MMA's operand type), the sums from the unrounded values
                if (g >= 2) {  // the buffer's last P V has completed
                    ok = __all_sync(0xffffffffu, mbar_wait(&s.pv_done[buf], ((g - 2) >> 1) & 1, ab)) && ok;
                }
                auto store_p = [&](auto pack) {
                    const float2 c2 = make_float2(c, c);
#pragma unroll
                    for (int h = 0; h < NR; h += HR) {
                        if (NR > HR) scores(h, sr);
#pragma unroll
                        for (int r = 0; r < HR; r += 8) {
                            uint32_t w2[4];
#pragma unroll
                            for (int e = 0; e < 8; e += 4) {
                                const float4 m = *reinterpret_cast<const float4*>(&s.negm[grp][h + r + e]);
                                const uint32_t* z = sr + r + e;
                                const float2 x = __ffma2_rn(make_float2(__uint_as_float(z[0]), __uint_as_float(z[1])), c2, make_float2(m.x, m.y));
                                const float2 y = __ffma2_rn(make_float2(__uint_as_float(z[2]), __uint_as_float(z[3])), c2, make_float2(m.z, m.w));
                                const float2 ex = make_float2(ex2(x.x), ex2(x.y)), ey = make_float2(ex2(y.x), ex2(y.y));
                                float2* sum = l + (h + r + e) / 2;
                                sum[0] = __fadd2_rn(sum[0], ex);
                                sum[1] = __fadd2_rn(sum[1], ey);
                                w2[e / 2] = pack(ex.x, ex.y);
                                w2[e / 2 + 1] = pack(ey.x, ey.y);
                            }
                            if constexpr (C::P_MN) {
                                // row `key` of the operand: its 16-byte unit u at position u ^ (key & 7)
                                *reinterpret_cast<uint4*>(&pbuf[key * 128 + (((((h + r) >> 3) ^ key) & 7) << 4)]) =
                                    make_uint4(w2[0], w2[1], w2[2], w2[3]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    *reinterpret_cast<uint16_t*>(&pbuf[p_at[e] + 128 * (h + r + e)]) = (uint16_t)(w2[e / 2] >> (16 * (e & 1)));
                            }
                        }
                    }
                };
                if (f16) store_p([](float x, float y) { return pack16<true>(x, y); });
                else store_p([](float x, float y) { return pack16<false>(x, y); });
                if (edge) {
                    // values at keys that no row sees may be anything (unused rows of a page): 0 * NaN
                    // would reach every row, so they are cleared
                    bool there = true;
                    // (S of this tile may be done ahead of the V before it, which then is still on its way
                    // into the slot; its product is not: the issuer has that tile's P)
                    if (C::V_AFTER_V && g >= 1) there = mbar_wait(&s.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, ab);
#pragma unroll
                    for (int h = 0; h < KU; ++h) {
                        const uint32_t n = 2 * KU * g + KU + h;
                        const int sl = C::slot_of(n);
                        there = there && mbar_wait(&s.full[sl], (n / RING) & 1, ab);
                        if (there && (j < lo || j > hi)) {
#pragma unroll
                            for (int x = 0; x < C::UC / 64; ++x)
#pragma unroll
                                for (int y = 0; y < 8; ++y)
                                    *reinterpret_cast<uint4*>(&s.ring[sl][x * C::CHUNK + key * 128 + y * 16]) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    ok = __all_sync(0xffffffffu, there) && ok;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[buf]);
            }
            // ---------------- epilogue ----------------
            const bool has_o = t1 > t0;
            // whether each group had a tile (of two, group gt & 1 has the item's first)
            const bool had0 = has_o && (NG == 1 || t1 - t0 > 1 || (gt & 1) == 0);
            const bool had1 = NG == 2 && has_o && (t1 - t0 > 1 || (gt & 1) == 1);
            const bool had = grp == 0 ? had0 : had1;
            if (had) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s.pv_done[(g - NG) & 1], ((g - NG) >> 1) & 1, ab)) && ok;
                tc_fence_after();
            }
            gt += max(t1 - t0, 0);
            // the group's sums over its keys: half of the rows to each half of the lanes, and so on, until a
            // lane holds the warp's sums of two rows (64 rows), one (32) or shares one with its neighbour (16)
            {
                float v[NR];
#pragma unroll
                for (int r = 0; r < NR; r += 2) {
                    v[r] = l[r / 2].x;
                    v[r + 1] = l[r / 2].y;
                }
                int o = 16;
#pragma unroll
                for (int n = NR / 2; n >= NR / 32 && n >= 1; n /= 2, o /= 2) {
                    const bool up = lane & o;
#pragma unroll
                    for (int r = 0; r < n; ++r) {
                        const float sent = __shfl_xor_sync(0xffffffffu, up ? v[r] : v[r + n], o);
                        v[r] = (up ? v[r + n] : v[r]) + sent;
                    }
                }
                if constexpr (NR == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
                if constexpr (NR == 64) *reinterpret_cast<float2*>(&grid[NR * sub + 2 * lane]) = make_float2(v[0], v[1]);
                else grid[NR * sub + (NR == 32 ? lane : lane >> 1)] = v[0];
                group_sync(grp);
                if (key < NR) {
                    s.lsum[grp][key] = joined([](float a, float b) { return a + b; }, key);
                    if (!had) s.mref[grp][key] = -INFINITY;
                }
            }
            if (vote_at<3, 128 * NG>(!ok)) break;
            tc_fence_after();
            const int rows = w.rows, part = w.part, gh = w.g, q0 = w.q0;
            const int h0 = grp * GR;  // the group finishes the rows [h0, h0 + GR)
            if (key < GR && h0 + key < rows) {
                const int r = h0 + key;
                const float ma = s.mref[0][r], mb = s.mref[NG - 1][r], m = fmaxf(ma, mb);
                float fa = ma == -INFINITY ? 0.f : ex2(ma - m), fb = NG == 1 || mb == -INFINITY ? 0.f : ex2(mb - m);
                const float sum = s.lsum[0][r] * fa + (NG == 2 ? s.lsum[NG - 1][r] * fb : 0.f);
                if (part >= 0) {
                    a.part_ml[0][(long)part * NR + r] = make_float2(m, sum);
                } else {
                    const int i = (int)((unsigned)(r0 + r) / G), h = gh * p.G + r0 + r - i * p.G;
                    const float s2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
                    const float mf = fmaxf(m, s2);
                    const float wgt = m == -INFINITY ? 0.f : ex2(m - mf);
                    const float lt = sum * wgt + (p.sinks && mf != -INFINITY ? ex2(s2 - mf) : 0.f);
                    const float f = lt != 0.f ? wgt / lt : 0.f;
                    fa *= f;
                    fb *= f;
                    if (a.lse) a.lse[(long)h * p.T_q + q0 + i] = lt != 0.f ? (mf + log2f(lt)) * kLn2 : -INFINITY;
                }
                s.alpha[0][r] = fa;
                if (NG == 2) s.alpha[NG - 1][r] = fb;
            }
            group_sync(grp);
            // O^T to rows: through shared memory (the P buffer), a warp to a row, 4 columns to a lane (in loops:
            // 32 x 16000 keys, d = 64 and 40 rows 128 us, 134 in straight-line code)
#pragma unroll 1
            for (int h = 0; h < C::OH; ++h) {
                if (has_o) {
                    const uint32_t at = tmem + lane_base + cO + NR * h + h0;
                    constexpr int OC = 16 < GR ? 16 : GR;  // rows at a time
#pragma unroll 1
                    for (int y = 0; y < GR; y += OC) {
                        // (an accumulator that no tile went into holds anything)
                        uint32_t o[OC];
                        tmem_ld_cols<OC>(at + y, o);
#pragma unroll
                        for (int r = 0; r < OC; ++r) o[r] = had0 ? __float_as_uint(__uint_as_float(o[r]) * s.alpha[0][h0 + y + r]) : 0u;
                        if constexpr (NG == 2) {
                            uint32_t o1[OC];
                            tmem_ld_cols<OC>(at + C::OH * NR + y, o1);
                            if (had1)
#pragma unroll
                                for (int r = 0; r < OC; ++r)
                                    o[r] = __float_as_uint(fmaf(__uint_as_float(o1[r]), s.alpha[NG - 1][h0 + y + r], __uint_as_float(o[r])));
                        }
#pragma unroll
                        for (int r = 0; r < OC; ++r) grid[(y + r) * kKeyTile + key] = __uint_as_float(o[r]);
                    }
                    if (h == C::OH - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s.o_free);
                    }
                }
                group_sync(grp);
                const bool mine = D == 64 ? lane < 16 : D == 192 && h == 1 ? lane >= 16 : true;
                const int col = (D == 192 ? 64 : 128) * h + 4 * lane;
                if (mine) {
#pragma unroll 1
                    for (int rr = sub; rr < GR && h0 + rr < rows; rr += 4) {
                        const int r = h0 + rr;
                        float4 x = *reinterpret_cast<const float4*>(&grid[rr * kKeyTile + 4 * lane]);
                        if (!has_o || (s.alpha[0][r] == 0.f && s.alpha[NG - 1][r] == 0.f)) x = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (part >= 0) {
                            *reinterpret_cast<float4*>(&a.part_o[0][((long)part * NR + r) * D + col]) = x;
                        } else {
                            const int i = (int)((unsigned)(r0 + r) / G), hh = gh * p.G + r0 + r - i * p.G;
                            uint2 v;
                            v.x = f16 ? pack16<true>(x.x, x.y) : pack16<false>(x.x, x.y);
                            v.y = f16 ? pack16<true>(x.z, x.w) : pack16<false>(x.z, x.w);
                            *reinterpret_cast<uint2*>(&a.o[(((long)q0 + i) * p.h_q + hh) * D + col]) = v;
                        }
                    }
                }
                group_sync(grp);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.item_empty[slot]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------------------------------
// combine: the items that a stretch's end cut
// ------------------------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

// A warp merges R rows of a cut item, from r1 on, from the partials of the CTA c that holds its start
// (slot 1) and of the next ones (their slot 0), in the order of the keys.  The weights are those of
// an online softmax: 2^(m_k - max).
template <int D, bool F16, int R>
__device__ __forceinline__ void merge_rows(const PagedArgs& a, const PagedCut& cut, int which, int c, int r1) {
    constexpr int VW = D / 32;  // columns of a lane, consecutive
    const Problem& p = a.p;
    const int lane = threadIdx.x & 31, held = which ? a.many_rows : a.few_rows;
    // the partials' row of piece y, row r
    auto at = [&](int y, int r) { return (long)(2 * (c + y) + (y == 0 ? 1 : 0)) * held + r; };
    auto load = [&](int y, int z, float2* x) {  // piece y of row r1 + z; a row past the end is the last one again, not stored
        const float2* src = reinterpret_cast<const float2*>(a.part_o[which] + at(y, min(r1 + z, cut.rows - 1)) * D + VW * lane);
#pragma unroll
        for (int e = 0; e < VW / 2; ++e) x[e] = src[e];
    };
    // the first two pieces (there are two at least) are on their way while their weights are worked out
    float2 ahead[2][R][VW / 2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int z = 0; z < R; ++z) load(k, z, ahead[k][z]);
    float m[R], l[R], acc[R][VW];
#pragma unroll
    for (int z = 0; z < R; ++z) {
        m[z] = -INFINITY;
        l[z] = 0.f;
#pragma unroll
        for (int e = 0; e < VW; ++e) acc[z][e] = 0.f;
    }
    for (int y0 = 0; y0 < cut.pieces; y0 += 32) {
        const int y = y0 + lane, cnt = min(32, cut.pieces - y0);
        float wy[R];
#pragma unroll
        for (int z = 0; z < R; ++z) {
            const int r = min(r1 + z, cut.rows - 1);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < cnt) ml = a.part_ml[which][at(y, r)];
            float mx = ml.x;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m[z], mx);
            const float base = mn == -INFINITY ? 0.f : mn, keep = ex2(m[z] - base);
            wy[z] = ex2(ml.x - base);
            float ls = ml.y * wy[z];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            l[z] = l[z] * keep + ls;
            m[z] = mn;
#pragma unroll
            for (int e = 0; e < VW; ++e) acc[z][e] *= keep;
        }
        auto add = [&](int k, int z, const float2* x) {
            const float wk = __shfl_sync(0xffffffffu, wy[z], k);
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) {
                acc[z][2 * e] = fmaf(wk, x[e].x, acc[z][2 * e]);
                acc[z][2 * e + 1] = fmaf(wk, x[e].y, acc[z][2 * e + 1]);
            }
        };
        int k = 0;
        if (y0 == 0)
#pragma unroll
            for (; k < 2; ++k)
#pragma unroll
                for (int z = 0; z < R; ++z) add(k, z, ahead[k][z]);
#pragma unroll 2
        for (; k < cnt; ++k)
#pragma unroll
            for (int z = 0; z < R; ++z) {
                float2 x[VW / 2];
                load(y0 + k, z, x);
                add(k, z, x);
            }
    }
#pragma unroll
    for (int z = 0; z < R; ++z) {
        const int r = r1 + z;
        if (r >= cut.rows) break;
        const int i = (int)((unsigned)(cut.r0 + r) / (unsigned)p.G), h = cut.g * p.G + (cut.r0 + r) - i * p.G;
        const float s2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
        const float mf = fmaxf(m[z], s2);
        const float wgt = m[z] == -INFINITY ? 0.f : ex2(m[z] - mf);
        const float lt = l[z] * wgt + (p.sinks && mf != -INFINITY ? ex2(s2 - mf) : 0.f);
        const float f = lt != 0.f ? wgt / lt : 0.f;
        if (a.lse && lane == 0) a.lse[(long)h * p.T_q + cut.q0 + i] = lt != 0.f ? (mf + log2f(lt)) * kLn2 : -INFINITY;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (((long)cut.q0 + i) * p.h_q + h) * D + VW * lane);
#pragma unroll
        for (int e = 0; e < VW; e += 2) {
            const float x = acc[z][e] * f, y = acc[z][e + 1] * f;
            out[e / 2] = f == 0.f ? 0u : F16 && p.cache8 ? pack_out8<F16>(x, y) : pack16<F16>(x, y);
        }
    }
}

// blockIdx.x: the CTA that holds the start of a cut item.  blockIdx.y numbers the row groups of the
// few-row kernel's items, a row to a warp, then those of the other's, two to a warp: there are many
// of them.  (A decode step of 4 sequences one row 16.5 us, two 17.7; verifying 5 tokens in 32
// sequences 60.7 / 62.0; but a mixed batch with chunks of 387 tokens 69.5 / 64.9.)
constexpr int kFewMergeRows = 1, kManyMergeRows = 2;

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const PagedArgs a, int few_groups) {
    const int warp = threadIdx.x >> 5, c = blockIdx.x, which = (int)blockIdx.y < few_groups ? 0 : 1;
    wait_previous_kernel();
    // (read ahead of the checks: without a stretch, or in a failed call, it holds anything)
    const PagedCut cut = a.cut[which * gridDim.x + c];
    if (c >= a.line[which].n || *reinterpret_cast<volatile const int*>(a.status) != 0) return;
    const int unit = ((int)blockIdx.y - (which ? few_groups : 0)) * kMergeWarps + warp;
    if (which) {
        if (unit * kManyMergeRows < cut.rows) merge_rows<D, F16, kManyMergeRows>(a, cut, 1, c, unit * kManyMergeRows);
    } else {
        if (unit * kFewMergeRows < cut.rows) merge_rows<D, F16, kFewMergeRows>(a, cut, 0, c, unit * kFewMergeRows);
    }
}

template <int D, int NR>
cudaError_t launch_few(const PagedArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t st) {
    constexpr size_t smem = sizeof(FewSmem<D, NR>) + 1024;
    static_assert(smem <= kSmemMax, "the few-row kernel's shared memory");
    cudaError_t e = cudaFuncSetAttribute(paged_few_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (FewCfg<D, NR>::NG == 2) {
        // the warp groups' setmaxnreg shares must fit in the registers the CTA is launched with (an
        // increase beyond them would never be granted)
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, paged_few_kernel<D, NR>)) != cudaSuccess) return e;
        if (fa.numRegs * FewCfg<D, NR>::THREADS < 128 * kFewRegLow + 256 * kFewRegHigh) return cudaErrorLaunchOutOfResources;
    }
    return launch_after(paged_few_kernel<D, NR>, dim3(ctas), FewCfg<D, NR>::THREADS, smem, st, a, tk, tv);
}

template <int D>
cudaError_t launch_few_d(const PagedArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t st) {
    switch (a.few_rows) {
        case 16: return launch_few<D, 16>(a, tk, tv, ctas, st);
        case 32: return launch_few<D, 32>(a, tk, tv, ctas, st);
        case 64: return launch_few<D, 64>(a, tk, tv, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

template <int D>
cudaError_t launch_merge_d(const PagedArgs& a, const dim3& grid, int few_groups, cudaStream_t st) {
    auto kernel = a.p.dtype == FA_DTYPE_F16 ? paged_merge_kernel<D, true> : paged_merge_kernel<D, false>;
    return launch_after(kernel, grid, 32 * kMergeWarps, 0, st, a, few_groups);
}

}  // namespace

cudaError_t launch_paged_prep(const PagedArgs& a, cudaStream_t st) {
    if (a.p.cache8) paged_prep_kernel<kLeadFew8, kLead><<<1, kPrepThreads, 0, st>>>(a);
    else paged_prep_kernel<kLead, kLead><<<1, kPrepThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_few(const PagedArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t st) {
    switch (a.p.d) {
        case 64: return launch_few_d<64>(a, tk, tv, ctas, st);
        case 128: return launch_few_d<128>(a, tk, tv, ctas, st);
        case 192: return launch_few_d<192>(a, tk, tv, ctas, st);
        case 256: return launch_few_d<256>(a, tk, tv, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_paged_merge(const PagedArgs& a, bool many, cudaStream_t st) {
    if (a.few_ctas < 2 || a.no_split) return cudaSuccess;
    const int few_groups = a.few_max > 0 ? cdiv(a.few_rows, kMergeWarps * kFewMergeRows) : 0;
    const dim3 grid(a.few_ctas, few_groups + (many ? cdiv(a.many_rows, kMergeWarps * kManyMergeRows) : 0));
    switch (a.p.d) {
        case 64: return launch_merge_d<64>(a, grid, few_groups, st);
        case 128: return launch_merge_d<128>(a, grid, few_groups, st);
        case 192: return launch_merge_d<192>(a, grid, few_groups, st);
        case 256: return launch_merge_d<256>(a, grid, few_groups, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
