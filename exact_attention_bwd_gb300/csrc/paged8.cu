// Attention of packed queries over a paged e4m3 cache with a scale for each block of tokens and head
// (include/fa.h, fa_params.cache_dtype), few query rows per key/value head.
//
// The true keys and values are K = k8 ks, V = v8 vs, with one ks and vs for 16 keys and more, so the scales
// stay out of the products: ks multiplies the scores, vs the probabilities.  Every e4m3
// value is an fp16 value, and so is a query row once its largest value has been brought near 2^7 by a
// power of two (what falls below fp16's range there is 2^-31 of it and less), so both
// products run on fp16 operands, the first without any rounding, for bf16 queries too.  P vs
// is rounded to fp16 (2^-11, where the 16-bit cache's kernels round P to the inputs' type).
//
// A decode step reads each byte of the cache once and does little with it: what counts is that the
// bytes keep coming.  Each warp streams its own 16 keys of every 128-key tile by TMA copies through a private ring
// and keeps its own online softmax, so the warps wait for each other only where
// an item ends and their states are joined.  With the cache on the long side of the products
// (mma.sync, S^T = K Q^T: 16 keys x 8 rows, O^T = V^T P^T: 16 of d x 8 rows) a tile of 8 rows wastes
// nothing; converted to fp16 in registers, a byte passes shared memory once, where the
// 5th-generation tensor cores would want it stored again as 16-bit operands, five bytes of shared memory
// traffic for each of the cache's, more than the memory's rate leaves.
//
// The contraction's order is free, so the fragments need no transposition on the way from shared memory: a lane
// takes 16 consecutive bytes of a key's row for four k-steps of S^T, and for O^T d / 8
// consecutive columns' bytes of its four keys, which byte permutes pair up.
//
// Rounding: per row a running reference m of the scores (moved where some score passes it by 2^9) and a
// power of two u with P' = P vs u <= 2^9, so that neither blocks of tiny nor of huge values leave fp16's range:
// what a row's product loses is relative to its own largest term.
//
// Measured, decode of 64 requests over 2k to 32k keys, 32 / 8 heads of 128 (1.3 GB, 195 us at the copy rate): 227 to 235 us,
// 5.6 to 5.8 TB/s.  Bound by the memory's path and the ends of items; the arithmetic issues in half of the cycles.
// One warp to a group of keys (8 warps) with 16-byte asynchronous copies 302, two tiles side by side (16 warps) 262,
// their bytes by TMA 256, the table's entry asked for a tile ahead and a lead of 6 units for an item 235.
// Up to 32 rows at d <= 128 and 16 above are this kernel's where the chunks' kernel would be slower over long caches; both sides at the rule
// in api.cu.  (16 and 24 bytes of the widest states are spilled there: <128, 4>, <256, 2>.)
#include "cache8.cuh"
#include "paged.cuh"

namespace fa {
namespace {

constexpr int kGroups8 = 8;                   // 16-key groups of a tile: a warp each
constexpr int kGroup = 16;                    // keys of a warp in a tile: they share a page and a scale
constexpr float kNoRef = -1e30f;              // reference of a row without a key so far
constexpr float kNoUnit = 8.507059173e37f;    // u of a row without a value so far: 2^126
constexpr float kTop = 512.f;                 // P and P vs u stay below

template <int D, int NT>
struct Few8Cfg {
    static constexpr int NR = 8 * NT;
    // tiles side by side (d = 128: above; at d = 64 a mixed batch of short items takes 82 us with two, 76 with one, and
    // beyond that registers or shared memory do not hold 16 warps' states)
    static constexpr int TILES = NT == 1 && D == 128 ? 2 : 1;
    static constexpr int WARPS = kGroups8 * TILES, THREADS = 32 * WARPS;
    static constexpr int GROUP_BYTES = kGroup * D;  // K (or V) rows of a warp's group
    static constexpr int STAGES = D == 64 ? 8 : D == 128 ? (TILES == 2 ? 2 : 5) : D == 192 ? 4 : 3;
    static constexpr int BOX = D % 128 ? 64 : 128, BOXES = D / BOX;  // bytes of a copy's rows (swizzled in as many), copies
    static constexpr int MT = D / 16;               // 16-row tiles of O^T
    static constexpr int MERGE = D <= 128 ? D : NT == 2 ? 32 : 64;  // columns that the warps join at a time
    static constexpr int Q_STRIDE = 2 * D + 16;     // bytes of a query row
    static constexpr bool Q_REGS = NT * D <= 256;   // query fragments held in registers
};

constexpr int kPieces = 16, kLook = 8;  // places for pieces (a power of two), pieces looked ahead for

struct Piece8 {
    int q0, off, nk, r0;     // first query row, nk - nq, keys, first row
    int rows, g, part, t0;   // rows, head, partial slot or -1, first tile
    int t1, in_lo, in_hi, lo;  // end; keys that every row sees; keys that any row sees
    int hi, b, pad[2];       // sequence
};

template <int D, int NT>
struct __align__(1024) Few8Smem {
    using C = Few8Cfg<D, NT>;
    uint8_t ring[C::WARPS][C::STAGES][2][C::GROUP_BYTES];
    uint8_t q[C::NR * C::Q_STRIDE];       // query rows as fp16
    alignas(16) uint16_t raw[C::NR][D];  // those of the next piece as they come
    float merge[C::WARPS][8][C::MERGE];
    float scale[C::WARPS][C::STAGES][2];
    uint64_t full[C::WARPS][C::STAGES];
    int abort_flag;
    float qf[C::NR];                 // the power of two that a query row was divided by
    float m[C::WARPS][C::NR], l[C::WARPS][C::NR], u[C::WARPS][C::NR];  // the warps' states; u becomes the weight of its output
    float f[C::NR];                  // factor of a whole item's output
    Piece8 piece[kPieces];
    int pieces[2];                   // found so far, as of each second meeting
    PagedWalkFew8 walk[32];          // the last warp's walk over the CTA's stretch: a lane's state each
};

// Where chunk `col` of row `row` of a group lies: boxes of 16 rows, 64- or 128-byte swizzled.
template <int D>
__device__ __forceinline__ int at_chunk(int row, int col) {
    constexpr int BOX = Few8Cfg<D, 1>::BOX, PER = BOX / 16;
    return col / PER * (kGroup * BOX) + row * BOX + ((col % PER ^ (BOX == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}
// The key of row g of a fragment (and 8 on, of row g + 8).  The reads of K go two neighbouring rows and four
// chunks at a time, which 128-byte rows then have in different banks.
template <int D>
__device__ __forceinline__ int key_of(int g) {
    return Few8Cfg<D, 1>::BOX == 128 ? g ^ ((g & 1) << 2) : g;
}

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}
// The power of two at or below x (x > 0 and normal).
__device__ __forceinline__ float power_below(float x) { return __uint_as_float(__float_as_uint(x) & 0x7f800000u); }

template <int D, int NT>
__global__ void __launch_bounds__(Few8Cfg<D, NT>::THREADS, 1) paged8_few_kernel(const PagedArgs a, const Cache8 kv, const __grid_constant__ CUtensorMap tmk,
                                                                               const __grid_constant__ CUtensorMap tmv) {
    using C = Few8Cfg<D, NT>;
    constexpr int NR = C::NR, S = C::STAGES, WARPS = C::WARPS, TILES = C::TILES;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Few8Smem<D, NT>& s = *reinterpret_cast<Few8Smem<D, NT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Problem& p = a.p;
    const bool f16 = p.dtype == FA_DTYPE_F16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const unsigned G = (unsigned)p.G;
    allow_next_kernel();
    Abort ab{&s.abort_flag, a.status, p.wait_ns};
    if (tid == 0) s.abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&s.full[warp][i], 3);  // the rows' arrival, and two lanes' copies of scales
        fence_mbar_init();
    }
    wait_previous_kernel();
    // (one thread looks, so that all leave or none)
    if (__syncthreads_or(tid == 0 && (cta >= a.line->n || *reinterpret_cast<volatile int*>(a.status) != 0))) return;

    // ---- the pieces of the CTA's stretch, found by the last warp (the walk's state lies in shared memory: it needs as many
    // registers as an accumulator tile of 16 rows) ----
    int found = 0;
    bool more = true;
    auto find = [&](int most) {
        PagedWalkFew8 walk = s.walk[lane];
        const PagedLine line = *a.line;
        while (more && found < most) {
            if (!(more = walk.next(p, a.pre, line, cta, NR, a.no_split))) break;
            const PagedSeq& sq = walk.seq;
            const int r0 = walk.x.rt * NR, rows = min(NR, sq.nq * p.G - r0), off = sq.nk - sq.nq;
            const int i0 = (int)((unsigned)r0 / G), i1 = (int)((unsigned)(r0 + rows - 1) / G);
            if (walk.t1 > walk.t0) {
                if (lane == 0) {
                    const Band bd{off, p.left, p.right, sq.nk};
                    Piece8& x = s.piece[found % kPieces];
                    x.q0 = sq.q0;
                    x.off = off;
                    x.nk = sq.nk;
                    x.r0 = r0;
                    x.rows = rows;
                    x.g = walk.x.g;
                    x.part = walk.from_start && walk.to_end ? -1 : 2 * cta + (walk.from_start ? 1 : 0);
                    x.t0 = walk.t0;
                    x.t1 = walk.t1;
                    x.b = walk.b;
                    x.lo = bd.lo(i0);
                    x.hi = bd.hi(i1);
                    x.in_lo = p.left >= 0 ? i1 + off - p.left : 0;
                    x.in_hi = p.right >= 0 ? min(sq.nk - 1, i0 + off + p.right) : sq.nk - 1;
                }
                ++found;
            } else {
                // no key for any row (such a piece is whole): its rows are written here
                for (int r = 0; r < rows; ++r) {
                    const int i = (int)((unsigned)(r0 + r) / G), h = walk.x.g * p.G + r0 + r - i * p.G;
                    uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (((long)sq.q0 + i) * p.h_q + h) * D);
                    for (int x = lane; x < D / 2; x += 32) out[x] = 0u;
                    if (lane == 0 && a.lse) a.lse[(long)h * p.T_q + sq.q0 + i] = p.sinks ? p.sinks[h] : -INFINITY;
                }
            }
        }
        s.walk[lane] = walk;
        if (!more && lane == 0) a.cut[cta] = walk.cut;
    };
    if (warp == WARPS - 1) {
        PagedWalkFew8 walk;
        walk.start(p, a.pre, a.line, cta);
        s.walk[lane] = walk;
        find(2);
        if (lane == 0) s.pieces[0] = found;
    }

    // ---- a warp's 16 keys of every TILES-th tile ----
    const int lg = lane >> 2, lt = lane & 3;  // a fragment's row (or column) and its pair
    const int group = warp % kGroups8, side = warp / kGroups8;
    // the warp's stream: tiles of one piece after another, S of them ahead of the arithmetic
    int at_t = 0, end_t = 0;           // of the piece that is being fetched
    int ahead = 0, known = 0;          // pieces begun to be fetched, found
    int b_lo = 0, b_hi = 0, b_g = 0;   // its keys that any row sees, its head
    const int32_t* table = nullptr;
    int issued = 0;
    int st_in = 0;                       // stage to be filled
    uint32_t filled = 0, phase = 0;      // stages with copies on their way or not yet read, parities that they complete
    // looks at the next tile: the warp's keys' entry of the table is on its way until the tile's copies are started
    bool looked = false, mine = false;
    int entry = 0, row = 0;
    auto look = [&]() {
        if (at_t >= end_t && ahead < known) {
            const Piece8& x = s.piece[ahead++ % kPieces];
            at_t = x.t0;
            end_t = x.t1;
            b_g = x.g;
            b_lo = x.lo;
            b_hi = x.hi;
            table = p.block_table + (long)x.b * p.max_blocks;
        }
        looked = at_t < end_t;
        if (looked) {
            const int j0 = (at_t + side) * kKeyTile + kGroup * group;
            mine = at_t + side < end_t && j0 <= b_hi && j0 + kGroup > b_lo;
            if (mine) {
                const int at = quotient(j0, kv.by_page);
                entry = table[at];
                row = j0 - at * p.page_size;
            }
        }
    };
    auto fetch = [&]() {
        if (!looked) look();
        if (looked) {
            if (mine) {
                const int page = entry;
                const bool there = (unsigned)page < (unsigned)a.num_pages;
                uint64_t* bar = &s.full[warp][st_in];
                if (lane < 2) {
                    if (there)
                        copy4_async(&s.scale[warp][st_in][lane], (lane ? kv.v_scale : kv.k_scale) +
                                    ((long)page * kv.blocks + quotient(row, kv.by_block)) * p.h_kv + b_g);
                    mbar_arrive_copies(bar);
                }
                if (lane == 0) {
                    if (!there) atomicCAS(a.status, 0, kStatusDeviceCheck);
                    mbar_expect_tx(bar, 2 * C::GROUP_BYTES);
#pragma unroll
                    for (int x = 0; x < C::BOXES; ++x) {  // (the pool's end reads as zeros)
                        tma_load_4d(&s.ring[warp][st_in][0][x * kGroup * C::BOX], &tmk, bar, x * C::BOX, b_g, row, there ? page : a.num_pages);
                        tma_load_4d(&s.ring[warp][st_in][1][x * kGroup * C::BOX], &tmv, bar, x * C::BOX, b_g, row, there ? page : a.num_pages);
                    }
                }
                filled |= 1u << st_in;
            }
            st_in = st_in + 1 == S ? 0 : st_in + 1;
            at_t += TILES;
            ++issued;
            look();
        }
    };

    // The query rows of a piece: asked for a piece ahead, turned to fp16 where the piece before ends (a warp its own).
    auto ask = [&](const Piece8& x) {
        for (int r = warp; r < NR; r += WARPS) {
            const int i = (int)((unsigned)(x.r0 + r) / G), h = x.g * p.G + x.r0 + r - i * p.G;
            const uint16_t* src = r < x.rows ? a.q + (((long)x.q0 + i) * p.h_q + h) * D : a.q;
            if (lane < D / 8) copy16_async(&s.raw[r][8 * lane], src + 8 * lane, r < x.rows);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    auto take = [&]() {
        asm volatile("cp.async.wait_group 0;\n" ::: "memory");  // (not for the scales' copies since, which are in no group)
        __syncwarp();
        for (int r = warp; r < NR; r += WARPS) {
            float top = 0.f;
            float2 v[D / 64];
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(&s.raw[r][2 * (lane + 32 * e)]);
                v[e] = f16 ? make_float2(lo16<true>(x), hi16<true>(x)) : make_float2(lo16<false>(x), hi16<false>(x));
                top = fmaxf(top, fmaxf(fabsf(v[e].x), fabsf(v[e].y)));
            }
            top = warp_max(top);
            // (rows of zeros, or with infinities, are left as they are)
            const float unit = top >= 1e-30f && top < INFINITY ? power_below(top) * 0x1p-7f : 1.f, inv = 1.f / unit;
#pragma unroll
            for (int e = 0; e < D / 64; ++e)
                *reinterpret_cast<uint32_t*>(&s.q[r * C::Q_STRIDE + 4 * (lane + 32 * e)]) = pack16<true>(v[e].x * inv, v[e].y * inv);
            if (lane == 0) s.qf[r] = unit * p.scale_log2;
        }
        __syncwarp();
    };

    int done = 0, st = 0;  // tiles, stage of the next
    bool ok = true;
    __syncthreads();
    known = s.pieces[0];
    if (known > 0) {
        ask(s.piece[0]);
        while (issued < S && (at_t < end_t || ahead < known)) fetch();
        take();
    }
#pragma unroll 1
    for (int piece = 0;; ++piece) {
        // (the pieces found are there; the rows and states of the piece before have been read; one warp that gave up ends all)
        if (__syncthreads_or(!ok)) break;
        known = s.pieces[piece & 1];
        if (piece >= known) break;
        while (issued < done + S && (at_t < end_t || ahead < known)) fetch();
        const Piece8 w = s.piece[piece % kPieces];
        if (piece + 1 < known) ask(s.piece[(piece + 1) % kPieces]);
        // ---- state: rows 8 n + 2 lt and 8 n + 2 lt + 1 ----
        float m[NT][2], u[NT][2], l[NT][2], qf[NT][2], acc[C::MT][NT][4];
        uint4 qr[C::Q_REGS ? NT : 1][D / 64][2];
        auto q_frag = [&](int n, int i, int h) {
            return *reinterpret_cast<const uint4*>(&s.q[(8 * n + lg) * C::Q_STRIDE + 32 * (lt + 4 * i) + 16 * h]);
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = kNoRef;
                u[n][e] = kNoUnit;
                l[n][e] = 0.f;
                qf[n][e] = s.qf[8 * n + 2 * lt + e];
            }
            if constexpr (C::Q_REGS) {
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) qr[n][i][h] = q_frag(n, i, h);
            }
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[x][n][e] = 0.f;
        }
#pragma unroll 1
        for (int t = w.t0; t < w.t1; t += TILES, ++done, st = st + 1 == S ? 0 : st + 1) {
            const int j0 = (t + side) * kKeyTile + kGroup * group;
            if (t + side < w.t1 && j0 <= w.hi && j0 + kGroup > w.lo) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait_copy(&s.full[warp][st], (phase >> st) & 1, ab)))) break;
                phase ^= 1u << st;
                filled &= ~(1u << st);
                const uint8_t *k8 = s.ring[warp][st][0], *v8 = s.ring[warp][st][1];
                const float ks = s.scale[warp][st][0], vs = s.scale[warp][st][1];
                // ---- S^T = K Q^T ----
                float sc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const uint4 ka = *reinterpret_cast<const uint4*>(k8 + at_chunk<D>(key_of<D>(lg), lt + 4 * i));
                    const uint4 kb = *reinterpret_cast<const uint4*>(k8 + at_chunk<D>(key_of<D>(lg) + 8, lt + 4 * i));
                    uint4 q0[NT], q1[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        q0[n] = C::Q_REGS ? qr[C::Q_REGS ? n : 0][i][0] : q_frag(n, i, 0);
                        q1[n] = C::Q_REGS ? qr[C::Q_REGS ? n : 0][i][1] : q_frag(n, i, 1);
                    }
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t a0 = widen_e4m3x2<false>(wa[x]), a1 = widen_e4m3x2<false>(wb[x]), a2 = widen_e4m3x2<true>(wa[x]), a3 = widen_e4m3x2<true>(wb[x]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4& qq = x < 2 ? q0[n] : q1[n];
                            mma16816(sc[n], a0, a1, a2, a3, x & 1 ? qq.z : qq.x, x & 1 ? qq.w : qq.y);
                        }
                    }
                }
                // ---- scores in log2 units; keys j0 + key_of(lg) and 8 on ----
                const bool edge = j0 < w.in_lo || j0 + kGroup - 1 > w.in_hi;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float c0 = qf[n][0] * ks, c1 = qf[n][1] * ks;
                    sc[n][0] *= c0;
                    sc[n][1] *= c1;
                    sc[n][2] *= c0;
                    sc[n][3] *= c1;
                }
                if (edge) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = j0 + key_of<D>(lg) + 8 * h;
                        // rows [ra, rb] see key j: positions j - off - right <= i <= j - off + left
                        int ra = 0, rb = NR - 1;
                        if (p.right >= 0) ra = (int)max(min(((long)j - w.off - p.right) * p.G - w.r0, (long)NR), 0l);
                        if (p.left >= 0) rb = (int)min(max(((long)j - w.off + p.left + 1) * p.G - 1 - w.r0, -1l), (long)NR);
                        if (j >= w.nk) ra = NR;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int r = 8 * n + 2 * lt + e;
                                if (r < ra || r > rb) sc[n][2 * h + e] = -INFINITY;
                            }
                    }
                }
                // ---- P = 2^(x - m), P' = P vs u ----
                float pr[NT][4], over = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        pr[n][e] = ex2(sc[n][e] - m[n][e]);
                        pr[n][2 + e] = ex2(sc[n][2 + e] - m[n][e]);
                        over = fmaxf(over, fmaxf(pr[n][e], pr[n][2 + e]) * fmaxf(1.f, vs * u[n][e]));
                    }
                if (__any_sync(0xffffffffu, over > kTop)) {
                    // some row's reference or unit moves: to the maxima so far
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = fmaxf(sc[n][e], sc[n][2 + e]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            const float mo = m[n][e], mn = fmaxf(mo, top), keep = ex2(mo - mn);
                            // the largest term so far, at 1 / u in units of the old reference, and of these keys
                            const float most = fmaxf(keep / u[n][e], ex2(top - mn) * vs);
                            const float un = most > 0x1p-126f && most < INFINITY ? 1.f / power_below(most) : kNoUnit;
                            // (un / u alone may pass fp32's range, and 0 * inf would be NaN; keep / u is one of the terms of `most`)
                            const float by = un / u[n][e], f = by < INFINITY ? keep * by : keep / u[n][e] * un;
                            m[n][e] = mn;
                            l[n][e] *= keep;
                            u[n][e] = un;
#pragma unroll
                            for (int x = 0; x < C::MT; ++x) {
                                acc[x][n][e] *= f;
                                acc[x][n][2 + e] *= f;
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) pr[n][2 * h + e] = ex2(sc[n][2 * h + e] - mn);
                        }
                }
                uint32_t pb[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    l[n][0] += pr[n][0] + pr[n][2];
                    l[n][1] += pr[n][1] + pr[n][3];
                    // (vs u may pass fp32's range where P is small, or 0 in a row without a value so far: P vs first, then)
                    float f0 = vs * u[n][0], f1 = vs * u[n][1];
                    if (f0 > 0x1p100f) {
                        pr[n][0] *= vs;
                        pr[n][2] *= vs;
                        f0 = u[n][0];
                    }
                    if (f1 > 0x1p100f) {
                        pr[n][1] *= vs;
                        pr[n][3] *= vs;
                        f1 = u[n][1];
                    }
                    pb[n][0] = transpose8x8(pack16<true>(pr[n][0] * f0, pr[n][1] * f1));
                    pb[n][1] = transpose8x8(pack16<true>(pr[n][2] * f0, pr[n][3] * f1));
                }
                // ---- O^T += V^T P^T: the lane's columns are [lg D / 8, (lg + 1) D / 8), its keys 2 lt, 2 lt + 1 and those + 8 ----
                constexpr int WORDS = D / 32;  // 4-byte words of the lane's columns
                uint32_t vw[4][WORDS];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int r = key_of<D>(2 * lt + (y & 1)) + 8 * (y >> 1);
                    if constexpr (D >= 128 && D != 192) {
#pragma unroll
                        for (int z = 0; z < WORDS / 4; ++z) {
                            const uint4 x = *reinterpret_cast<const uint4*>(v8 + at_chunk<D>(r, lg * (WORDS / 4) + z));
                            vw[y][4 * z] = x.x;
                            vw[y][4 * z + 1] = x.y;
                            vw[y][4 * z + 2] = x.z;
                            vw[y][4 * z + 3] = x.w;
                        }
                    } else {
#pragma unroll
                        for (int z = 0; z < WORDS / 2; ++z) {
                            const int byte = lg * (D / 8) + 8 * z;
                            const uint2 x = *reinterpret_cast<const uint2*>(v8 + at_chunk<D>(r, byte >> 4) + (byte & 8));
                            vw[y][2 * z] = x.x;
                            vw[y][2 * z + 1] = x.y;
                        }
                    }
                }
                if (edge) {
                    // (values that no query sees may be anything, and 0 * NaN is NaN)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int j = j0 + key_of<D>(2 * lt + (y & 1)) + 8 * (y >> 1);
                        if (j < w.lo || j > w.hi)
#pragma unroll
                            for (int z = 0; z < WORDS; ++z) vw[y][z] = 0u;
                    }
                }
#pragma unroll
                for (int z = 0; z < WORDS; ++z)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = __byte_perm(vw[0][z], vw[1][z], h ? 0x7362 : 0x5140);
                        const uint32_t y = __byte_perm(vw[2][z], vw[3][z], h ? 0x7362 : 0x5140);
                        const uint32_t a0 = widen_e4m3x2<false>(x), a1 = widen_e4m3x2<true>(x), a2 = widen_e4m3x2<false>(y), a3 = widen_e4m3x2<true>(y);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(acc[2 * z + h][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    }
            }
            __syncwarp();  // the stage has been read
            fetch();
        }
        // ---- the warps' states join ----
        // (the next piece's rows, asked for ahead of the tiles, have long been there: each warp's wait covers its own)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
                if (lg == 0) {
                    const int r = 8 * n + 2 * lt + e;
                    s.m[warp][r] = m[n][e];
                    s.l[warp][r] = l[n][e];
                    s.u[warp][r] = u[n][e];
                }
            }
        __syncthreads();
        if (piece + 1 < known) take();
        if (tid < NR) {
            float top = kNoRef, sum = 0.f;
#pragma unroll
            for (int x = 0; x < WARPS; ++x) top = fmaxf(top, s.m[x][tid]);
#pragma unroll
            for (int x = 0; x < WARPS; ++x) {
                const float keep = ex2(s.m[x][tid] - top);
                sum += s.l[x][tid] * keep;
                s.u[x][tid] = keep / s.u[x][tid];
            }
            if (top <= 0.5f * kNoRef) top = -INFINITY;
            if (tid < w.rows) {
                if (w.part >= 0) {
                    a.part_ml[0][(long)w.part * NR + tid] = make_float2(top, sum);
                    s.f[tid] = 1.f;
                } else {
                    const int i = (int)((unsigned)(w.r0 + tid) / G), h = w.g * p.G + w.r0 + tid - i * p.G;
                    const float s2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
                    const float mf = fmaxf(top, s2);
                    const float wgt = top == -INFINITY ? 0.f : ex2(top - mf);
                    const float lt2 = sum * wgt + (p.sinks && mf != -INFINITY ? ex2(s2 - mf) : 0.f);
                    s.f[tid] = lt2 != 0.f ? wgt / lt2 : 0.f;
                    if (a.lse) a.lse[(long)h * p.T_q + w.q0 + i] = lt2 != 0.f ? (mf + log2f(lt2)) * kLn2 : -INFINITY;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float w0 = s.u[warp][8 * n + 2 * lt], w1 = s.u[warp][8 * n + 2 * lt + 1];
            // (MERGE columns at a time: of each lane's D / 8 columns MERGE / 8)
            constexpr int EACH = C::MERGE / 8;
#pragma unroll
            for (int y = 0; y < D / C::MERGE; ++y) {
                if (n + y > 0) __syncthreads();
#pragma unroll
                for (int x = 0; x < EACH / 2; ++x) {
                    const float* c = acc[EACH / 2 * y + x][n];
                    *reinterpret_cast<float2*>(&s.merge[warp][2 * lt][EACH * lg + 2 * x]) = make_float2(c[0] * w0, c[2] * w0);
                    *reinterpret_cast<float2*>(&s.merge[warp][2 * lt + 1][EACH * lg + 2 * x]) = make_float2(c[1] * w1, c[3] * w1);
                }
                __syncthreads();
                // a warp to a row and 64 columns
#pragma unroll
                for (int z = warp; z < 8 * ((C::MERGE + 63) / 64); z += WARPS) {
                    const int rr = z & 7, r = 8 * n + rr, at = 64 * (z >> 3) + 2 * lane;
                    if (r >= w.rows || at >= C::MERGE) continue;
                    float2 o = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < WARPS; ++x) o = __fadd2_rn(o, *reinterpret_cast<const float2*>(&s.merge[x][rr][at]));
                    const float f = s.f[r];
                    const int col = at / EACH * (D / 8) + EACH * y + at % EACH;
                    if (w.part >= 0) {
                        *reinterpret_cast<float2*>(&a.part_o[0][((long)w.part * NR + r) * D + col]) = o;
                    } else {
                        const int i = (int)((unsigned)(w.r0 + r) / G), h = w.g * p.G + w.r0 + r - i * p.G;
                        const float ox = f == 0.f ? 0.f : o.x * f, oy = f == 0.f ? 0.f : o.y * f;
                        *reinterpret_cast<uint32_t*>(&a.o[(((long)w.q0 + i) * p.h_q + h) * D + col]) =
                            f16 ? pack_out8<true>(ox, oy) : pack_out8<false>(ox, oy);
                    }
                }
            }
        }
        if (warp == WARPS - 1) {  // one or two pieces on
            if (more) find(min(piece + kLook, found + 2));
            if (lane == 0) s.pieces[(piece + 1) & 1] = found;
        }
    }
    // (given up: every copy still in flight lands before the CTA may exit)
    for (int i = 0; i < S; ++i)
        if ((filled >> i) & 1) mbar_wait_quiet(&s.full[warp][i], (phase >> i) & 1);
}

template <int D, int NT>
cudaError_t launch_few8(const PagedArgs& a, const Cache8& kv, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t st) {
    constexpr size_t smem = sizeof(Few8Smem<D, NT>) + 1024;
    static_assert(smem <= 227 * 1024, "the few-row kernel's shared memory");
    cudaError_t e = cudaFuncSetAttribute(paged8_few_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(paged8_few_kernel<D, NT>, dim3(ctas), Few8Cfg<D, NT>::THREADS, smem, st, a, kv, tk, tv);
}

template <int D>
cudaError_t launch_few8_d(const PagedArgs& a, const Cache8& kv, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t st) {
    switch (a.few_rows) {
        case 8: return launch_few8<D, 1>(a, kv, tk, tv, ctas, st);
        case 16: return launch_few8<D, 2>(a, kv, tk, tv, ctas, st);
        case 32:
            if constexpr (D <= 128) return launch_few8<D, 4>(a, kv, tk, tv, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_paged8_few(const PagedArgs& a, const Cache8& kv, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t st) {
    switch (a.p.d) {
        case 64: return launch_few8_d<64>(a, kv, tk, tv, ctas, st);
        case 128: return launch_few8_d<128>(a, kv, tk, tv, ctas, st);
        case 192: return launch_few8_d<192>(a, kv, tk, tv, ctas, st);
        case 256: return launch_few8_d<256>(a, kv, tk, tv, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
