// A paged cache in 8 bits on its way to the 5th-generation tensor cores: half tiles of 64 keys' e4m3
// bytes with their blocks' scales in a ring in shared memory, filled by one warp's TMA copies, emptied by four
// warps that write the 16-bit operand tiles (128-byte-swizzled chunks of 64 columns).
#pragma once
#include <type_traits>

#include "common.cuh"

namespace fa {

// The pages of a tile of TILE keys, 16 rows to a lane, worked out a tile ahead (one warp).
template <int TILE>
struct Pages8 {
    static constexpr int GROUPS = TILE / 16;
    const Cache8& c;
    const Problem& p;
    const int32_t* table;
    int num_pages, lo, hi;  // keys that any query of the item sees
    int ahead_page = 0, ahead_row = 0, ahead_block = 0;  // of the next tile
    int page = 0, row = 0;                               // page of the lane's rows, first row in it
    long scale = 0;                                      // place of their scale, head 0 (-1: none)
    __device__ __forceinline__ Pages8(const Cache8& c_, const Problem& p_, const int32_t* t, int pages, int lo_, int hi_)
        : c(c_), p(p_), table(t), num_pages(pages), lo(lo_), hi(hi_) {}
    __device__ __forceinline__ void look(int t, int end) {
        const int lane = threadIdx.x & 31, key = t * TILE + 16 * lane, at = quotient(key, c.by_page);
        ahead_page = lane < GROUPS && t < end && key <= hi ? table[at] : num_pages;
        ahead_row = key - at * p.page_size;
        ahead_block = quotient(ahead_row, c.by_block);
    }
    // Tile t is the one to load.  A lane's page is the pool's end, which reads as zeros, past the keys that are seen and for
    // an entry outside the pool, which sets the status if any of the lane's keys is seen.
    __device__ __forceinline__ void take(int t, int end, int* status) {
        const int lane = threadIdx.x & 31;
        page = ahead_page;
        row = ahead_row;
        if (lane < GROUPS && (unsigned)page >= (unsigned)num_pages) {
            const int key = t * TILE + 16 * lane;
            if (key <= hi && key + 16 > lo) atomicCAS(status, 0, kStatusDeviceCheck);
            page = num_pages;
        }
        scale = page < num_pages ? ((long)page * c.blocks + ahead_block) * p.h_kv : -1;
        look(t + 1, end);
    }
};

// Powers of two that bring the largest scales of an item's keys and of their values to at most 2^7 (and more than 2^6), so that
// every e4m3 value times its scale fits fp16 wherever the cache's values lie: (keys, values).  What is 2^-22 of
// the item's largest scale and more is exact where the scales are powers of two, and what is less loses the bits below 2^-31 of it.
// [lo, hi] are the keys that any row of the item sees (a whole warp; four looks at the table and the scales in flight).
struct Fit8 {
    float key, value;
    static __device__ __forceinline__ float power(float most) {
        const uint32_t x = __float_as_uint(most), e = (x >> 23) + ((x & 0x7fffffu) ? 1 : 0);  // most <= 2^(e - 127)
        return most > 0.f ? __uint_as_float(min(261u - e, 223u) << 23) : 1.f;                 // 2^-121 to 2^96
    }
    static __device__ __forceinline__ float inverse(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }
    __device__ __forceinline__ void look(const Cache8& c, const Problem& p, const int32_t* table, int num_pages, int g, int lo, int hi) {
        float k = 0.f, v = 0.f;
        if (lo <= hi) {
            const int last = quotient(hi, c.by_block);
#pragma unroll 4
            for (int b = quotient(lo, c.by_block) + (threadIdx.x & 31); b <= last; b += 32) {
                const int at = quotient(b * c.block, c.by_page), page = table[at];
                if ((unsigned)page < (unsigned)num_pages) {
                    const long x = ((long)page * c.blocks + quotient(b * c.block - at * p.page_size, c.by_block)) * p.h_kv + g;
                    k = fmaxf(k, c.k_scale[x]);
                    v = fmaxf(v, c.v_scale[x]);
                }
            }
        }
        key = power(warp_max(k));
        value = power(warp_max(v));
    }
};

// Two e4m3 bytes (the low or the high half of a word) as an fp16 pair, the lower byte low.
template <bool HI>
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t w) {
    uint32_t r;
    if constexpr (HI) asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(w));
    else asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(w));
    return r;
}

// A pair of an output's values in the 16-bit type.  fp16: kept within its range (NaN stays NaN), for a value near its
// largest may stand in the cache as the next e4m3 value above, which fp16 rounds to infinity.
template <bool F16>
__device__ __forceinline__ uint32_t pack_out8(float x, float y) {
    if constexpr (F16) {
        uint32_t r;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
        return r;
    }
    return pack16<F16>(x, y);
}

// Two e4m3 bytes times a scale, in the 16-bit type.
template <bool F16, bool HI>
__device__ __forceinline__ uint32_t scaled_e4m3x2(uint32_t w, float scale) {
    const uint32_t h = widen_e4m3x2<HI>(w);
    const float2 x = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h)), make_float2(scale, scale));
    return pack16<F16>(x.x, x.y);
}

template <int D, int UNITS>
struct Ring8 {
    static constexpr int ROWS = 64, CPR = D / 16;  // rows of a unit, 16-byte chunks of a row
    alignas(128) uint8_t rows[UNITS][ROWS * D];
    float scale[UNITS][ROWS / 16];
    uint64_t full[UNITS], empty[UNITS];

    __device__ __forceinline__ void init() {
        for (int i = 0; i < UNITS; ++i) {
            mbar_init(&full[i], 33);  // the bytes' arrival, and each lane's copies of scales
            mbar_init(&empty[i], 4);  // a converting warp each
        }
    }
    // Starts the loads of half h of the tile that `pages` holds, boxes of 16 << log_box rows (a whole warp).
    template <int TILE>
    __device__ __forceinline__ bool load(uint32_t& n, const Pages8<TILE>& pages, int h, int log_box, const CUtensorMap& map,
                                         const float* scales, int g, const Abort& ab) {
        const int lane = threadIdx.x & 31, st = n % UNITS;
        const long at = __shfl_sync(0xffffffffu, pages.scale, 4 * h + (lane & 3));  // lane x < 4: of rows 16 x and on
        const int src = 4 * h + ((lane << log_box) & 3);                            // lane x < 4 >> log_box: of box x
        const int page = __shfl_sync(0xffffffffu, pages.page, src), row = __shfl_sync(0xffffffffu, pages.row, src);
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ((n / UNITS) & 1) ^ 1, ab))) return false;
        if (lane == 0) mbar_expect_tx(&full[st], ROWS * D);
        __syncwarp();
        if (lane < 4 >> log_box) tma_load_4d(&rows[st][((lane << log_box) * 16) * D], &map, &full[st], 0, g, row, page);
        if (lane < 4 && at >= 0) copy4_async(&scale[st][lane], scales + at + g);
        mbar_arrive_copies(&full[st]);
        ++n;
        return true;
    }
    // Every load still in flight lands.
    __device__ __forceinline__ void drain(uint32_t n) {
        for (uint32_t back = 1; back <= UNITS && back <= n; ++back) mbar_wait_quiet(&full[(n - back) % UNITS], ((n - back) / UNITS) & 1);
    }
    // Rows 16 w and on of the next unit, keys j0 + 16 w and on, to rows of a tile (zeros outside the keys [lo, hi] that
    // any query sees: what lies there may be anything).  A lane turns 16 bytes into two 16-byte units, four times over
    // with their loads ahead; every other group of four chunks takes its second half first (swap_of), so that the
    // stores of a phase, and the loads where a row is a power of two, fall into different banks.  What no query sees
    // is cleared as bytes, in a branch of its own: conversions share the issue slots with the softmax, and a second copy
    // of them for edges costs more in instruction fetches than it saves (8 chunks of 1024 tokens at d = 128, 785 us, took 885
    // with it; 32 x 5 tokens at d = 256 72, 77 with outputs selected, 80 two chunks at a time and 92 eight).
    // fp16: scales times `by` (Fit8).
    template <bool F16>
    __device__ __forceinline__ bool widen(uint32_t& n, int w, uint8_t* tile, int chunk_bytes, int j0, int lo, int hi, float by,
                                          const Abort& ab) {
        constexpr int ALL = CPR / 2, BATCH = ALL % 4 == 0 ? 4 : ALL < 4 ? ALL : 3;  // chunks of a lane
        const int lane = threadIdx.x & 31, st = n % UNITS;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (n / UNITS) & 1, ab))) return false;
        // (a group that no query sees may have any scale)
        const float f = j0 + 16 * w <= hi && j0 + 16 * w + 15 >= lo ? (F16 ? scale[st][w] * by : scale[st][w]) : 0.f;
        const uint8_t* from = &rows[st][16 * w * D];
        const bool inside = j0 + 16 * w >= lo && j0 + 16 * w + 15 <= hi;
        auto swap_of = [](int x) { return (D == 64 ? x >> 3 : D == 192 ? (x % CPR) >> 2 : (x >> 2) ^ (x >> 3)) & 1; };
#pragma unroll 1
        for (int y0 = 0; y0 < ALL; y0 += BATCH) {
            uint2 b[BATCH][2];
#pragma unroll
            for (int y = 0; y < BATCH; ++y) {
                const int x = lane + 32 * (y0 + y), swap = swap_of(x);
                b[y][0] = *reinterpret_cast<const uint2*>(from + 16 * x + 8 * swap);
                b[y][1] = *reinterpret_cast<const uint2*>(from + 16 * x + 8 - 8 * swap);
            }
            if (!inside) {
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    const int j = j0 + 16 * w + (lane + 32 * (y0 + y)) / CPR;
                    if (j < lo || j > hi) b[y][0] = b[y][1] = make_uint2(0, 0);
                }
            }
#pragma unroll
            for (int y = 0; y < BATCH; ++y) {
                const int x = lane + 32 * (y0 + y), r = 16 * w + x / CPR, c = x % CPR, u = 2 * (c & 3), swap = swap_of(x);
                uint8_t* to = tile + (c >> 2) * chunk_bytes + r * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 o = make_uint4(scaled_e4m3x2<F16, false>(b[y][h].x, f), scaled_e4m3x2<F16, true>(b[y][h].x, f),
                                         scaled_e4m3x2<F16, false>(b[y][h].y, f), scaled_e4m3x2<F16, true>(b[y][h].y, f));
                    *reinterpret_cast<uint4*>(to + (((u + (swap ^ h)) ^ (r & 7)) << 4)) = o;
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        ++n;
        return true;
    }
};

}  // namespace fa
