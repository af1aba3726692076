// A paged cache in 8 bits on its way to the 5th-generation tensor cores: half tiles of 64 keys' e4m3
// bytes with their blocks' scales in a ring in shared memory, filled by one warp's TMA copies, emptied by four
// warps that write the 16-bit operand tiles (128-byte-swizzled chunks of 64 columns).
#pragma once
#include <type_traits>

#include "common.cuh"

namespace fa {

// The pages of a 128-key tile, a box of rows to a lane, the next tile's table entries fetched ahead (one warp).
struct Pages8 {
    const Cache8& c;
    const Problem& p;
    const int32_t* table;
    int num_pages, box, nk;
    int next = 0, page = 0, row = 0, tile = 0;
    __device__ __forceinline__ Pages8(const Cache8& c_, const Problem& p_, const int32_t* t, int pages, int box_, int nk_)
        : c(c_), p(p_), table(t), num_pages(pages), box(box_), nk(nk_) {}
    __device__ __forceinline__ int entry(int t, int end) const {
        const int lane = threadIdx.x & 31, j = t * 128 + lane * box;
        return lane < 128 / box && t < end && j < nk ? table[j / p.page_size] : num_pages;
    }
    __device__ __forceinline__ void look(int t, int end) { next = entry(t, end); }
    // tile t is the one to load; lane x then holds box x's page (the pool's end, which reads as zeros, past the used
    // keys and for an entry outside the pool, which sets the status) and first row
    __device__ __forceinline__ void take(int t, int end, int* status) {
        const int lane = threadIdx.x & 31, key = t * 128 + lane * box;
        page = next;
        next = entry(t + 1, end);
        tile = t;
        row = key % p.page_size;
        if (lane < 128 / box && (unsigned)page >= (unsigned)num_pages) {
            if (key < nk) atomicCAS(status, 0, kStatusDeviceCheck);
            page = num_pages;
        }
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

// Two e4m3 bytes times a scale, in the 16-bit type.  (fp16: kept within its range, so that a finite
// value does not become infinite where the scale was rounded up.)
template <bool F16, bool HI>
__device__ __forceinline__ uint32_t scaled_e4m3x2(uint32_t w, float scale) {
    const uint32_t h = widen_e4m3x2<HI>(w);
    float2 x = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h)), make_float2(scale, scale));
    if constexpr (F16) {
        x.x = x.x > 65504.f ? 65504.f : x.x < -65504.f ? -65504.f : x.x;  // (NaN stays)
        x.y = x.y > 65504.f ? 65504.f : x.y < -65504.f ? -65504.f : x.y;
    }
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
    // Starts the loads of half h of the tile that `pages` holds (a whole warp).
    __device__ __forceinline__ bool load(uint32_t& n, const Pages8& pages, int h, const CUtensorMap& map, const float* scales, int g,
                                         const Abort& ab) {
        const int lane = threadIdx.x & 31, st = n % UNITS;
        const int box = min(pages.box, ROWS), step = pages.box / box;  // (a page's 128 rows: two copies)
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ((n / UNITS) & 1) ^ 1, ab))) return false;
        if (lane == 0) mbar_expect_tx(&full[st], ROWS * D);
        // lane x < 4: the scale of rows 16 x and on
        const int at = 64 * h + 16 * (lane & 3), from = at / pages.box;
        const int page = __shfl_sync(0xffffffffu, pages.page, from), row = __shfl_sync(0xffffffffu, pages.row, from) + at % pages.box;
        if (lane < 4 && page < pages.num_pages)
            copy4_async(&scale[st][lane], scales + ((long)page * pages.c.blocks + row / pages.c.block) * pages.p.h_kv + g);
        __syncwarp();
        mbar_arrive_copies(&full[st]);
        const int per = ROWS / box;  // boxes of the half
        const int src = step == 2 ? 0 : h * per + (lane < per ? lane : 0);
        const int pg = __shfl_sync(0xffffffffu, pages.page, src), r0 = __shfl_sync(0xffffffffu, pages.row, src) + (step == 2 ? 64 * h : 0);
        if (lane < per) tma_load_4d(&rows[st][lane * box * D], &map, &full[st], 0, g, r0, pg);
        ++n;
        return true;
    }
    // Every load still in flight lands.
    __device__ __forceinline__ void drain(uint32_t n) {
        for (uint32_t back = 1; back <= UNITS && back <= n; ++back) mbar_wait_quiet(&full[(n - back) % UNITS], ((n - back) / UNITS) & 1);
    }
    // Rows 16 w and on of the next unit, keys j0 + 16 w and on, to rows of a tile (zeros outside the keys [lo, hi] that
    // any query sees: what lies there may be anything).  The unit's eight 16-byte chunks of a store
    // phase fall into different banks: every other group of four chunks stores its second half first.
    template <bool F16>
    __device__ __forceinline__ bool widen(uint32_t& n, int w, uint8_t* tile, int chunk_bytes, int j0, int lo, int hi, const Abort& ab) {
        const int lane = threadIdx.x & 31, st = n % UNITS;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (n / UNITS) & 1, ab))) return false;
        const float f = scale[st][w];
#pragma unroll 2
        for (int y = 0; y < CPR / 2; ++y) {
            const int x = lane + 32 * y, r = 16 * w + x / CPR, c = x % CPR, j = j0 + r;
            const uint4 b = *reinterpret_cast<const uint4*>(&rows[st][r * D + 16 * c]);
            uint4 o0 = make_uint4(0, 0, 0, 0), o1 = o0;
            if (j >= lo && j <= hi) {
                o0 = make_uint4(scaled_e4m3x2<F16, false>(b.x, f), scaled_e4m3x2<F16, true>(b.x, f), scaled_e4m3x2<F16, false>(b.y, f),
                                scaled_e4m3x2<F16, true>(b.y, f));
                o1 = make_uint4(scaled_e4m3x2<F16, false>(b.z, f), scaled_e4m3x2<F16, true>(b.z, f), scaled_e4m3x2<F16, false>(b.w, f),
                                scaled_e4m3x2<F16, true>(b.w, f));
            }
            uint8_t* to = tile + (c >> 2) * chunk_bytes + r * 128;
            const int u = 2 * (c & 3), swap = (c >> 2) & 1;
            *reinterpret_cast<uint4*>(to + (((u + swap) ^ (r & 7)) << 4)) = swap ? o1 : o0;
            *reinterpret_cast<uint4*>(to + (((u + 1 - swap) ^ (r & 7)) << 4)) = swap ? o0 : o1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        ++n;
        return true;
    }
};

}  // namespace fa
