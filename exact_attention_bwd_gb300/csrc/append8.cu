// Append of rotated keys and of values to an e4m3 paged cache (include/fa.h, fa_qk_norm_rope_append8).
//
// A block of the cache is `block` rows of a page, of one head; it has one scale, and its rows stand
// for byte * scale.  For each block that new tokens fall into:
//   amax = max |x| over the new rows,  need = the smallest power of two with amax <= 448 need,
//   s = max(s_old, need)  (s_old = 0 where the block's first row is a new one),
//   new rows: e4m3(x / s),  rows ahead of them where s grew: e4m3(byte s_old / s).
// The scale is a power of two so that neither division rounds: a new row is rounded once, to e4m3, and
// an older one again only where it falls below e4m3's normal range.  (Scales of another kind that the
// caller put there are kept while they suffice; x / s is then x times the reciprocal, within 2^-23, ahead of the rounding.)
//
// x is rotated in fp32 and its block's maximum is known only behind the last of its rows, so a warp keeps
// its first kKeep batches of rows in registers; what larger blocks have beyond is read, and turned, a second time.
// One CTA to a block and head, half of its warps on the keys and half on the values: what
// a decode step costs is one chain of loads (lengths, table, row), and a chunk has as many CTAs as blocks
// and heads.  The queries' rotation is the kernel of rope.cu, launched ahead; this one's CTAs start where that one's
// leave registers, most of them behind it.
//
// Measured, 8192 tokens in chunks, 16 / 2 heads of 256, blocks of 16 rows: 43 us with the queries' rotation (24 at
// the copy rate), 17 of them this kernel.  It is bound by its chains (issue slots 28 %, DRAM 11 %).  One batch kept 45.9,
// four 57.8 (registers).  A decode step of 32 tokens: 10.3 us on the device, with the queries' kernel.
#include "rope.cuh"

namespace fa {
namespace {

constexpr int kSideWarps = 4;  // warps on a block's keys, and on its values
constexpr int kThreads8 = 2 * 32 * kSideWarps;
constexpr int kKeep = 2;

// The sequence of unit u and its first unit: sequence b has the units from cu[b] / block + 2 b
// on, of which those behind its last block are idle (n tokens touch n / block + 2 blocks at most, and
// each sequence has as many units).  Units ahead of all sequences' (rows of no sequence come first) are given
// to sequence 0 with first > u, and are idle too; offsets that decrease can do the same.  Warp-wide.
__device__ __forceinline__ int unit_sequence(const Append8Args& a, int u, int& first) {
    const int lane = threadIdx.x & 31;
    auto start = [&](int b) { return quotient(min(max(a.cu[b], 0), a.T), a.by_block) + 2 * b; };
    int lo = 0, hi = a.B - 1;
#pragma unroll 1
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const bool le = at <= hi && start(at) <= u;
        lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
        hi = min(hi, lo + step - 1);
    }
    first = start(lo);
    return lo;
}

// The smallest power of two s >= 2^-126 with amax <= 448 s = 1.75 * 2^8 s.
__device__ __forceinline__ float block_scale(float amax) {
    const uint32_t x = __float_as_uint(amax), e = (x >> 23) + ((x & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((e > 9 ? e - 8 : 1) << 23);
}

// The angles of a lane's 16 values at the token's positions (pos[x]: of axis x), from the tables.
template <bool ADJ>
__device__ __forceinline__ void load_angles(const RopeArgs& a, const int* pos, int u0, int u1, Angles<ADJ>& ang) {
    const int half = a.rot / 2;
    if (a.axes <= 1) {  // a row of the tables
        const long row = (long)pos[0] * half;
        ang.load(a.cos + row, a.sin + row, u0, u1, a.rot);
        return;
    }
    auto at = [&](int j, float& c, float& s) {
        const int x = a.pair_axis[j];
        const int p = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
        c = a.cos[(long)p * half + j];
        s = a.sin[(long)p * half + j];
    };
    if constexpr (ADJ) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int u = e < 4 ? u0 : u1;
            float c = 1.f, s = 0.f;
            if (8 * u < a.rot) at(4 * u + (e & 3), c, s);
            ang.c[e] = make_float2(c, c);
            ang.s[e] = make_float2(-s, s);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float c0 = 1.f, s0 = 0.f, c1 = 1.f, s1 = 0.f;
            if (16 * u0 < a.rot) {
                at(8 * u0 + 2 * e, c0, s0);
                at(8 * u0 + 2 * e + 1, c1, s1);
            }
            ang.c[e] = make_float2(c0, c1);
            ang.s[e] = make_float2(s0, s1);
        }
    }
}

template <int D, bool F16, bool ADJ>
__device__ __forceinline__ void append8_block(const RopeArgs& a, const Append8Args& c, float* amax_of) {
    using C = RowCfg<D>;
    constexpr int LANES = C::LANES, ROWS = C::ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % LANES, lr = lane / LANES;
    const bool on = li < C::PAIRS;
    const int side = warp / kSideWarps, w = warp % kSideWarps, head = blockIdx.y;  // side 0: keys, 1: values
    // ---- the block: rows [r0, r1) of page `page` are new, r1 - r0 tokens from t0 on ----
    int first;
    const int u = blockIdx.x, b = unit_sequence(c, u, first);
    const int q0 = min(max(c.cu[b], 0), c.T), n = min(max(c.cu[b + 1], q0), c.T) - q0;
    const int total = c.used[b], start = total - n;  // places [start, total) in the sequence
    const int limit = c.max_blocks * c.page_size, from = max(start, 0), to = min(total, limit);
    if (n > 0 && (start < 0 || total > limit) && u == first && threadIdx.x == 0 && head == 0 && a.status)
        atomicCAS(a.status, 0, kStatusDeviceCheck);
    const long at_block = (long)quotient(from, c.by_block) + (u - first);
    if (u < first || n <= 0 || at_block * c.block >= to) return;  // (the one branch on all that was loaded)
    const int place = (int)at_block * c.block;  // of the block's first row
    const int nth = quotient(place, c.by_page), page = c.table[(long)b * c.max_blocks + nth];
    if ((unsigned)page >= (unsigned)c.num_pages) {
        if (threadIdx.x == 0 && head == 0 && a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
        return;
    }
    const int in_page = place - nth * c.page_size;
    const int r0 = max(from - place, 0), r1 = min(to - place, c.block);  // new rows of the block
    const int t0 = q0 + place - start;                                    // the token of the block's row 0
    uint8_t* rows8 = (side ? c.v_cache : c.k_cache) + (((long)page * c.page_size + in_page) * a.h_kv + head) * D;
    const long row_step = (long)a.h_kv * D;
    float* scale_at = (side ? c.v_scale : c.k_scale) + ((long)page * quotient(c.page_size, c.by_block) + quotient(in_page, c.by_block)) * a.h_kv + head;
    const uint16_t* src = (side ? a.v : a.k) + (long)head * D;
    const long src_step = side ? a.v_stride : a.k_stride;
    int u0, u1;
    lane_units<D, ADJ>(on ? li : 0, a.rot, u0, u1);
    float2 weight[8];
    load_weight<F16>(a, side ? nullptr : a.wk, u0, u1, weight);
    // the lane's values of row r (zeros and false for a token that is not stored)
    auto row_of = [&](int r, float2* v) {
        const long t = t0 + r;
        int pos[FA_ROPE_MAX_AXES] = {0, 0, 0, 0};
        bool there = r < r1;
        if (there) {
#pragma unroll
            for (int x = 0; x < FA_ROPE_MAX_AXES; ++x)
                if (x < max(a.axes, 1)) {
                    pos[x] = a.positions[x * (long)a.T + t];
                    if (pos[x] < 0 || pos[x] >= a.max_pos) {
                        if (pos[x] != -1 && a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
                        there = false;
                    }
                }
        }
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (there && on) {
            x0 = *reinterpret_cast<const uint4*>(src + t * src_step + 8 * u0);
            x1 = *reinterpret_cast<const uint4*>(src + t * src_step + 8 * u1);
        }
        widen8<F16>(x0, v);
        widen8<F16>(x1, v + 4);
        if (side == 0) {
            float rs = 1.f;
            if (!a.no_norm) {
                float2 ss = __fmul2_rn(v[0], v[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) ss = __ffma2_rn(v[e], v[e], ss);
                rs = rsqrtf(row_sum<LANES>(ss.x + ss.y) * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __fmul2_rn(v[e], weight[e]);
            }
            if (there) {
                if ((ADJ ? 8 : 16) * u0 < a.rot || (ADJ && 8 * u1 < a.rot)) {
                    Angles<ADJ> ang;
                    load_angles<ADJ>(a, pos, u0, u1, ang);
                    ang.template turn<false, true>(v, (ADJ ? 8 : 16) * u0 < a.rot, 8 * u1 < a.rot);
                }
                if (!a.no_norm) {
                    const float2 rs2 = make_float2(rs, rs);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __fmul2_rn(v[e], rs2);
                }
            }
        }
        return there;
    };
    // ---- the largest finite value (infinities are stored as the block's largest, NaN, which a maximum passes over, as NaN) ----
    float amax = -1.f;  // (no row)
    auto most_of = [&](bool there, const float2* v) {
        if (there && on) {
            float top = 0.f, x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fabsf(e & 1 ? v[e / 2].y : v[e / 2].x);
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, x[e]);
            if (top == INFINITY) {
                top = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (x[e] < INFINITY) top = fmaxf(top, x[e]);
            }
            amax = fmaxf(amax, top);
        }
    };
    constexpr int STEP = kSideWarps * ROWS;
    const int mine = r0 + w * ROWS + lr;  // the lane's first row
    float2 kept[kKeep][8];
    bool there[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        there[k] = mine - lr + k * STEP < r1 && row_of(mine + k * STEP, kept[k]);
        most_of(there[k], kept[k]);
    }
#pragma unroll 1
    for (int r = mine + kKeep * STEP; r < r1 + lr; r += STEP) {
        float2 v[8];
        const bool y = row_of(r, v);
        most_of(y, v);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) amax_of[warp] = amax;
    float old = 0.f;
    if (place < from) old = *scale_at;
    if (!(old > 0.f && old < INFINITY)) old = 0.f;  // no scale yet
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSideWarps; ++x) amax = fmaxf(amax, amax_of[side * kSideWarps + x]);
    if (amax < 0.f) return;  // no token to store
    const float s = fmaxf(old, block_scale(amax)), inv = 1.f / s;
    if (w == 0 && lane == 0) *scale_at = s;  // (every warp has read it)
    // ---- the rows ahead of the new ones, where the scale grew ----
    if (place < from && s > old) {
        const float f = old * inv;
        for (int x = w * 32 + lane; x < r0 * (D / 4); x += 32 * kSideWarps) {
            uint32_t* y = reinterpret_cast<uint32_t*>(rows8 + (x / (D / 4)) * row_step) + x % (D / 4);
            float z[4];
            unpack_e4m3x4(*y, z);
            *y = pack_e4m3x4(z[0] * f, z[1] * f, z[2] * f, z[3] * f);
        }
    }
    // ---- the new rows ----
    auto store = [&](int r, const float2* v) {
        uint8_t* out = rows8 + r * row_step;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2* x = v + 4 * h;
            *reinterpret_cast<uint2*>(out + 8 * (h ? u1 : u0)) =
                make_uint2(pack_e4m3x4(x[0].x * inv, x[0].y * inv, x[1].x * inv, x[1].y * inv),
                           pack_e4m3x4(x[2].x * inv, x[2].y * inv, x[3].x * inv, x[3].y * inv));
        }
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
        if (there[k] && on) store(mine + k * STEP, kept[k]);
#pragma unroll 1
    for (int r = mine + kKeep * STEP; r < r1 + lr; r += STEP) {
        float2 v[8];
        if (row_of(r, v) && on) store(r, v);
    }
}

template <int D, bool F16, bool ADJ>
__global__ void __launch_bounds__(kThreads8) append8_kernel(const RopeArgs a, const Append8Args c) {
    __shared__ float amax_of[2 * kSideWarps];
    append8_block<D, F16, ADJ>(a, c, amax_of);
    if (blockIdx.x == 0 && blockIdx.y == 0 && a.status) {  // (where offsets decrease the search may miss a sequence)
        bool bad = false;
        for (int b = threadIdx.x; b < c.B; b += kThreads8) bad |= min(max(c.cu[b + 1], 0), c.T) < min(max(c.cu[b], 0), c.T);
        if (bad) atomicCAS(a.status, 0, kStatusDeviceCheck);
    }
    wait_previous_kernel();  // (what comes next in the stream waits for both)
}

template <int D, bool F16>
cudaError_t launch_df(const RopeArgs& a, const Append8Args& c, const dim3& grid, cudaStream_t st) {
    return launch_after(a.adjacent ? append8_kernel<D, F16, true> : append8_kernel<D, F16, false>, grid, kThreads8, 0, st, a, c);
}
template <int D>
cudaError_t launch_d(const RopeArgs& a, const Append8Args& c, const dim3& grid, cudaStream_t st) {
    return a.f16 ? launch_df<D, true>(a, c, grid, st) : launch_df<D, false>(a, c, grid, st);
}

}  // namespace

cudaError_t launch_append8(const RopeArgs& a, const Append8Args& c, cudaStream_t st) {
    if (c.B == 0 || c.T == 0) return cudaSuccess;
    const dim3 grid((unsigned)(c.T / c.block + 2 * c.B), (unsigned)a.h_kv);
    switch (a.d) {
        case 64: return launch_d<64>(a, c, grid, st);
        case 128: return launch_d<128>(a, c, grid, st);
        case 192: return launch_d<192>(a, c, grid, st);
        case 256: return launch_d<256>(a, c, grid, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
